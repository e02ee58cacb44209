// The linear layer with its epilogue, and its backward pass:
//
//   z = x W^T + b,  y = act(z) + residual
//   dz = dy act'(z),  db = sum_t dz_t,  dW = dz^T x,  dx = dz W
//
// Three forms of the product:
//   linear_rows_kernel    few tokens (one sequence being extended): bound by reading W once.  A warp
//                         holds four output rows of W against every token, 16 bytes a lane; where
//                         there are few output rows the warps of a CTA split the contraction.
//   linear_gemm_kernel    tcgen05 GEMM, persistent and warp-specialised: one warp feeds a TMA ring, one
//                         thread issues the MMAs of a 128-token tile into one of two accumulators in
//                         tensor memory, eight warps run the epilogue of the previous tile from the other.
//                         B is W [d_out, d_in], K-major in the forward product and MN-major in dx.
//   the contraction of dust_wgrad.cu for dW.
// dz is formed once (linear_dz_kernel) as a bf16 operand, or as hi + lo bf16 terms (dz = hi + lo to
// about 16 bits), with the column sums for db on the way.
#include <algorithm>

#include "dust_device.cuh"
#include "dust_internal.h"

namespace dust {
namespace {

// ------------------------------------------------------------------ activations
// GELU's tanh form and SiLU are z p with the logistic function p = 1 / (1 + exp(-u)): u = z for SiLU,
// u = 2 sqrt(2/pi) (z + 0.044715 z^3) for the tanh form (1 + tanh(u/2) = 2 p).
constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.07135481282553578f;  // 0.044715 * 2 sqrt(2 / pi)
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

__device__ __forceinline__ float logistic(float u) { return __fdividef(1.0f, 1.0f + __expf(-u)); }

template <int kAct>
__device__ __forceinline__ float act_fn(float z) {
    if (kAct == DUST_ACT_RELU) return z <= 0.f ? 0.f : z;  // keeps a NaN
    if (kAct == DUST_ACT_GELU) return 0.5f * z * (1.0f + erff(z * kSqrtHalf));
    if (kAct == DUST_ACT_GELU_TANH) return z * logistic(z * fmaf(kGeluB, z * z, kGeluA));
    if (kAct == DUST_ACT_SILU) return z * logistic(z);
    return z;
}
// Far from zero the slope's second term is 0 times something that may have overflowed: it is dropped.
template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
    if (kAct == DUST_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (kAct == DUST_ACT_GELU) {
        const float cdf = 0.5f * (1.0f + erff(z * kSqrtHalf)), e = __expf(-0.5f * z * z);
        return e == 0.f ? cdf : fmaf(z * kInvSqrt2Pi, e, cdf);
    }
    if (kAct == DUST_ACT_GELU_TANH) {
        const float z2 = z * z;
        const float p = logistic(z * fmaf(kGeluB, z2, kGeluA)), pq = p * (1.0f - p);
        return pq == 0.f ? p : fmaf(pq, z * fmaf(3.0f * kGeluB, z2, kGeluA), p);
    }
    if (kAct == DUST_ACT_SILU) {
        const float p = logistic(z), pq = p * (1.0f - p);
        return pq == 0.f ? p : fmaf(pq, z, p);
    }
    return 1.f;
}
__device__ __forceinline__ float act_any(int act, float z) {
    switch (act) {
        case DUST_ACT_RELU: return act_fn<DUST_ACT_RELU>(z);
        case DUST_ACT_GELU: return act_fn<DUST_ACT_GELU>(z);
        case DUST_ACT_GELU_TANH: return act_fn<DUST_ACT_GELU_TANH>(z);
        case DUST_ACT_SILU: return act_fn<DUST_ACT_SILU>(z);
    }
    return z;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// ------------------------------------------------------------------ few tokens
constexpr int kRThreads = 256;
constexpr int kRWarps = kRThreads / 32;
constexpr int kRRows = 4;  // output rows a warp holds

struct RowsArgs {
    const __nv_bfloat16* x;
    const __nv_bfloat16* W;
    const float* bias;
    const void* res;
    void* y;
    __nv_bfloat16* z;
    int64_t ld_x, ld_res, ld_y, ld_z;
    int N, d_in, d_out, act, out_bf16;
    int split;  // warps of a CTA that share four output rows (1, 2, 4 or 8)
};

template <int kTok>
__global__ void __launch_bounds__(kRThreads) linear_rows_kernel(const __grid_constant__ RowsArgs A) {
    __shared__ float part[kRWarps][kRRows * kTok];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / A.split, share = warp % A.split;
    const int o0 = (blockIdx.x * (kRWarps / A.split) + group) * kRRows;
    float acc[kRRows][kTok] = {};
    // d_out is a multiple of 16, so the four rows are inside or outside together
    if (o0 < A.d_out) {
        const uint4* w[kRRows];
#pragma unroll
        for (int r = 0; r < kRRows; ++r)
            w[r] = reinterpret_cast<const uint4*>(A.W + static_cast<int64_t>(o0 + r) * A.d_in);
        const int nv = A.d_in >> 3;
#pragma unroll 2
        for (int v = share * 32 + lane; v < nv; v += A.split * 32) {
            uint4 ww[kRRows];
#pragma unroll
            for (int r = 0; r < kRRows; ++r) ww[r] = __ldg(w[r] + v);
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                if (t >= A.N) break;
                const uint4 xx = __ldg(reinterpret_cast<const uint4*>(A.x + t * A.ld_x) + v);
                const float xf[8] = {bf_lo(xx.x), bf_hi(xx.x), bf_lo(xx.y), bf_hi(xx.y),
                                     bf_lo(xx.z), bf_hi(xx.z), bf_lo(xx.w), bf_hi(xx.w)};
#pragma unroll
                for (int r = 0; r < kRRows; ++r) {
                    float a = acc[r][t];
                    a = fmaf(bf_lo(ww[r].x), xf[0], a);
                    a = fmaf(bf_hi(ww[r].x), xf[1], a);
                    a = fmaf(bf_lo(ww[r].y), xf[2], a);
                    a = fmaf(bf_hi(ww[r].y), xf[3], a);
                    a = fmaf(bf_lo(ww[r].z), xf[4], a);
                    a = fmaf(bf_hi(ww[r].z), xf[5], a);
                    a = fmaf(bf_lo(ww[r].w), xf[6], a);
                    a = fmaf(bf_hi(ww[r].w), xf[7], a);
                    acc[r][t] = a;
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRRows; ++r)
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            float a = acc[r][t];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            if (lane == 0) part[warp][r * kTok + t] = a;
        }
    __syncthreads();
    if (share != 0 || o0 >= A.d_out) return;
    for (int e = lane; e < kRRows * kTok; e += 32) {
        const int r = e / kTok, t = e % kTok;
        if (t >= A.N) continue;
        float a = 0.f;
        for (int k = 0; k < A.split; ++k) a += part[warp + k][e];
        const int o = o0 + r;
        if (A.bias) a += __ldg(A.bias + o);
        if (A.z) A.z[t * A.ld_z + o] = __float2bfloat16_rn(a);
        float v = act_any(A.act, a);
        if (A.out_bf16) {
            if (A.res) v += __bfloat162float(static_cast<const __nv_bfloat16*>(A.res)[t * A.ld_res + o]);
            static_cast<__nv_bfloat16*>(A.y)[t * A.ld_y + o] = __float2bfloat16_rn(v);
        } else {
            if (A.res) v += static_cast<const float*>(A.res)[t * A.ld_res + o];
            static_cast<float*>(A.y)[t * A.ld_y + o] = v;
        }
    }
}

// ------------------------------------------------------------------ tensor-core GEMM
constexpr int kBM = 128;
constexpr int kBK = 64;
constexpr int kThreads = 320;  // TMA warp, MMA warp, eight epilogue warps
constexpr uint32_t kABytes = kBM * kBK * 2;

template <int kBN>
struct Shape {
    static constexpr uint32_t kBBytes = kBN * kBK * 2;
    static constexpr uint32_t kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = kBN == 256 ? 4 : kBN == 128 ? 6 : 8;
    static constexpr uint32_t kSmem = kStages * kStageBytes + 1024 + 256;
    static constexpr uint32_t kTmemCols = 2 * kBN;
};

struct GemmArgs {
    CUtensorMap ta;  // A [terms M, K], 64 x 128 boxes
    CUtensorMap tb;  // K-major: B [n_out, K], 64 x kBN boxes; MN-major: B [K, n_out], 64 x 64 boxes
    const float* bias;
    const void* res;
    void* y;
    __nv_bfloat16* z;
    ErrorWord* ew;
    int64_t M, ld_res, ld_y, ld_z;
    int n_out, k_blocks, terms, m_tiles, n_tiles, out_bf16;
};

template <int kBN, bool kBmn, int kAct>
__global__ void __launch_bounds__(kThreads, 1) linear_gemm_kernel(const __grid_constant__ GemmArgs A) {
    using S = Shape<kBN>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * S::kStageBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;   // [2]
    uint64_t* acc_empty = acc_full + 2;     // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_tiles = A.m_tiles * A.n_tiles;
    const int nk = A.k_blocks * A.terms;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);  // one arrival per epilogue warp
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tensormap(&A.ta);
            prefetch_tensormap(&A.tb);
            uint32_t kc = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
                const int m0 = tile % A.m_tiles * kBM;
                const int n0 = tile / A.m_tiles * kBN;
                for (int kb = 0; kb < nk; ++kb, ++kc) {
                    const int s = kc % kStages;
                    if (kc >= kStages &&
                        !mbar_wait_bounded(&empty[s], ((kc / kStages) - 1) & 1, A.ew, 501)) {
                        ok = false;
                        break;
                    }
                    uint8_t* a = smem + s * S::kStageBytes;
                    // the second term's rows follow the first's; B starts over with each term
                    const int term = kb >= A.k_blocks ? 1 : 0;
                    const int k0 = (kb - term * A.k_blocks) * kBK;
                    mbar_arrive_expect_tx(&full[s], S::kStageBytes);
                    tma_load_2d(a, &A.ta, &full[s], k0, m0 + (term ? static_cast<int32_t>(A.M) : 0));
                    if (kBmn) {
#pragma unroll
                        for (int j = 0; j < kBN / 64; ++j)
                            tma_load_2d(a + kABytes + j * (kBK * 128), &A.tb, &full[s], n0 + 64 * j, k0);
                    } else {
                        tma_load_2d(a + kABytes, &A.tb, &full[s], k0, n0);
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(kBM, kBN, 0, kBmn ? 1 : 0);
            uint32_t kc = 0;
            int lt = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x, ++lt) {
                const int buf = lt & 1;
                // the epilogue of the tile that last used this accumulator has read it
                if (lt >= 2 && !mbar_wait_bounded(&acc_empty[buf], ((lt >> 1) - 1) & 1, A.ew, 502)) break;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(buf * kBN);
                for (int kb = 0; kb < nk; ++kb, ++kc) {
                    const int s = kc % kStages;
                    if (!mbar_wait_bounded(&full[s], (kc / kStages) & 1, A.ew, 503)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(smem + s * S::kStageBytes);
                    const uint32_t b_addr = a_addr + kABytes;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        const uint64_t ad = sdesc_sw128(a_addr + kk * 32, 16, 1024);
                        // MN-major: 16 contraction rows of 128 bytes per instruction, 8-row groups 1024
                        // bytes apart, 64-column boxes kBK * 128 bytes apart
                        const uint64_t bd = kBmn ? sdesc_sw128(b_addr + kk * 2048, kBK * 128, 1024)
                                                 : sdesc_sw128(b_addr + kk * 32, 16, 1024);
                        umma_bf16(d, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
                    }
                    umma_commit(&empty[s]);
                }
                umma_commit(&acc_full[buf]);
            }
        }
    } else {
        // epilogue warps 2 .. 9: tensor-memory lane quarter warp % 4, column half hf
        const int q = warp & 3;
        const int hf = (warp - 2) >> 2;
        int lt = 0;
        for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x, ++lt) {
            const int buf = lt & 1;
            const int n0 = tile / A.m_tiles * kBN;
            if (!mbar_wait_bounded(&acc_full[buf], (lt >> 1) & 1, A.ew, 504)) break;
            __syncwarp();
            tc_fence_after();
            const int64_t t = static_cast<int64_t>(tile % A.m_tiles) * kBM + q * 32 + lane;
            const bool valid = t < A.M;
            const uint32_t trow = tmem + static_cast<uint32_t>(buf * kBN) + (static_cast<uint32_t>(q * 32) << 16);
            const int nchunks = min(kBN, A.n_out - n0) / 16;
            const int c_end = min(nchunks, (hf + 1) * (kBN / 32));
            for (int c = hf * (kBN / 32); c < c_end; ++c) {
                float v[16];
                tmem_ld16(trow + c * 16, v);
                tmem_wait_ld();
                if (!valid) continue;
                const int o = n0 + c * 16;
                if (A.bias) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 b = __ldg(reinterpret_cast<const float4*>(A.bias + o) + j);
                        v[4 * j] += b.x;
                        v[4 * j + 1] += b.y;
                        v[4 * j + 2] += b.z;
                        v[4 * j + 3] += b.w;
                    }
                }
                if (A.z) {
                    uint4* zp = reinterpret_cast<uint4*>(A.z + t * A.ld_z + o);
                    zp[0] = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
                    zp[1] = make_uint4(pack2(v[8], v[9]), pack2(v[10], v[11]), pack2(v[12], v[13]), pack2(v[14], v[15]));
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = act_fn<kAct>(v[j]);
                if (A.out_bf16) {
                    if (A.res) {
                        const uint4* rp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(A.res) +
                                                                         t * A.ld_res + o);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 r = rp[h];
                            const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                v[8 * h + 2 * j] += bf_lo(rw[j]);
                                v[8 * h + 2 * j + 1] += bf_hi(rw[j]);
                            }
                        }
                    }
                    uint4* yp = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(A.y) + t * A.ld_y + o);
                    yp[0] = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
                    yp[1] = make_uint4(pack2(v[8], v[9]), pack2(v[10], v[11]), pack2(v[12], v[13]), pack2(v[14], v[15]));
                } else {
                    if (A.res) {
                        const float4* rp = reinterpret_cast<const float4*>(static_cast<const float*>(A.res) +
                                                                           t * A.ld_res + o);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 r = rp[j];
                            v[4 * j] += r.x;
                            v[4 * j + 1] += r.y;
                            v[4 * j + 2] += r.z;
                            v[4 * j + 3] += r.w;
                        }
                    }
                    float4* yp = reinterpret_cast<float4*>(static_cast<float*>(A.y) + t * A.ld_y + o);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        yp[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                }
            }
            // the accumulator may be refilled once every epilogue warp has read it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, S::kTmemCols);
}

// ------------------------------------------------------------------ dz and its column sums
constexpr int kDThreads = 256;
constexpr int kDWarps = kDThreads / 32;
constexpr int kDCols = 256;  // 32 lanes x 8 columns
constexpr int kDRows = 256;  // rows of one partial sum

struct DzArgs {
    const void* dy;
    const __nv_bfloat16* z;
    __nv_bfloat16* hi;  // [N, d_out], or null (dy itself is the operand)
    __nv_bfloat16* lo;  // [N, d_out], or null
    float* part;        // [row chunks, d_out] column sums, or null
    int64_t N, ld_dy, ld_z;
    int d_out;
};

template <typename T, int kAct>
__global__ void __launch_bounds__(kDThreads) linear_dz_kernel(const __grid_constant__ DzArgs A) {
    __shared__ float sh[kDWarps][kDCols + 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * kDCols + lane * 8;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kDRows;
    const int64_t r1 = min(A.N, r0 + kDRows);
    float s[8] = {};
    if (col < A.d_out) {
#pragma unroll 2
        for (int64_t t = r0 + warp; t < r1; t += kDWarps) {
            float g[8];
            if (sizeof(T) == 2) {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(A.dy) + t * A.ld_dy + col));
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    g[2 * j] = bf_lo(ww[j]);
                    g[2 * j + 1] = bf_hi(ww[j]);
                }
            } else {
                const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(A.dy) + t * A.ld_dy + col);
                const float4 a = __ldg(p), b = __ldg(p + 1);
                g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w;
                g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
            }
            if (kAct != DUST_ACT_NONE) {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(A.z + t * A.ld_z + col));
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    g[2 * j] *= act_slope<kAct>(bf_lo(ww[j]));
                    g[2 * j + 1] *= act_slope<kAct>(bf_hi(ww[j]));
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += g[j];
            if (A.hi) {
                uint32_t h[4], l[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = pack2(g[2 * j], g[2 * j + 1]);
                    // the remainder is exact in fp32
                    l[j] = pack2(g[2 * j] - bf_lo(h[j]), g[2 * j + 1] - bf_hi(h[j]));
                }
                const int64_t at = t * A.d_out + col;
                *reinterpret_cast<uint4*>(A.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
                if (A.lo) *reinterpret_cast<uint4*>(A.lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
    }
    if (!A.part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) sh[warp][lane * 8 + j] = s[j];
    __syncthreads();
    const int c = blockIdx.x * kDCols + threadIdx.x;
    if (c < A.d_out) {
        float a = 0.f;
        for (int w = 0; w < kDWarps; ++w) a += sh[w][threadIdx.x];
        A.part[static_cast<int64_t>(blockIdx.y) * A.d_out + c] = a;
    }
}

// db (+)= the partial sums: 32 columns a CTA, its eight warps over consecutive runs of chunks.
__global__ void __launch_bounds__(256) linear_db_kernel(const float* part, int chunks, int d_out, float* db,
                                                        int accumulate) {
    __shared__ float sh[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    const int per = (chunks + 7) / 8;
    const int a = warp * per, b = min(chunks, a + per);
    float s = 0.f;
    if (c < d_out) {
#pragma unroll 4
        for (int k = a; k < b; ++k) s += __ldg(part + static_cast<int64_t>(k) * d_out + c);
    }
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < d_out) {
        for (int w = 1; w < 8; ++w) s += sh[w][lane];
        db[c] = accumulate ? db[c] + s : s;
    }
}

// ------------------------------------------------------------------ host side
template <int kBN, bool kBmn, int kAct>
dust_status launch_gemm(const GemmArgs& A, cudaStream_t s) {
    static PerContextOnce attr;
    if (!attr.run([] {
            return cudaFuncSetAttribute(linear_gemm_kernel<kBN, kBmn, kAct>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(Shape<kBN>::kSmem)) == cudaSuccess;
        }))
        return DUST_ERR_CUDA;
    const int64_t tiles = static_cast<int64_t>(A.m_tiles) * A.n_tiles;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, num_sms()));
    linear_gemm_kernel<kBN, kBmn, kAct><<<grid, kThreads, Shape<kBN>::kSmem, s>>>(A);
    return DUST_OK;
}

template <int kBN>
dust_status launch_fwd(const GemmArgs& A, int act, cudaStream_t s) {
    switch (act) {
        case DUST_ACT_RELU: return launch_gemm<kBN, false, DUST_ACT_RELU>(A, s);
        case DUST_ACT_GELU: return launch_gemm<kBN, false, DUST_ACT_GELU>(A, s);
        case DUST_ACT_GELU_TANH: return launch_gemm<kBN, false, DUST_ACT_GELU_TANH>(A, s);
        case DUST_ACT_SILU: return launch_gemm<kBN, false, DUST_ACT_SILU>(A, s);
    }
    return launch_gemm<kBN, false, DUST_ACT_NONE>(A, s);
}

// Output tile width: the one whose waves of tiles over the SMs cost least, a tile of 128 x bn taking
// about as long as the larger of its MMAs (bn) and its operand loads (bn + 128, at 0.6 each).
int choose_bn(int64_t m_tiles, int n_out) {
    int best = 256;
    double least = 0;
    for (int bn : {256, 128, 64}) {
        const int64_t tiles = m_tiles * ((n_out + bn - 1) / bn);
        const double cost = static_cast<double>((tiles + num_sms() - 1) / num_sms()) *
                            std::max<double>(bn, 0.6 * (bn + 128));
        if (bn == 256 || cost < least) {
            least = cost;
            best = bn;
        }
    }
    return best;
}

// y [M, n_out] = A [terms M, K] B, B K-major [n_out, K] or MN-major [K, n_out].
dust_status gemm(const void* a, int64_t ld_a, int terms, int64_t M, int K, const void* b, bool b_mn, int n_out,
                 GemmArgs& G, int act, const char* name, cudaStream_t s) {
    const int64_t m_tiles = (M + kBM - 1) / kBM;
    const int bn = choose_bn(m_tiles, n_out);
    G.ew = device_error_word();
    G.M = M;
    G.n_out = n_out;
    G.k_blocks = (K + kBK - 1) / kBK;
    G.terms = terms;
    G.n_tiles = (n_out + bn - 1) / bn;
    if (m_tiles * G.n_tiles > 2147483647LL) return DUST_ERR_UNSUPPORTED;
    G.m_tiles = static_cast<int>(m_tiles);
    if (!make_tmap_bf16_2d_ld(&G.ta, a, static_cast<uint64_t>(terms * M), K, ld_a, kBM, kBK)) return DUST_ERR_CUDA;
    if (b_mn ? !make_tmap_bf16_2d_ld(&G.tb, b, K, n_out, n_out, kBK, 64)
             : !make_tmap_bf16_2d_ld(&G.tb, b, n_out, K, K, bn, kBK))
        return DUST_ERR_CUDA;
    prof_begin(s);
    dust_status st;
    if (b_mn)
        st = bn == 256   ? launch_gemm<256, true, DUST_ACT_NONE>(G, s)
             : bn == 128 ? launch_gemm<128, true, DUST_ACT_NONE>(G, s)
                         : launch_gemm<64, true, DUST_ACT_NONE>(G, s);
    else
        st = bn == 256 ? launch_fwd<256>(G, act, s) : bn == 128 ? launch_fwd<128>(G, act, s) : launch_fwd<64>(G, act, s);
    prof_end(s, name);
    return st;
}

template <typename T>
void launch_dz(const DzArgs& A, int act, dim3 grid, cudaStream_t s) {
    switch (act) {
        case DUST_ACT_RELU: linear_dz_kernel<T, DUST_ACT_RELU><<<grid, kDThreads, 0, s>>>(A); return;
        case DUST_ACT_GELU: linear_dz_kernel<T, DUST_ACT_GELU><<<grid, kDThreads, 0, s>>>(A); return;
        case DUST_ACT_GELU_TANH: linear_dz_kernel<T, DUST_ACT_GELU_TANH><<<grid, kDThreads, 0, s>>>(A); return;
        case DUST_ACT_SILU: linear_dz_kernel<T, DUST_ACT_SILU><<<grid, kDThreads, 0, s>>>(A); return;
    }
    linear_dz_kernel<T, DUST_ACT_NONE><<<grid, kDThreads, 0, s>>>(A);
}

size_t dz_bytes(int64_t N, int32_t d_out) { return align_up(static_cast<size_t>(2 * N) * d_out * 2, 256); }
size_t db_bytes(int64_t N, int32_t d_out) {
    return align_up(static_cast<size_t>((N + kDRows - 1) / kDRows) * d_out * 4, 256);
}

// Tokens up to which W is streamed through the CUDA cores.
constexpr int kFewTokens = 8;

template <int kTok>
void launch_rows(const RowsArgs& A, unsigned blocks, cudaStream_t s) {
    linear_rows_kernel<kTok><<<blocks, kRThreads, 0, s>>>(A);
}

}  // namespace

dust_status linear_launch(const void* x, int64_t ld_x, const void* W, const float* bias, int act, const void* res,
                          int64_t ld_res, int64_t N, int32_t d_in, int32_t d_out, void* y, int out_bf16,
                          int64_t ld_y, void* z, int64_t ld_z, cudaStream_t s) {
    if (N <= kFewTokens) {
        RowsArgs A{static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(W), bias, res, y,
                   static_cast<__nv_bfloat16*>(z), ld_x, ld_res, ld_y, ld_z, static_cast<int>(N), d_in, d_out, act,
                   out_bf16, 1};
        // warps to share four rows: while the SMs have fewer than 16 warps each and a share keeps at
        // least two steps of 256 elements
        const int groups = d_out / kRRows;
        while (A.split < kRWarps && static_cast<int64_t>(groups) * A.split < num_sms() * 16 &&
               d_in / (A.split * 2) >= 512)
            A.split *= 2;
        const int per_cta = kRWarps / A.split;
        const unsigned blocks = static_cast<unsigned>((groups + per_cta - 1) / per_cta);
        prof_begin(s);
        if (N == 1)
            launch_rows<1>(A, blocks, s);
        else if (N == 2)
            launch_rows<2>(A, blocks, s);
        else if (N <= 4)
            launch_rows<4>(A, blocks, s);
        else
            launch_rows<8>(A, blocks, s);
        prof_end(s, "linear_rows");
        return cudaGetLastError() == cudaSuccess ? DUST_OK : DUST_ERR_CUDA;
    }
    GemmArgs G{};
    G.bias = bias;
    G.res = res;
    G.y = y;
    G.z = static_cast<__nv_bfloat16*>(z);
    G.ld_res = ld_res;
    G.ld_y = ld_y;
    G.ld_z = ld_z;
    G.out_bf16 = out_bf16;
    const dust_status st = gemm(x, ld_x, 1, N, d_in, W, false, d_out, G, act, "linear_tcgen05", s);
    if (st != DUST_OK) return st;
    return cudaGetLastError() == cudaSuccess ? DUST_OK : DUST_ERR_CUDA;
}

size_t linear_backward_workspace_bytes(int64_t N, int32_t d_in, int32_t d_out) {
    return dz_bytes(N, d_out) + db_bytes(N, d_out) + contract_workspace_bytes(N, d_in, d_out);
}

dust_status linear_backward_launch(const void* dy, int dy_bf16, int64_t ld_dy, const void* z, int64_t ld_z,
                                   const void* x, int64_t ld_x, const void* W, int act, int64_t N, int32_t d_in,
                                   int32_t d_out, int terms, void* dx, int dx_bf16, int64_t ld_dx, float* dW,
                                   float* db, int accumulate, void* ws, cudaStream_t s) {
    char* w = static_cast<char*>(ws);
    __nv_bfloat16* hi = reinterpret_cast<__nv_bfloat16*>(w);
    float* part = reinterpret_cast<float*>(w + dz_bytes(N, d_out));
    void* split = w + dz_bytes(N, d_out) + db_bytes(N, d_out);
    // without an activation a bf16 dy is the operand itself, exactly, in one term
    const bool direct = act == DUST_ACT_NONE && dy_bf16;
    const bool products = dx || dW;
    if (direct) terms = 1;
    if (db || (products && !direct)) {
        const int chunks = static_cast<int>((N + kDRows - 1) / kDRows);
        DzArgs A{dy, static_cast<const __nv_bfloat16*>(z), nullptr, nullptr, db ? part : nullptr, N, ld_dy, ld_z, d_out};
        if (products && !direct) {
            A.hi = hi;
            A.lo = terms == 2 ? hi + N * d_out : nullptr;
        }
        const dim3 grid((d_out + kDCols - 1) / kDCols, chunks);
        prof_begin(s);
        if (dy_bf16)
            launch_dz<__nv_bfloat16>(A, act, grid, s);
        else
            launch_dz<float>(A, act, grid, s);
        prof_end(s, "linear_dz");
        if (db) {
            prof_begin(s);
            linear_db_kernel<<<(d_out + 31) / 32, 256, 0, s>>>(part, chunks, d_out, db, accumulate);
            prof_end(s, "linear_db");
        }
    }
    const void* op = direct ? dy : hi;
    const int64_t ld_op = direct ? ld_dy : d_out;
    if (dx) {
        GemmArgs G{};
        G.y = dx;
        G.ld_y = ld_dx;
        G.out_bf16 = dx_bf16;
        // a bf16 dx is rounded as coarsely as one term of dz; an fp32 dx takes both terms
        const dust_status st = gemm(op, ld_op, dx_bf16 ? 1 : terms, N, d_out, W, true, d_in, G, DUST_ACT_NONE,
                                    "linear_dx_tcgen05", s);
        if (st != DUST_OK) return st;
    }
    if (dW) {
        const dust_status st = contract_launch(op, ld_op, terms, x, ld_x, N, d_in, d_out, dW, accumulate, split, s);
        if (st != DUST_OK) return st;
    }
    return cudaGetLastError() == cudaSuccess ? DUST_OK : DUST_ERR_CUDA;
}

}  // namespace dust
