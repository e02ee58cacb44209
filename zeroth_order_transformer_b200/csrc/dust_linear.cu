// The linear layer with its epilogue, and its backward pass:
//
//   z = x W^T + b,  y = act(z) + residual
//   dz = dy act'(z),  db = sum_t dz_t,  dW = dz^T x,  dx = dz W
//
// Three forms of the product:
//   linear_rows_kernel    one or two tokens: bound by reading W once.  A warp holds four output rows of W
//                         against the tokens, 16 bytes a lane; where there are few output rows the
//                         warps of a CTA split the contraction (8192 -> 8192 23 us, 134 MB at 5.8 TB/s).
//   linear_gemm_kernel    tcgen05 GEMM, persistent and warp-specialised: one warp feeds a TMA ring, one
//                         thread issues the MMAs of a 128-row tile into one of two accumulators in
//                         tensor memory, eight warps run the epilogue of the previous tile from the other.
//                         The forward product, dx and dW differ in which operands are MN-major.  Long
//                         contractions into bf16 take 256 x 256 tiles by pairs of CTAs (cta_group::2).
//                         16384 tokens, 2048 <-> 8192: dx 331 us, 1.66 PFLOP/s; the forward product with GELU
//                         and both outputs 373 us, 1.47; dW with two terms of dz 717 us, 1.53.  Run without a
//                         pause the chip's power holds them to about 1.2 (a plain library product: 1.42).
//   linear_tokens_kernel  the same pipeline for outputs of few tiles: W's rows are the 128 rows of an MMA, the
//                         tokens its columns, the contraction cut over the CTAs of a cluster and
//                         joined through distributed shared memory (24 tokens 8192 -> 8192 26 us, 5.2 TB/s).
// dz is formed once (linear_dz_kernel) as a bf16 operand, or as hi + lo bf16 terms (dz = hi + lo to
// about 16 bits; lo = 0 where hi is infinite), with the column sums for db on the way.
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

__device__ __forceinline__ F2 both(float x) { return F2{x, x}; }
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// The activations work on pairs with packed fp32 arithmetic: the GEMM epilogues have two warps to a scheduler
// and pay for every instruction (the GELU with an exponential and a quotient an element took 4.7 us a 128 x
// 256 tile, this one 2.1).  Infinities keep their limits: the factor that is 0 far out meets a finite number.
//
// z / (1 + 2^e), e = -u log2 of e
__device__ __forceinline__ F2 gated(F2 z, F2 e) {
    const F2 d = add2(F2{ex2_approx(e.x), ex2_approx(e.y)}, both(1.0f));
    return mul2(F2{fmaxf(z.x, -3.0e38f), fmaxf(z.y, -3.0e38f)}, F2{rcp_approx(d.x), rcp_approx(d.y)});
}
template <int kAct>
__device__ __forceinline__ F2 act_pair(F2 z) {
    if (kAct == DUST_ACT_RELU) return F2{z.x <= 0.f ? 0.f : z.x, z.y <= 0.f ? 0.f : z.y};  // keeps a NaN
    if (kAct == DUST_ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| erfc(|z| / sqrt 2) / 2 with 7.1.28 of Abramowitz and Stegun, erfc(x) =
        // (1 + a1 x + ... + a6 x^6)^-16 to 3e-7: one reciprocal, no exponential.  0 from |z| = 64 on.
        const F2 az{fminf(fabsf(z.x), 64.0f), fminf(fabsf(z.y), 64.0f)};
        const F2 x = mul2(az, both(kSqrtHalf));
        F2 p = fma2(both(0.0000430638f), x, both(0.0002765672f));
        p = fma2(p, x, both(0.0001520143f));
        p = fma2(p, x, both(0.0092705272f));
        p = fma2(p, x, both(0.0422820123f));
        p = fma2(p, x, both(0.0705230784f));
        p = fma2(p, x, both(1.0f));
        p = mul2(p, p);
        p = mul2(p, p);
        p = mul2(p, p);
        p = mul2(p, p);  // overflows to infinity far out: its reciprocal is 0
        const F2 r{rcp_approx(p.x), rcp_approx(p.y)};
        return fma2(mul2(az, both(-0.5f)), r, F2{z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y});
    }
    if (kAct == DUST_ACT_GELU_TANH)
        return gated(z, mul2(z, fma2(mul2(z, z), both(-kGeluB * kLog2e), both(-kGeluA * kLog2e))));
    if (kAct == DUST_ACT_SILU) return gated(z, mul2(z, both(-kLog2e)));
    return z;
}
__device__ __forceinline__ float act_any(int act, float z) {
    switch (act) {
        case DUST_ACT_RELU: return act_pair<DUST_ACT_RELU>(both(z)).x;
        case DUST_ACT_GELU: return act_pair<DUST_ACT_GELU>(both(z)).x;
        case DUST_ACT_GELU_TANH: return act_pair<DUST_ACT_GELU_TANH>(both(z)).x;
        case DUST_ACT_SILU: return act_pair<DUST_ACT_SILU>(both(z)).x;
    }
    return z;
}
template <int kAct, int kN>
__device__ __forceinline__ void act_all(float (&v)[kN]) {
#pragma unroll
    for (int j = 0; j < kN; j += 2) {
        const F2 y = act_pair<kAct>(F2{v[j], v[j + 1]});
        v[j] = y.x;
        v[j + 1] = y.y;
    }
}

// Slopes, for the backward pass's HBM-bound sweep.  Phi(-|z|) = erfc(|z| / sqrt 2) / 2 by 7.1.26 of Abramowitz and
// Stegun (error of erf at most 1.5e-7, falling with exp(-z^2 / 2)); e returns exp(-z^2 / 2), which the density shares.
__device__ __forceinline__ float logistic(float u) { return __fdividef(1.0f, 1.0f + __expf(-u)); }
__device__ __forceinline__ float lower_tail(float z, float& e) {
    const float x = fabsf(z) * kSqrtHalf;
    const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
    e = __expf(-x * x);
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    return 0.5f * p * t * e;
}
// Far from zero the slope's second term is 0 times something that may have overflowed: it is dropped.
template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
    if (kAct == DUST_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if (kAct == DUST_ACT_GELU) {
        float e;
        const float q = lower_tail(z, e);
        const float cdf = z > 0.f ? 1.0f - q : q;
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
template <int kN>
__device__ __forceinline__ void act_block(int act, float (&v)[kN]) {
    switch (act) {  // uniform over the grid
        case DUST_ACT_RELU: act_all<DUST_ACT_RELU>(v); break;
        case DUST_ACT_GELU: act_all<DUST_ACT_GELU>(v); break;
        case DUST_ACT_GELU_TANH: act_all<DUST_ACT_GELU_TANH>(v); break;
        case DUST_ACT_SILU: act_all<DUST_ACT_SILU>(v); break;
    }
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
    pdl_trigger();
    pdl_wait();
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
#pragma unroll(kTok == 1 ? 4 : 2)
        for (int v = share * 32 + lane; v < nv; v += A.split * 32) {
            uint4 ww[kRRows];
#pragma unroll
            for (int r = 0; r < kRRows; ++r) ww[r] = w[r][v];
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                if (t >= A.N) break;
                const uint4 xx = reinterpret_cast<const uint4*>(A.x + t * A.ld_x)[v];
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
        if (A.bias) a += A.bias[o];
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
// C [M, n_out] = sum over kTerms of A_term B, in 128 x kBN tiles and blocks of 64 along the contraction.  A is
// K-major [M, K] (x, dz) or MN-major [K, M] (dz in dW, the tokens being the contraction); the second
// term's rows follow the first's.  B is K-major [n_out, K] (W) or MN-major [K, n_out] (W in dx, x in dW).
constexpr int kBM = 128;
constexpr int kBK = 64;
constexpr int kThreads = 320;  // TMA warp, MMA warp, eight epilogue warps
// A kernel that collects its sums holds up to 128 of them a thread, and with the shared memory all taken a spilled
// register goes to L2 (64 -> 2304 over 8192 tokens 39 us, of which a third waited for spills).  It launches three
// warpgroups of 168 registers: the first (TMA, MMA, two idle warps) gives up 112 a thread, the two of
// the epilogue take 56 more each: 128 x 56 + 256 x 224 = 384 x 168.
constexpr int kPromoteThreads = 384;
constexpr int kIssueRegs = 56, kSumRegs = 224;
static_assert(128 * kIssueRegs + 256 * kSumRegs <= kPromoteThreads * 168, "more registers than the block has");
constexpr uint32_t kABytes = kBM * kBK * 2;
constexpr uint32_t kBox = kBK * 128;          // a 64-row x 64-element box of an MN-major operand
// Each epilogue warp: 32 rows x 64 bytes of y and of z, and the biases of 32 columns.
constexpr uint32_t kWarpStaging = 2 * 2048;
constexpr uint32_t kStaging = 8 * (kWarpStaging + 128);
// The tensor cores truncate as they add to the accumulator: a sum of K products is off toward zero by about K 1.1e-9 of
// its size where the products' signs are mixed (measured: 4.7e-7 at K = 512, 9.1e-6 at K = 8192), by up to K 6e-9
// where all have one (3.3e-5 at K = 8192, 7.8e-4 at 131072).  An fp32 output is therefore collected in registers,
// rounded to nearest, after every 8 blocks (512 products) in the accumulator.  A bf16 output is so from K > 16384 on: up to
// there its own rounding (2^-9 of its size on average) is 20 times the largest of these errors, and the chain is
// faster (8192 tokens, 16384 -> 4096: 712 us, collected 746).
constexpr int kFlush = 8;
constexpr int kLongest = 256;  // blocks of one chain into a bf16 output
// How a tile's sums leave: straight from the accumulator (bf16), or collected in registers, into fp32 or bf16.
enum Sums { kChain = 0, kToF32 = 1, kToBf16 = 2 };

template <int kBN, int kTerms, bool kPair>
struct Shape {
    static constexpr uint32_t kBBytes = (kPair ? kBN / 2 : kBN) * kBK * 2;
    static constexpr uint32_t kStageBytes = kTerms * kABytes + kBBytes;
    static constexpr int kStages = static_cast<int>(192 * 1024 / kStageBytes);
    static constexpr uint32_t kSmem = kStages * kStageBytes + kStaging + 1024 + 256;
    static constexpr uint32_t kTmemCols = 2 * kBN;
};
static_assert(Shape<256, 1, false>::kSmem <= 227 * 1024 && Shape<256, 2, true>::kSmem <= 227 * 1024 &&
                  Shape<256, 1, true>::kSmem <= 227 * 1024,
              "exceeds shared memory");

struct Epilogue {
    const float* bias;
    const void* res;
    void* y;
    __nv_bfloat16* z;
    int64_t M, ld_res, ld_y, ld_z;  // strides in elements
    int n_out, act, out_bf16;
};

struct GemmArgs {
    CUtensorMap ta;  // K-major: 64 x 128 boxes; MN-major: 64 x 64
    CUtensorMap tb;  // K-major: 64 x kBN boxes; MN-major: 64 x 64
    Epilogue e;
    ErrorWord* ew;
    int64_t term_rows;   // rows of A from the first term to the second
    int64_t split_elems; // elements of y from one split's partial to the next
    int k_blocks, per_split, splits, m_tiles, n_tiles;
    int late;  // dW only: see pdl_begin
};

// What late means: the kernel uses nothing that the one before it writes, so that it starts while that one still runs
// and waits for it at its end only, for those that come after.  Each kernel here triggers behind its own wait: what
// lies further back has then completed.  dW runs so beside the last tiles of dx, the column sums of a dz
// that is dy itself beside all of dx (1024 -> 1024 over 5001 tokens, all three outputs in a graph: 33 us, one after the other 38).
__device__ __forceinline__ void pdl_begin(int late) {
    if (!late) pdl_wait();
    pdl_trigger();
}
__device__ __forceinline__ void pdl_end(int late) {
    if (late) pdl_wait();
}

// One thread of a converged warp.  The warps that issue TMA and MMAs take it in place of a lane test: with
// it the compiler keeps descriptors in uniform registers (24 tokens 8192 -> 2048: 11.8 us from 15.9).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0); }

struct Pipe {
    uint64_t *full, *empty, *acc_full, *acc_empty;
    uint32_t tmem;
    uint8_t* stages;
    uint8_t* staging;
};

// With kPair two CTAs (a cluster, on neighbouring SMs) work on one 256-row tile: each holds its 128 rows of A and of
// the sums, and half of B's columns, so that an SM loads 32 KB a block where one alone loads 48.  The even CTA
// issues the MMAs for both; its full barriers take the bytes of both CTAs' loads, its commits free the
// stages and announce the sums in both.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void umma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on `bar` of this CTA, or of both CTAs of the pair.
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if (kPair)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        umma_commit(bar);
}
template <bool kPair>
__device__ __forceinline__ void tmem_get(uint32_t* slot, uint32_t cols) {
    if (kPair) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(slot, cols);
        tmem_relinquish();
    }
}
template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
    if (kPair)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
    else
        tmem_dealloc(tmem, cols);
}

// Barriers, tensor memory; every thread of the CTA calls it.
template <int kBN, int kTerms, bool kPair>
__device__ __forceinline__ Pipe pipe_setup(uint8_t* smem, int epilogue_warps) {
    using S = Shape<kBN, kTerms, kPair>;
    Pipe P;
    P.stages = smem;
    P.staging = smem + S::kStages * S::kStageBytes;
    P.full = reinterpret_cast<uint64_t*>(P.staging + kStaging);
    P.empty = P.full + S::kStages;
    P.acc_full = P.empty + S::kStages;  // [2]
    P.acc_empty = P.acc_full + 2;       // [2]
    uint32_t* slot = reinterpret_cast<uint32_t*>(P.acc_empty + 2);
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&P.full[s], 1);
            mbar_init(&P.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&P.acc_full[b], 1);
            mbar_init(&P.acc_empty[b], epilogue_warps * (kPair ? 2 : 1));
        }
        fence_barrier_init();
    }
    if (threadIdx.x >> 5 == 1) tmem_get<kPair>(slot, S::kTmemCols);
    tc_fence_before();
    __syncthreads();
    if (kPair) {  // both CTAs' barriers and tensor memory exist
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after();
    P.tmem = *slot;
    return P;
}

// One thread: loads blocks [kb0, kb1) of tile (m0, n0) into the ring; kc counts blocks over the CTA's life.  m0
// and n0 are this CTA's own first rows; `lead`: it is the pair's even CTA.
template <int kBN, bool kAmn, bool kBmn, int kTerms, bool kPair>
__device__ __forceinline__ bool pipe_load(const GemmArgs& A, const Pipe& P, int m0, int n0, int kb0, int kb1, bool lead,
                                          uint32_t& kc) {
    using S = Shape<kBN, kTerms, kPair>;
    for (int kb = kb0; kb < kb1; ++kb, ++kc) {
        const int s = kc % S::kStages;
        if (kc >= S::kStages && !mbar_wait_bounded(&P.empty[s], ((kc / S::kStages) - 1) & 1, A.ew, 501)) return false;
        uint8_t* a = P.stages + s * S::kStageBytes;
        uint8_t* b = a + kTerms * kABytes;
        const int k0 = kb * kBK;
        if (!kPair || lead) mbar_arrive_expect_tx(&P.full[s], S::kStageBytes * (kPair ? 2 : 1));
        const uint32_t bar = kPair ? cluster_addr(&P.full[s], 0) : 0u;
        auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
            if (kPair)
                tma_load_2d_pair(dst, map, bar, x, y);
            else
                tma_load_2d(dst, map, &P.full[s], x, y);
        };
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
            const int32_t off = t ? static_cast<int32_t>(A.term_rows) : 0;
            if (kAmn) {
                load(a + t * kABytes, &A.ta, m0, off + k0);
                load(a + t * kABytes + kBox, &A.ta, m0 + 64, off + k0);
            } else {
                load(a + t * kABytes, &A.ta, k0, off + m0);
            }
        }
        if (kBmn) {
#pragma unroll
            for (int j = 0; j < (kPair ? kBN / 2 : kBN) / 64; ++j) load(b + j * kBox, &A.tb, n0 + 64 * j, k0);
        } else {
            load(b, &A.tb, k0, n0);
        }
    }
    return true;
}

// One thread: the MMAs of blocks [kb0, kb1) into accumulator columns d.
template <int kBN, bool kAmn, bool kBmn, int kTerms, bool kPair>
__device__ __forceinline__ bool pipe_mma(const GemmArgs& A, const Pipe& P, uint32_t d, int kb0, int kb1, uint32_t& kc) {
    using S = Shape<kBN, kTerms, kPair>;
    constexpr uint32_t idesc = idesc_bf16_f32(kPair ? 2 * kBM : kBM, kBN, kAmn ? 1 : 0, kBmn ? 1 : 0);
    for (int kb = kb0; kb < kb1; ++kb, ++kc) {
        const int s = kc % S::kStages;
        if (!mbar_wait_bounded(&P.full[s], (kc / S::kStages) & 1, A.ew, 502)) return false;
        tc_fence_after();
        const uint32_t a_addr = smem_u32(P.stages + s * S::kStageBytes);
        // K-major: 32 bytes along the swizzled row per instruction.  MN-major: 16 contraction rows of 128
        // bytes; 8-row groups 1024 bytes apart, 64-element boxes kBox apart.  Descriptors count 16 bytes.
        const uint64_t ad = sdesc_sw128(a_addr, kAmn ? kBox : 16, 1024);
        const uint64_t bd = sdesc_sw128(a_addr + kTerms * kABytes, kBmn ? kBox : 16, 1024);
        constexpr uint32_t kAStep = kAmn ? 2048 / 16 : 2, kBStep = kBmn ? 2048 / 16 : 2;
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
                const uint32_t more = (kb > kb0 || kk > 0 || t > 0) ? 1u : 0u;
                if (kPair)
                    umma_bf16_pair(d, ad + t * (kABytes / 16) + kk * kAStep, bd + kk * kBStep, idesc, more);
                else
                    umma_bf16(d, ad + t * (kABytes / 16) + kk * kAStep, bd + kk * kBStep, idesc, more);
            }
        commit<kPair>(&P.empty[s]);
    }
    return true;
}

// A warp's 32 rows x 64 bytes in shared memory, 16-byte piece j of row r at j ^ (r / 2 mod 4): rows are
// written and read thread by thread and written out four lanes to a row, both without bank conflicts.
__device__ __forceinline__ uint4* staged(uint8_t* buf, int row, int piece) {
    return reinterpret_cast<uint4*>(buf + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}
// The 64 bytes from column byte col_b of the warp's rows t0 .. t0 + 31, those inside [0, M) and below end_b.
__device__ __forceinline__ void rows_out(uint8_t* buf, void* base, int64_t t0, int64_t M, int64_t pitch_b, int64_t col_b,
                                         int64_t end_b, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (lane >> 2) + 8 * i, piece = lane & 3;
        if (t0 + row < M && col_b + 16 * piece < end_b)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + (t0 + row) * pitch_b + col_b + 16 * piece) =
                *staged(buf, row, piece);
    }
}
// The other way, in two steps: four loads, and their values into shared memory.
struct Rows {
    uint4 w[4];
};
__device__ __forceinline__ void rows_load(Rows& r, const void* base, int64_t t0, int64_t M, int64_t pitch_b, int64_t col_b,
                                          int64_t end_b, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (lane >> 2) + 8 * i, piece = lane & 3;
        r.w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (t0 + row < M && col_b + 16 * piece < end_b)
            r.w[i] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + (t0 + row) * pitch_b + col_b +
                                                     16 * piece);
    }
}
__device__ __forceinline__ void rows_stage(const Rows& r, uint8_t* buf, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *staged(buf, (lane >> 2) + 8 * i, lane & 3) = r.w[i];
}

// Bias, pre-activation, activation, residual and store of kN columns from o of the warp's rows t0 .. + 31 (lane:
// row), chunk c of the warp's columns, which end at o_end; bias: those of its columns 4 lane .. + 3; res: the
// residual's rows of this chunk.  kN = 32 for a bf16 y, 16 for an fp32 one: 64 bytes of a row.  kLayer false: no
// bias, z or activation.  All lanes call it.
template <int kN, bool kLayer>
__device__ __forceinline__ void finish(const Epilogue& E, void* y, float (&v)[kN], int64_t t0, int o, int o_end, uint8_t* sy,
                                       uint8_t* sz, float4* sb, float4 bias, Rows& res, int c, int lane) {
    constexpr int kEs = 64 / kN;  // bytes of an element of y
    if (E.res) {  // this chunk's residual is here; the next one's is sent for
        rows_stage(res, sy, lane);
        rows_load(res, E.res, t0, E.M, E.ld_res * kEs, static_cast<int64_t>(o + kN) * kEs,
                  static_cast<int64_t>(min(E.n_out, o_end)) * kEs, lane);
    }
    if (kLayer && E.bias) {
        if (lane / (kN / 4) == c) sb[lane % (kN / 4)] = bias;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kN / 4; ++j) {
            const float4 b = sb[j];
            v[4 * j] += b.x;
            v[4 * j + 1] += b.y;
            v[4 * j + 2] += b.z;
            v[4 * j + 3] += b.w;
        }
    }
    if (kLayer && E.z) {
        uint32_t w[kN / 2];
#pragma unroll
        for (int j = 0; j < kN / 2; ++j) w[j] = pack2(v[2 * j], v[2 * j + 1]);
        if (kN == 32) {
#pragma unroll
            for (int p = 0; p < kN / 8; ++p)
                *staged(sz, lane, p) = make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
        } else if (t0 + lane < E.M) {  // 32 bytes of a row: written by its thread
            uint4* zp = reinterpret_cast<uint4*>(E.z + (t0 + lane) * E.ld_z + o);
#pragma unroll
            for (int p = 0; p < kN / 8; ++p) zp[p] = make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
        }
    }
    if (kLayer) act_block(E.act, v);
    __syncwarp();
    uint32_t w[16];
    if (E.res) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint4 r = *staged(sy, lane, p);
            w[4 * p] = r.x, w[4 * p + 1] = r.y, w[4 * p + 2] = r.z, w[4 * p + 3] = r.w;
        }
        if (kN == 32) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                v[(2 * j) % kN] += bf_lo(w[j]);
                v[(2 * j + 1) % kN] += bf_hi(w[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kN && j < 16; ++j) v[j] += __uint_as_float(w[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
        w[j] = kN == 32 ? pack2(v[(2 * j) % kN], v[(2 * j + 1) % kN]) : __float_as_uint(v[j % kN]);
#pragma unroll
    for (int p = 0; p < 4; ++p) *staged(sy, lane, p) = make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
    __syncwarp();
    rows_out(sy, y, t0, E.M, E.ld_y * kEs, static_cast<int64_t>(o) * kEs, static_cast<int64_t>(E.n_out) * kEs, lane);
    if (kLayer && kN == 32 && E.z)
        rows_out(sz, E.z, t0, E.M, E.ld_z * 2, static_cast<int64_t>(o) * 2, static_cast<int64_t>(E.n_out) * 2, lane);
    __syncwarp();
}

// fp32 sums of kCols columns from o0 of the warp's rows t0 .. + 31 (lane: row), 16 columns at a time.
template <int kCols>
__device__ __forceinline__ void plain_out(const Epilogue& E, void* y, const float (&acc)[kCols], int64_t t0, int o0,
                                          uint8_t* sy, int lane) {
    const int piece = lane & 3, sub = lane >> 2;
    float* to[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        to[i] = t0 + sub + 8 * i < E.M ? static_cast<float*>(y) + (t0 + sub + 8 * i) * E.ld_y + o0 + 4 * piece : nullptr;
#pragma unroll
    for (int c = 0; c < kCols / 16; ++c) {
        if (o0 + c * 16 >= E.n_out) break;  // uniform over the warp; n_out is a multiple of 16
#pragma unroll
        for (int p = 0; p < 4; ++p)
            *staged(sy, lane, p) = make_uint4(__float_as_uint(acc[16 * c + 4 * p]), __float_as_uint(acc[16 * c + 4 * p + 1]),
                                              __float_as_uint(acc[16 * c + 4 * p + 2]), __float_as_uint(acc[16 * c + 4 * p + 3]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (to[i]) {
                float4 v = *reinterpret_cast<const float4*>(staged(sy, sub + 8 * i, piece));
                float4* at = reinterpret_cast<float4*>(to[i] + 16 * c);
                if (E.res) {  // y itself, to be added to
                    const float4 old = *at;
                    v = make_float4(old.x + v.x, old.y + v.y, old.z + v.z, old.w + v.w);
                }
                *at = v;
            }
        __syncwarp();
    }
}

// Tiles in groups of sixteen row tiles, columns slow within a group: the CTAs at work share few tiles of A and B.
constexpr int kGroup = 16;
__device__ __forceinline__ void tile_of(int tile, int m_tiles, int n_tiles, int& m, int& n) {
    const int per = kGroup * n_tiles, g = tile / per, r = tile - g * per;
    const int rows = min(kGroup, m_tiles - g * kGroup);
    n = r / rows;
    m = g * kGroup + r - n * rows;
}

// Persistent: one CTA per SM walks (tile, split) items; each accumulator (two of them) is read by the
// epilogue warps while the MMAs fill the other.  kSums: see kFlush.
template <int kBN, bool kAmn, bool kBmn, int kTerms, int kSums, bool kPair>
__global__ void __launch_bounds__(kSums != kChain ? kPromoteThreads : kThreads, 1) linear_gemm_kernel(const __grid_constant__ GemmArgs A) {
    using S = Shape<kBN, kTerms, kPair>;
    constexpr bool kPromote = kSums != kChain;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const Pipe P = pipe_setup<kBN, kTerms, kPair>(smem, 8);
    pdl_begin(kAmn && A.late);
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int rank = kPair ? static_cast<int>(blockIdx.x & 1) : 0;  // the clusters are CTAs 2 i, 2 i + 1
    const int first = kPair ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
    const int step = kPair ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
    const int tiles = A.m_tiles * A.n_tiles;
    const int items = tiles * A.splits;
    constexpr int kChunk = kPromote ? kFlush : 1 << 30;
    constexpr int kFirst = kPromote ? 4 : 2;  // first epilogue warp

    if (warp < kFirst) {
        if (kPromote) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0) {
            if (elect_one()) {
                prefetch_tensormap(&A.ta);
                prefetch_tensormap(&A.tb);
                uint32_t kc = 0;
                for (int it = first; it < items; it += step) {
                    int m, n;
                    tile_of(it % tiles, A.m_tiles, A.n_tiles, m, n);
                    const int kb0 = it / tiles * A.per_split, kb1 = min(A.k_blocks, kb0 + A.per_split);
                    const int m0 = kPair ? (2 * m + rank) * kBM : m * kBM;
                    const int n0 = n * kBN + (kPair ? rank * (kBN / 2) : 0);
                    if (!pipe_load<kBN, kAmn, kBmn, kTerms, kPair>(A, P, m0, n0, kb0, kb1, rank == 0, kc)) break;
                }
                if (kPair) {
                    // the commits that free the last stages arrive here too: not before this CTA ends
                    for (uint32_t c = kc > S::kStages ? kc - S::kStages : 0; c < kc; ++c)
                        if (!mbar_wait_bounded(&P.empty[c % S::kStages], (c / S::kStages) & 1, A.ew, 506)) break;
                }
            }
        } else if (warp == 1) {
            if (rank == 0 && elect_one()) {
                uint32_t kc = 0;
                uint32_t ci = 0;  // chunks so far: chunk ci goes to accumulator ci mod 2
                bool ok = true;
                for (int it = first; it < items && ok; it += step) {
                    const int kb0 = it / tiles * A.per_split, kb1 = min(A.k_blocks, kb0 + A.per_split);
                    for (int k = kb0; k < kb1 && ok; ++ci) {
                        const int k2 = kb1 - k > kChunk ? k + kChunk : kb1;
                        const uint32_t buf = ci & 1;
                        // the epilogue of the chunk that last used this accumulator has read it
                        if (ci >= 2 && !mbar_wait_bounded(&P.acc_empty[buf], ((ci >> 1) - 1) & 1, A.ew, 503)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        ok = pipe_mma<kBN, kAmn, kBmn, kTerms, kPair>(A, P, P.tmem + buf * kBN, k, k2, kc);
                        commit<kPair>(&P.acc_full[buf]);
                        k = k2;
                    }
                }
            }
        }
    } else {
        if (kPromote) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        // eight epilogue warps: tensor-memory lane quarter warp % 4 (32 rows), column half hf
        const int q = warp & 3;
        const int hf = (warp - kFirst) >> 2;
        uint8_t* sy = P.staging + (warp - kFirst) * kWarpStaging;
        uint8_t* sz = sy + 2048;
        float4* sb = reinterpret_cast<float4*>(P.staging + 8 * kWarpStaging) + (warp - kFirst) * 8;
        constexpr int kCols = kBN / 2;
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        auto release = [&](uint32_t buf) {  // the warp has read its part of the accumulator: it may be refilled
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kPair)
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                     cluster_addr(&P.acc_empty[buf], 0))
                                 : "memory");
                else
                    mbar_arrive(&P.acc_empty[buf]);
            }
        };
        uint32_t ci = 0;
        bool ok = true;
        for (int it = first; it < items && ok; it += step) {
            int m, n;
            tile_of(it % tiles, A.m_tiles, A.n_tiles, m, n);
            const int split = it / tiles;
            const int kb0 = split * A.per_split, kb1 = min(A.k_blocks, kb0 + A.per_split);
            const int64_t t0 = static_cast<int64_t>(kPair ? 2 * m + rank : m) * kBM + q * 32;
            const int o0 = n * kBN + hf * kCols;
            void* y = static_cast<uint8_t*>(A.e.y) + split * A.split_elems * (A.e.out_bf16 ? 2 : 4);
            float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);  // on its way before the wait for the tile
            if (!kBmn && A.e.bias && 4 * lane < kCols && o0 + 4 * lane < A.e.n_out)
                bias = reinterpret_cast<const float4*>(A.e.bias + o0)[lane];
            Rows res;
            if (!kPromote && A.e.res)
                rows_load(res, A.e.res, t0, A.e.M, A.e.ld_res * 2, static_cast<int64_t>(o0) * 2,
                          static_cast<int64_t>(min(A.e.n_out, o0 + kCols)) * 2, lane);
            if (kPromote) {
                float acc[kCols];
#pragma unroll
                for (int j = 0; j < kCols; ++j) acc[j] = 0.f;
                for (int k = kb0; k < kb1 && ok; k += kChunk, ++ci) {
                    const uint32_t buf = ci & 1;
                    if (!mbar_wait_bounded(&P.acc_full[buf], (ci >> 1) & 1, A.ew, 504)) {
                        ok = false;
                        break;
                    }
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t trow = P.tmem + buf * kBN + hf * kCols + lane_base;
#pragma unroll
                    for (int c = 0; c < kCols / 16; ++c) {
                        float v[16];
                        tmem_ld16(trow + c * 16, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[c * 16 + j] += v[j];
                    }
                    release(buf);
                }
                if (!ok) break;
                if (kSums == kToBf16) {
                    if (A.e.res)
                        rows_load(res, A.e.res, t0, A.e.M, A.e.ld_res * 2, static_cast<int64_t>(o0) * 2,
                                  static_cast<int64_t>(min(A.e.n_out, o0 + kCols)) * 2, lane);
                    // a copy of the epilogue for each chunk, in its own registers: picked by predicates, 32 at a time
                    // beside 128 sums spill into the loop over the blocks (8192 tokens, 16384 -> 4096: 872 us, so 746)
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) {
                        if (o0 + c * 32 >= A.e.n_out) break;  // uniform over the warp
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = acc[c * 32 + j];
                        finish<32, !kBmn>(A.e, y, v, t0, o0 + c * 32, o0 + kCols, sy, sz, sb, bias, res, c, lane);
                    }
                } else if (kBmn) {
                    // dW and dx: no more than the sums, added to what is there if A.e.res says so
                    plain_out<kCols>(A.e, y, acc, t0, o0, sy, lane);
                } else {
                    if (A.e.res)
                        rows_load(res, A.e.res, t0, A.e.M, A.e.ld_res * 4, static_cast<int64_t>(o0) * 4,
                                  static_cast<int64_t>(min(A.e.n_out, o0 + kCols)) * 4, lane);
                    // one copy of the epilogue's code, the chunk's registers picked by predicates
#pragma unroll 1
                    for (int c = 0; c < kCols / 16; ++c) {
                        if (o0 + c * 16 >= A.e.n_out) break;  // uniform over the warp
                        float v[16];
#pragma unroll
                        for (int k = 0; k < kCols / 16; ++k)
                            if (k == c) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[j] = acc[k * 16 + j];
                            }
                        finish<16, true>(A.e, y, v, t0, o0 + c * 16, o0 + kCols, sy, sz, sb, bias, res, c, lane);
                    }
                }
            } else {
                const uint32_t buf = ci & 1;
                if (!mbar_wait_bounded(&P.acc_full[buf], (ci >> 1) & 1, A.ew, 505)) break;
                __syncwarp();
                tc_fence_after();
                const uint32_t trow = P.tmem + buf * kBN + hf * kCols + lane_base;
                const int left = A.e.n_out - o0;
                const int cnt = left <= 0 ? 0 : min(kCols, left + 31) / 32;  // chunks of 32 columns
                float next[32];
                if (cnt > 0) {
                    tmem_ld32(trow, next);
                    tmem_wait_ld32(next);
                }
#pragma unroll 1
                for (int c = 0; c < cnt; ++c) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = next[j];
                    if (c + 1 < cnt) {
                        tmem_ld32(trow + (c + 1) * 32, next);  // on its way while this chunk is worked on
                    } else {
                        release(buf);
                    }
                    finish<32, !kBmn>(A.e, y, v, t0, o0 + c * 32, o0 + kCols, sy, sz, sb, bias, res, c, lane);
                    if (c + 1 < cnt) tmem_wait_ld32(next);
                }
                if (cnt == 0) release(buf);
                ++ci;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) {  // the pair's MMAs, commits and arrivals are over
        cluster_arrive();
        cluster_wait();
    }
    if (warp == 1) tmem_free<kPair>(P.tmem, S::kTmemCols);
    pdl_end(kAmn && A.late);
}

// Few tokens, more than a handful: W streams through the tensor cores as the operand of 128 rows (output
// channels), against up to kTok tokens as the columns, and the contraction is cut over the CTAs of a cluster.
// Each CTA sums its share as the persistent kernel does, sends its sums to the CTAs that own their channels
// (128 / ranks of them each) through distributed shared memory, and each owner adds the shares in rank
// order and runs the epilogue.  (With the tokens as the 128 rows and 64 channels as columns an MMA moves half
// of W: 344 ns a block of 64, which an SM could load in 186.)
template <int kTok>
struct CShape {
    static constexpr uint32_t kXBytes = kTok * 128;
    static constexpr uint32_t kStageBytes = kABytes + kXBytes;
    static constexpr uint32_t kStaging = kBM * kTok * 4;  // the shares of one owner
    static constexpr int kFit = static_cast<int>((225 * 1024 - kStaging) / kStageBytes);
    static constexpr int kStages = kFit < 10 ? kFit : 10;
    static constexpr uint32_t kSmem = kStages * kStageBytes + kStaging + 1024 + 512;
    static constexpr uint32_t kTmemCols = 2 * kTok;
};
static_assert(CShape<128>::kSmem <= 227 * 1024 && CShape<64>::kSmem <= 227 * 1024 && CShape<32>::kSmem <= 227 * 1024,
              "exceeds shared memory");

// GemmArgs: ta is W (64 x 128 boxes; kAmn, for dx, where the output channels are W's columns: 64 x 64), tb is the
// tokens (64 x kTok); m tiles are of channels and n tiles of tokens.
template <int kTok, bool kAmn>
__global__ void __launch_bounds__(kThreads, 1) linear_tokens_kernel(const __grid_constant__ GemmArgs A) {
    using S = CShape<kTok>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    float* staging = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kStages * S::kStageBytes + S::kStaging);
    uint64_t* empty = full + S::kStages;
    uint64_t* acc_full = empty + S::kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    const int warp = warp_index(), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(slot, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    pdl_begin(0);
    cluster_arrive();  // waited for before the first remote store: the peers are running by then
    const int ranks = A.splits, rank = static_cast<int>(blockIdx.x) % ranks;
    const int o0 = static_cast<int>(blockIdx.x) / ranks * kBM;
    const int t0 = static_cast<int>(blockIdx.y) * kTok;
    const int kb0 = min(A.k_blocks, rank * A.per_split), kb1 = min(A.k_blocks, kb0 + A.per_split);
    const int w = kBM / ranks;  // channels that a rank owns: 16, 32, 64 or 128
    constexpr int kHalf = kTok / 2;
    float acc[kHalf];  // epilogue warps: channel q 32 + lane, tokens hf kHalf ..
    const int q = warp & 3, hf = (warp - 2) >> 2;
    if (warp == 0) {
        if (elect_one()) {
            prefetch_tensormap(&A.ta);
            prefetch_tensormap(&A.tb);
            for (int kb = kb0; kb < kb1; ++kb) {
                const int i = kb - kb0, s = i % S::kStages;
                if (i >= S::kStages && !mbar_wait_bounded(&empty[s], ((i / S::kStages) - 1) & 1, A.ew, 511)) break;
                uint8_t* a = smem + s * S::kStageBytes;
                mbar_arrive_expect_tx(&full[s], S::kStageBytes);
                if (kAmn) {
                    tma_load_2d(a, &A.ta, &full[s], o0, kb * kBK);
                    tma_load_2d(a + kBox, &A.ta, &full[s], o0 + 64, kb * kBK);
                } else {
                    tma_load_2d(a, &A.ta, &full[s], kb * kBK, o0);
                }
                tma_load_2d(a + kABytes, &A.tb, &full[s], kb * kBK, t0);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_bf16_f32(kBM, kTok, kAmn ? 1 : 0, 0);
            uint32_t ci = 0;
            bool ok = true;
            for (int k = kb0; k < kb1 && ok; k += kFlush, ++ci) {
                const uint32_t buf = ci & 1;
                if (ci >= 2 && !mbar_wait_bounded(&acc_empty[buf], ((ci >> 1) - 1) & 1, A.ew, 513)) break;
                tc_fence_after();
                for (int kb = k; kb < min(kb1, k + kFlush); ++kb) {
                    const int i = kb - kb0, s = i % S::kStages;
                    if (!mbar_wait_bounded(&full[s], (i / S::kStages) & 1, A.ew, 512)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(smem + s * S::kStageBytes);
                    const uint64_t ad = sdesc_sw128(a_addr, kAmn ? kBox : 16, 1024);
                    const uint64_t bd = sdesc_sw128(a_addr + kABytes, 16, 1024);
                    constexpr uint32_t kAStep = kAmn ? 2048 / 16 : 2;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        umma_bf16(tmem + buf * kTok, ad + kAStep * kk, bd + 2 * kk, idesc, (kb > k || kk > 0) ? 1u : 0u);
                    umma_commit(&empty[s]);
                }
                umma_commit(&acc_full[buf]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;
        uint32_t ci = 0;
        for (int k = kb0; k < kb1; k += kFlush, ++ci) {
            const uint32_t buf = ci & 1;
            if (!mbar_wait_bounded(&acc_full[buf], (ci >> 1) & 1, A.ew, 514)) break;
            __syncwarp();
            tc_fence_after();
            const uint32_t at = tmem + buf * kTok + hf * kHalf + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
            for (int c = 0; c < kHalf / 8; ++c) {
                float v[8];
                tmem_ld8(at + c * 8, v);
                tmem_wait_ld8(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[c * 8 + j] += v[j];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
    }
    __syncwarp();
    cluster_wait();
    const int tokens = static_cast<int>(min(static_cast<int64_t>(kTok), A.e.M - t0));
    if (warp >= 2) {
        // share [rank][token][channel of the owner]: a warp's lanes write consecutive channels
        const int ch = q * 32 + lane, owner = ch / w;
        const uint32_t mine = smem_u32(staging + (rank * kTok + hf * kHalf) * w + (ch - owner * w));
        uint32_t remote;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(mine), "r"(owner));
#pragma unroll
        for (int j = 0; j < kHalf; ++j)
            if (hf * kHalf + j < tokens)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote + static_cast<uint32_t>(j * w * 4)), "f"(acc[j])
                             : "memory");
    }
    cluster_arrive();
    cluster_wait();
    // this CTA's channels o0 + rank w .. + w - 1 of the tile's tokens, four channels a thread
    const int quads = w / 4;
    for (int e = threadIdx.x; e < tokens * quads; e += kThreads) {
        const int row = e / quads, c = 4 * (e - row * quads);
        const int o = o0 + rank * w + c;
        if (o >= A.e.n_out) continue;  // n_out is a multiple of 16
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < ranks; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(staging + (k * kTok + row) * w + c);
            a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
        }
        const int64_t t = t0 + row;
        if (A.e.bias) {
            const float4 b = *reinterpret_cast<const float4*>(A.e.bias + o);
            a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
        }
        if (A.e.z)
            *reinterpret_cast<uint2*>(A.e.z + t * A.e.ld_z + o) = make_uint2(pack2(a.x, a.y), pack2(a.z, a.w));
        float v[4] = {a.x, a.y, a.z, a.w};
        act_block(A.e.act, v);
        if (A.e.out_bf16) {
            if (A.e.res) {
                const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(A.e.res) + t * A.e.ld_res + o);
                v[0] += bf_lo(r.x), v[1] += bf_hi(r.x), v[2] += bf_lo(r.y), v[3] += bf_hi(r.y);
            }
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(A.e.y) + t * A.e.ld_y + o) =
                make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
        } else {
            if (A.e.res) {
                const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(A.e.res) + t * A.e.ld_res + o);
                v[0] += r.x, v[1] += r.y, v[2] += r.z, v[3] += r.w;
            }
            *reinterpret_cast<float4*>(static_cast<float*>(A.e.y) + t * A.e.ld_y + o) = make_float4(v[0], v[1], v[2], v[3]);
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
// Rows of one partial sum: 256, fewer (down to 32) while there are fewer than six CTAs an SM.
int dz_rows(int64_t N, int32_t d_out) {
    int rows = 256;
    while (rows > 32 && (N + rows - 1) / rows * ((d_out + kDCols - 1) / kDCols) < static_cast<int64_t>(num_sms()) * 6)
        rows /= 2;
    return rows;
}

struct DzArgs {
    const void* dy;
    const __nv_bfloat16* z;
    __nv_bfloat16* hi;  // [N, d_out], or null (dy itself is the operand)
    __nv_bfloat16* lo;  // [N, d_out], or null
    float* part;        // [row chunks, d_out] column sums, or null
    int64_t N, ld_dy, ld_z;
    int d_out, rows, late;
};

// Four CTAs an SM (16384 x 8192, GELU: 192 us, 5.6 TB/s; with the registers for three 204).
template <typename T, int kAct>
__global__ void __launch_bounds__(kDThreads, 4) linear_dz_kernel(const __grid_constant__ DzArgs A) {
    __shared__ float sh[kDWarps][kDCols + 8];
    pdl_begin(A.late);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * kDCols + lane * 8;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * A.rows;
    const int64_t r1 = min(A.N, r0 + A.rows);
    float s[8] = {};
    constexpr int kRaw = sizeof(T) / 2;  // 16-byte pieces of eight elements of dy
    struct Row {
        uint4 dy[kRaw], z;
    };
    auto load = [&](Row& r, int64_t t) {
        const T* p = static_cast<const T*>(A.dy) + t * A.ld_dy + col;
#pragma unroll
        for (int j = 0; j < kRaw; ++j) r.dy[j] = load_l2(p + 8 / kRaw * j);
        if (kAct != DUST_ACT_NONE) r.z = load_l2(A.z + t * A.ld_z + col);
    };
    auto take = [&](const Row& r, int64_t t) {
        float g[8];
        if (sizeof(T) == 2) {
            const uint32_t ww[4] = {r.dy[0].x, r.dy[0].y, r.dy[0].z, r.dy[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g[2 * j] = bf_lo(ww[j]);
                g[2 * j + 1] = bf_hi(ww[j]);
            }
        } else {
            const uint4 a = r.dy[0], b = r.dy[kRaw - 1];
            const uint32_t ww[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = __uint_as_float(ww[j]);
        }
        if (kAct != DUST_ACT_NONE) {
            const uint32_t ww[4] = {r.z.x, r.z.y, r.z.z, r.z.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g[2 * j] *= act_slope<kAct>(bf_lo(ww[j]));
                g[2 * j + 1] *= act_slope<kAct>(bf_hi(ww[j]));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += g[j];
        if (A.hi) {
            uint32_t h[4], l[4], far = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = pack2(g[2 * j], g[2 * j + 1]);
                // the remainder is exact in fp32
                l[j] = pack2(g[2 * j] - bf_lo(h[j]), g[2 * j + 1] - bf_hi(h[j]));
                far |= (h[j] & 0x7F807F80u) + 0x00800080u;  // an exponent of ones carries into the sign's place
            }
            if (far & 0x80008000u) {  // an infinite value has no remainder
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (fabsf(bf_lo(h[j])) == INFINITY) l[j] &= 0xFFFF0000u;
                    if (fabsf(bf_hi(h[j])) == INFINITY) l[j] &= 0x0000FFFFu;
                }
            }
            const int64_t at = t * A.d_out + col;
            *reinterpret_cast<uint4*>(A.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
            if (A.lo) *reinterpret_cast<uint4*>(A.lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    };
    if (col < A.d_out) {
        if (kAct == DUST_ACT_NONE) {
            // little to compute: several rows on their way together (sums over 16384 x 8192 of bf16 51 us, one row ahead 59)
            constexpr int kRows = 4 / kRaw;
            for (int64_t t = r0 + warp; t < r1; t += kRows * kDWarps) {
                Row r[kRows];
#pragma unroll
                for (int k = 0; k < kRows; ++k) load(r[k], min(t + k * kDWarps, r1 - 1));
#pragma unroll
                for (int k = 0; k < kRows; ++k)
                    if (t + k * kDWarps < r1) take(r[k], t + k * kDWarps);
            }
        } else {
            Row a;  // the next row is on its way while this one is worked on
            if (r0 + warp < r1) load(a, r0 + warp);
#pragma unroll 2
            for (int64_t t = r0 + warp; t < r1; t += kDWarps) {
                Row b;
                load(b, min(t + kDWarps, r1 - 1));
                take(a, t);
                a = b;
            }
        }
    }
    if (!A.part) return;  // never late
#pragma unroll
    for (int j = 0; j < 8; ++j) sh[warp][lane * 8 + j] = s[j];
    __syncthreads();
    const int c = blockIdx.x * kDCols + threadIdx.x;
    if (c < A.d_out) {
        float a = 0.f;
        for (int w = 0; w < kDWarps; ++w) a += sh[w][threadIdx.x];
        A.part[static_cast<int64_t>(blockIdx.y) * A.d_out + c] = a;
    }
    pdl_end(A.late);
}

// What the partial sums still lack, in one launch: db (+)= its chunks' sums, 32 columns a CTA, the CTA's eight warps over
// consecutive runs of chunks; then dW (+)= the sum of its splits in order, four elements a thread.
struct JoinArgs {
    const float* db_part;
    float* db;
    const float4* dw_part;
    float4* dW;
    int64_t n4;
    int chunks, d_out, db_blocks, splits, accumulate;
};

__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ JoinArgs A) {
    __shared__ float sh[8][32];
    pdl_begin(0);
    if (static_cast<int>(blockIdx.x) < A.db_blocks) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int c = blockIdx.x * 32 + lane;
        const int per = (A.chunks + 7) / 8;
        const int a = warp * per, b = min(A.chunks, a + per);
        float s = 0.f;
        if (c < A.d_out) {
            int k = a;
            for (; b - k > 8; k += 16) {
                // sixteen loads on their way together (768 columns over 16384 tokens: the call takes 2 us less); a
                // condition around each, or none of min, and they were made one after the other
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] = A.db_part[static_cast<int64_t>(min(k + j, b - 1)) * A.d_out + c];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (k + j < b) s += v[j];
            }
#pragma unroll 4
            for (; k < b; ++k) s += A.db_part[static_cast<int64_t>(k) * A.d_out + c];
        }
        sh[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && c < A.d_out) {
            for (int w = 1; w < 8; ++w) s += sh[w][lane];
            A.db[c] = A.accumulate ? A.db[c] + s : s;
        }
        return;
    }
    const int64_t step = static_cast<int64_t>(gridDim.x - A.db_blocks) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x - A.db_blocks) * blockDim.x + threadIdx.x; i < A.n4; i += step) {
        float4 s = A.accumulate ? A.dW[i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = 0; k < A.splits; ++k) {
            const float4 v = A.dw_part[static_cast<int64_t>(k) * A.n4 + i];
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        A.dW[i] = s;
    }
}

// ------------------------------------------------------------------ host side
template <int kBN, bool kAmn, bool kBmn, int kTerms, int kSums, bool kPair>
dust_status launch_gemm(const GemmArgs& A, cudaStream_t s) {
    using S = Shape<kBN, kTerms, kPair>;
    static PerContextOnce attr;
    if (!attr.run([] {
            return cudaFuncSetAttribute(linear_gemm_kernel<kBN, kAmn, kBmn, kTerms, kSums, kPair>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(S::kSmem)) == cudaSuccess;
        }))
        return DUST_ERR_CUDA;
    const int64_t items = static_cast<int64_t>(A.m_tiles) * A.n_tiles * A.splits;
    const unsigned grid = static_cast<unsigned>(
        kPair ? 2 * std::min<int64_t>(items, num_sms() / 2) : std::min<int64_t>(items, num_sms()));
    return dependent_launch(linear_gemm_kernel<kBN, kAmn, kBmn, kTerms, kSums, kPair>, dim3(grid),
                            kSums != kChain ? kPromoteThreads : kThreads, S::kSmem, s, kPair ? 2 : 1, A)
               ? DUST_OK
               : DUST_ERR_CUDA;
}

// Output tile width: the one that costs least, an SM's tiles one after the other, each as long as the longer of its
// blocks of 64 and the epilogue of the one before it, and the last epilogue (us, about as measured).
int choose_bn(int64_t m_tiles, int n_out, int k_blocks) {
    struct Width {
        int bn;
        double block, epilogue;
    };
    int best = 0;
    double least = 0;
    for (const Width w : {Width{256, 0.41, 2.5}, Width{128, 0.28, 1.3}, Width{64, 0.23, 0.7}}) {
        const int64_t tiles = m_tiles * ((n_out + w.bn - 1) / w.bn);
        const double cost = static_cast<double>((tiles + num_sms() - 1) / num_sms()) *
                                std::max(w.block * k_blocks, w.epilogue) +
                            w.epilogue;
        if (best == 0 || cost < least) {
            least = cost;
            best = w.bn;
        }
    }
    return best;
}

// 256-column tiles of a bf16 output go to pairs of CTAs where the contraction is long enough to pay for
// the pair's set-up (2304 columns over 8192 tokens, kernel times on one set of buffers after a pause, alone and in pairs:
// K = 256 15.5 and 18.5 us, 768 25.8 and 23.9, 1536 43.1 and 40.9).  Sums that change hands every 512 products do so more slowly in a pair.
bool in_pairs(int bn, int k_blocks, int out_bf16) { return bn == 256 && out_bf16 && k_blocks >= 12 && k_blocks <= kLongest; }

template <bool kBmn, int kTerms, int kSums>
dust_status launch_width(int bn, bool pair, const GemmArgs& A, cudaStream_t s) {
    if constexpr (kSums == kChain)
        if (pair) return launch_gemm<256, false, kBmn, kTerms, kSums, true>(A, s);
    return bn == 256   ? launch_gemm<256, false, kBmn, kTerms, kSums, false>(A, s)
           : bn == 128 ? launch_gemm<128, false, kBmn, kTerms, kSums, false>(A, s)
                       : launch_gemm<64, false, kBmn, kTerms, kSums, false>(A, s);
}

template <int kTok, bool kAmn>
dust_status launch_tokens(const GemmArgs& A, cudaStream_t s) {
    using S = CShape<kTok>;
    static PerContextOnce attr;
    if (!attr.run([] {
            return cudaFuncSetAttribute(linear_tokens_kernel<kTok, kAmn>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(S::kSmem)) == cudaSuccess;
        }))
        return DUST_ERR_CUDA;
    return dependent_launch(linear_tokens_kernel<kTok, kAmn>,
                            dim3(static_cast<unsigned>(A.m_tiles * A.splits), static_cast<unsigned>(A.n_tiles)), kThreads,
                            S::kSmem, s, static_cast<unsigned>(A.splits), A)
               ? DUST_OK
               : DUST_ERR_CUDA;
}

// What a launch is called in the profile: the product and its form.
const char* form_name(const char* const (&names)[4], int bn, bool pair) {
    return names[pair ? 3 : bn == 256 ? 2 : bn == 128 ? 1 : 0];
}
const char* token_form_name(const char* const (&names)[4], int tok) {
    return names[tok == 16 ? 0 : tok == 32 ? 1 : tok == 64 ? 2 : 3];
}
constexpr const char* kForward[4] = {"linear_tcgen05_64", "linear_tcgen05_128", "linear_tcgen05_256", "linear_tcgen05_256_pair"};
constexpr const char* kDx[4] = {"linear_dx_tcgen05_64", "linear_dx_tcgen05_128", "linear_dx_tcgen05_256",
                                "linear_dx_tcgen05_256_pair"};
constexpr const char* kDw[3] = {"linear_dw_tcgen05_64", "linear_dw_tcgen05_128", "linear_dw_tcgen05_256"};
constexpr const char* kDw2[3] = {"linear_dw_tcgen05_64_two_terms", "linear_dw_tcgen05_128_two_terms",
                                 "linear_dw_tcgen05_256_two_terms"};
constexpr const char* kTokens[4] = {"linear_tokens_tcgen05_16", "linear_tokens_tcgen05_32", "linear_tokens_tcgen05_64",
                                    "linear_tokens_tcgen05_128"};
constexpr const char* kDxTokens[4] = {"linear_dx_tokens_tcgen05_16", "linear_dx_tokens_tcgen05_32",
                                      "linear_dx_tokens_tcgen05_64", "linear_dx_tokens_tcgen05_128"};

// How many CTAs share a tile's contraction in linear_tokens_kernel.  Clusters of four fit on the SMs about 33 at
// a time (36 of them took two waves: 768 -> 2304 over 256 tokens 15.3 us, with clusters of two 10.3).
int token_ranks(int64_t tiles, int k_blocks) {
    return tiles * 4 <= 132 && k_blocks >= 8 ? 4 : tiles * 2 <= num_sms() && k_blocks >= 4 ? 2 : 1;
}

int token_width(int64_t N) { return N <= 16 ? 16 : N <= 32 ? 32 : N <= 64 ? 64 : 128; }

// Whether linear_tokens_kernel takes the product.  Up to 32 tokens always (24 tokens, 8192 -> 24576: 77 us against 93 in the
// persistent kernel, 2048 -> 65536 63 against 67; with 64 tokens 81 against 56, its sums leaving through shared
// memory one by one); more where a long contraction is shared (here and in the persistent kernel: 64 tokens 2048 ->
// 2048 6.1 and 7.8 us, 512 tokens 11.7 and 8.6; 512 tokens 8192 -> 2048 23 and 31; 64 tokens 2048 -> 8192 11.5 and 10.3).
bool tokens_form(int64_t N, int n_out, int K) {
    if (N <= 32) return true;
    const int tok = token_width(N), k_blocks = (K + kBK - 1) / kBK;
    const int r = token_ranks((N + tok - 1) / tok * ((n_out + kBM - 1) / kBM), k_blocks);
    return r == 4 ? k_blocks >= (N <= 64 ? 24 : 40) : r == 2 && k_blocks >= 64;
}

// y [N, n_out] = x W^T, or with w_mn x W (W [K, n_out]).
dust_status gemm_tokens(const void* x, int64_t ld_x, int K, const void* W, bool w_mn, GemmArgs& G,
                        cudaStream_t s) {
    const int64_t N = G.e.M;
    const int n_out = G.e.n_out;
    const int tok = token_width(N);
    G.ew = device_error_word();
    G.k_blocks = (K + kBK - 1) / kBK;
    G.m_tiles = (n_out + kBM - 1) / kBM;
    G.n_tiles = static_cast<int>((N + tok - 1) / tok);
    G.splits = token_ranks(static_cast<int64_t>(G.m_tiles) * G.n_tiles, G.k_blocks);
    G.per_split = (G.k_blocks + G.splits - 1) / G.splits;
    if (w_mn ? !make_tmap_bf16_2d_ld(&G.ta, W, K, n_out, n_out, kBK, 64)
             : !make_tmap_bf16_2d_ld(&G.ta, W, n_out, K, K, kBM, kBK))
        return DUST_ERR_CUDA;
    if (!make_tmap_bf16_2d_ld(&G.tb, x, static_cast<uint64_t>(N), K, ld_x, tok, kBK)) return DUST_ERR_CUDA;
    prof_begin(s);
    dust_status st;
    if (w_mn)
        st = tok == 16   ? launch_tokens<16, true>(G, s)
             : tok == 32 ? launch_tokens<32, true>(G, s)
             : tok == 64 ? launch_tokens<64, true>(G, s)
                         : launch_tokens<128, true>(G, s);
    else
        st = tok == 16   ? launch_tokens<16, false>(G, s)
             : tok == 32 ? launch_tokens<32, false>(G, s)
             : tok == 64 ? launch_tokens<64, false>(G, s)
                         : launch_tokens<128, false>(G, s);
    prof_end(s, token_form_name(w_mn ? kDxTokens : kTokens, tok));
    return st;
}

// y [M, n_out] = A [terms M, K] B with the epilogue of G.e; B K-major [n_out, K] or MN-major [K, n_out].
dust_status gemm_rows(const void* a, int64_t ld_a, int terms, int K, const void* b, bool b_mn, GemmArgs& G,
                      cudaStream_t s) {
    const int64_t M = G.e.M;
    const int n_out = G.e.n_out;
    const int64_t m_tiles = (M + kBM - 1) / kBM;
    const int bn = choose_bn(m_tiles, n_out, (K + kBK - 1) / kBK);
    G.ew = device_error_word();
    G.term_rows = M;
    G.split_elems = 0;
    G.k_blocks = (K + kBK - 1) / kBK;
    G.per_split = G.k_blocks;
    G.splits = 1;
    G.n_tiles = (n_out + bn - 1) / bn;
    if (m_tiles * G.n_tiles > 1 << 30) return DUST_ERR_UNSUPPORTED;
    const int sums = !G.e.out_bf16 ? kToF32 : G.k_blocks > kLongest ? kToBf16 : kChain;
    const bool pair = in_pairs(bn, G.k_blocks, G.e.out_bf16);  // 256-row tiles, half of B's columns in each CTA
    G.m_tiles = static_cast<int>(pair ? (m_tiles + 1) / 2 : m_tiles);
    if (!make_tmap_bf16_2d_ld(&G.ta, a, static_cast<uint64_t>(terms * M), K, ld_a, kBM, kBK)) return DUST_ERR_CUDA;
    if (b_mn ? !make_tmap_bf16_2d_ld(&G.tb, b, K, n_out, n_out, kBK, 64)
             : !make_tmap_bf16_2d_ld(&G.tb, b, n_out, K, K, pair ? bn / 2 : bn, kBK))
        return DUST_ERR_CUDA;
    prof_begin(s);
    dust_status st;
    if (b_mn)
        st = sums == kChain      ? launch_width<true, 1, kChain>(bn, pair, G, s)
             : sums == kToBf16   ? launch_width<true, 1, kToBf16>(bn, pair, G, s)
             : terms == 2        ? launch_width<true, 2, kToF32>(bn, pair, G, s)
                                 : launch_width<true, 1, kToF32>(bn, pair, G, s);
    else
        st = sums == kChain    ? launch_width<false, 1, kChain>(bn, pair, G, s)
             : sums == kToBf16 ? launch_width<false, 1, kToBf16>(bn, pair, G, s)
                               : launch_width<false, 1, kToF32>(bn, pair, G, s);
    prof_end(s, form_name(b_mn ? kDx : kForward, bn, pair));
    return st;
}

// dW [d_out, d_in] (+)= dz^T x: 128-row tiles (in pairs they take as long: two terms already load 64 KB for
// 1024 cycles of MMAs).  Tile width and splits of the tokens are those that cost least: the waves of items over
// the SMs, an item's blocks of 64 tokens and its epilogue (us, about as measured), and, with more than one
// split, the partials written and read back at about 6 GB/ms and one more launch.  The partials are added in order.
// (256 x 256 over 64 tokens 3.4 us, with 256 columns a tile 6.7; 1024 x 1024 over 5001 14.5 and 18.)
constexpr uint32_t kMinBlocks = 4;
constexpr uint32_t kMaxSplits = 64;
struct DwPlan {
    int bn, m_tiles, n_tiles, k_blocks, splits, per_split;
};
DwPlan dw_plan(int64_t N, int32_t d_in, int32_t d_out) {
    DwPlan p{};
    p.m_tiles = (d_out + kBM - 1) / kBM;
    p.k_blocks = static_cast<int>((N + kBK - 1) / kBK);
    const double join = 8.0 * d_out * d_in / 6e6;
    const uint32_t blocks = static_cast<uint32_t>(p.k_blocks);  // at most 2^17
    const int64_t sms = num_sms();
    struct Width {
        int bn;
        double block, epilogue;
    };
    double least = 0;
    for (const Width w : {Width{256, 0.45, 4.2}, Width{128, 0.32, 2.4}, Width{64, 0.26, 1.5}}) {
        const int n_tiles = (d_in + w.bn - 1) / w.bn;
        const int64_t tiles = static_cast<int64_t>(p.m_tiles) * n_tiles;
        for (uint32_t k = 1; k <= kMaxSplits && (k == 1 || k * kMinBlocks <= blocks); ++k) {
            const uint32_t per = (blocks + k - 1) / k;
            const double cost = static_cast<double>((tiles * k + sms - 1) / sms) * (w.block * per + w.epilogue) +
                                (k > 1 ? 3.0 + k * join : 0.0);
            if (p.bn == 0 || cost < least) {
                least = cost;
                p.bn = w.bn;
                p.n_tiles = n_tiles;
                p.per_split = static_cast<int>(per);
            }
        }
    }
    p.splits = (p.k_blocks + p.per_split - 1) / p.per_split;  // none of them empty
    return p;
}
size_t dw_bytes(int64_t N, int32_t d_in, int32_t d_out) {
    const DwPlan p = dw_plan(N, d_in, d_out);
    return p.splits > 1 ? align_up(static_cast<size_t>(p.splits) * d_out * d_in * 4, 256) : 0;
}
template <int kTerms>
dust_status launch_dw(int bn, const GemmArgs& A, cudaStream_t s) {
    return bn == 256   ? launch_gemm<256, true, true, kTerms, kToF32, false>(A, s)
           : bn == 128 ? launch_gemm<128, true, true, kTerms, kToF32, false>(A, s)
                       : launch_gemm<64, true, true, kTerms, kToF32, false>(A, s);
}
dust_status gemm_dw(const void* dz, int64_t ld_dz, int terms, const void* x, int64_t ld_x, int64_t N, int32_t d_in,
                    int32_t d_out, float* dW, int accumulate, float* part, int late, JoinArgs& join, cudaStream_t s) {
    const DwPlan p = dw_plan(N, d_in, d_out);
    GemmArgs G{};
    G.late = late;
    G.e.M = d_out;
    G.e.n_out = d_in;
    G.e.y = p.splits > 1 ? part : dW;
    G.e.ld_y = d_in;
    G.e.res = p.splits == 1 && accumulate ? dW : nullptr;
    G.e.ld_res = d_in;
    G.ew = device_error_word();
    G.term_rows = N;
    G.split_elems = static_cast<int64_t>(d_out) * d_in;
    G.k_blocks = p.k_blocks;
    G.per_split = p.per_split;
    G.splits = p.splits;
    G.m_tiles = p.m_tiles;
    G.n_tiles = p.n_tiles;
    if (static_cast<int64_t>(p.m_tiles) * p.n_tiles * p.splits > 1 << 30) return DUST_ERR_UNSUPPORTED;
    if (!make_tmap_bf16_2d_ld(&G.ta, dz, static_cast<uint64_t>(terms * N), d_out, ld_dz, kBK, 64) ||
        !make_tmap_bf16_2d_ld(&G.tb, x, static_cast<uint64_t>(N), d_in, ld_x, kBK, 64))
        return DUST_ERR_CUDA;
    prof_begin(s);
    const dust_status st = terms == 2 ? launch_dw<2>(p.bn, G, s) : launch_dw<1>(p.bn, G, s);
    prof_end(s, (terms == 2 ? kDw2 : kDw)[p.bn == 256 ? 2 : p.bn == 128 ? 1 : 0]);
    if (p.splits > 1) {
        join.dw_part = reinterpret_cast<const float4*>(part);
        join.dW = reinterpret_cast<float4*>(dW);
        join.n4 = G.split_elems / 4;
        join.splits = p.splits;
    }
    return st;
}

template <typename T>
bool launch_dz(const DzArgs& A, int act, dim3 grid, cudaStream_t s) {
    switch (act) {
        case DUST_ACT_RELU: return dependent_launch(linear_dz_kernel<T, DUST_ACT_RELU>, grid, kDThreads, 0, s, 1, A);
        case DUST_ACT_GELU: return dependent_launch(linear_dz_kernel<T, DUST_ACT_GELU>, grid, kDThreads, 0, s, 1, A);
        case DUST_ACT_GELU_TANH: return dependent_launch(linear_dz_kernel<T, DUST_ACT_GELU_TANH>, grid, kDThreads, 0, s, 1, A);
        case DUST_ACT_SILU: return dependent_launch(linear_dz_kernel<T, DUST_ACT_SILU>, grid, kDThreads, 0, s, 1, A);
    }
    return dependent_launch(linear_dz_kernel<T, DUST_ACT_NONE>, grid, kDThreads, 0, s, 1, A);
}

size_t dz_bytes(int64_t N, int32_t d_out) { return align_up(static_cast<size_t>(2 * N) * d_out * 2, 256); }
size_t db_bytes(int64_t N, int32_t d_out) {
    const int rows = dz_rows(N, d_out);
    return align_up(static_cast<size_t>((N + rows - 1) / rows) * d_out * 4, 256);
}

// Tokens up to which W is streamed through the CUDA cores.
constexpr int kFewTokens = 2;

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
        const bool ok = N == 1 ? dependent_launch(linear_rows_kernel<1>, dim3(blocks), kRThreads, 0, s, 1, A)
                               : dependent_launch(linear_rows_kernel<2>, dim3(blocks), kRThreads, 0, s, 1, A);
        prof_end(s, "linear_rows");
        return ok ? DUST_OK : DUST_ERR_CUDA;
    }
    GemmArgs G{};
    G.e = Epilogue{bias, res, y, static_cast<__nv_bfloat16*>(z), N, ld_res, ld_y, ld_z, d_out, act, out_bf16};
    const dust_status st = tokens_form(N, d_out, d_in)
                               ? gemm_tokens(x, ld_x, d_in, W, false, G, s)
                               : gemm_rows(x, ld_x, 1, d_in, W, false, G, s);
    if (st != DUST_OK) return st;
    return cudaGetLastError() == cudaSuccess ? DUST_OK : DUST_ERR_CUDA;
}

size_t linear_backward_workspace_bytes(int64_t N, int32_t d_in, int32_t d_out) {
    return dz_bytes(N, d_out) + db_bytes(N, d_out) + dw_bytes(N, d_in, d_out);
}

dust_status linear_backward_launch(const void* dy, int dy_bf16, int64_t ld_dy, const void* z, int64_t ld_z,
                                   const void* x, int64_t ld_x, const void* W, int act, int64_t N, int32_t d_in,
                                   int32_t d_out, int terms, void* dx, int dx_bf16, int64_t ld_dx, float* dW,
                                   float* db, int accumulate, void* ws, cudaStream_t s) {
    char* w = static_cast<char*>(ws);
    __nv_bfloat16* hi = reinterpret_cast<__nv_bfloat16*>(w);
    float* part = reinterpret_cast<float*>(w + dz_bytes(N, d_out));
    float* split = reinterpret_cast<float*>(w + dz_bytes(N, d_out) + db_bytes(N, d_out));
    // without an activation a bf16 dy is the operand itself, exactly, in one term
    const bool direct = act == DUST_ACT_NONE && dy_bf16;
    const bool products = dx || dW;
    if (direct) terms = 1;
    JoinArgs join{};
    join.accumulate = accumulate;
    const auto sweep = [&](int late) {
        const int rows = dz_rows(N, d_out), chunks = static_cast<int>((N + rows - 1) / rows);
        DzArgs A{dy,    static_cast<const __nv_bfloat16*>(z), nullptr, nullptr, db ? part : nullptr, N, ld_dy, ld_z, d_out,
                 rows, late};
        if (products && !direct) {
            A.hi = hi;
            A.lo = terms == 2 ? hi + N * d_out : nullptr;
        }
        if (db) {
            join.db_part = part;
            join.db = db;
            join.chunks = chunks;
            join.d_out = d_out;
            join.db_blocks = (d_out + 31) / 32;
        }
        const dim3 grid((d_out + kDCols - 1) / kDCols, chunks);
        prof_begin(s);
        const bool ok = dy_bf16 ? launch_dz<__nv_bfloat16>(A, act, grid, s) : launch_dz<float>(A, act, grid, s);
        prof_end(s, "linear_dz");
        return ok;
    };
    if (products && !direct && !sweep(0)) return DUST_ERR_CUDA;
    const void* op = direct ? dy : hi;
    const int64_t ld_op = direct ? ld_dy : d_out;
    if (dx) {
        GemmArgs G{};
        G.e.M = N;
        G.e.n_out = d_in;
        G.e.y = dx;
        G.e.ld_y = ld_dx;
        G.e.out_bf16 = dx_bf16;
        // a bf16 dx is rounded as coarsely as one term of dz; an fp32 dx takes both terms
        const int dx_terms = dx_bf16 ? 1 : terms;
        const dust_status st = dx_terms == 1 && tokens_form(N, d_in, d_out)
                                   ? gemm_tokens(op, ld_op, d_out, W, true, G, s)
                                   : gemm_rows(op, ld_op, dx_terms, d_out, W, true, G, s);
        if (st != DUST_OK) return st;
    }
    if (db && (direct || !products) && !sweep(dx != nullptr)) return DUST_ERR_CUDA;
    if (dW) {
        // dz is complete once dx has begun, or is dy
        const int late = dx || (direct && db);
        const dust_status st = gemm_dw(op, ld_op, terms, x, ld_x, N, d_in, d_out, dW, accumulate, split, late, join, s);
        if (st != DUST_OK) return st;
    }
    if (join.db || join.dW) {
        const unsigned blocks =
            static_cast<unsigned>(std::min<int64_t>((join.n4 + 255) / 256, static_cast<int64_t>(num_sms()) * 16));
        prof_begin(s);
        const bool ok = dependent_launch(linear_join_kernel, dim3(blocks + join.db_blocks), 256, 0, s, 1, join);
        prof_end(s, "linear_join");
        if (!ok) return DUST_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? DUST_OK : DUST_ERR_CUDA;
}

}  // namespace dust
