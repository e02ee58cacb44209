// Optimizer step over many tensors at once (dust_optimizer_step_grouped): the elementwise step of
// dust_opt.cu for up to kMaxTensors tensors in one launch, with the moments in fp32 or, for Adam,
// in 8 bits.
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,  g = g_scale G
//   w' = w - lr wd w;  w'' = w' - lr (m' / c1) / (sqrt(v') / sqrt(c2) + eps),  c = 1 - beta^t
//
// 8-bit moments: a block of 256 consecutive elements of a tensor (the last one may be shorter)
// holds m / s_m and r / s_r, r = sqrt(v), as e4m3 codes with fp32 scales s = max / 448.  Choices:
//   - sqrt(v) and not v: e4m3 spans 2^18 from its largest value to its smallest, which for v
//     itself would be 2^9 in gradient size; an element whose v rounded to 0 while its m did not
//     would take a step of m / eps.  For the same reason a positive r never gets code 0.
//   - An fp32 scale and not a power of two: 1 - b2 = 0.001 is far below the codes' half step of
//     2^-4, so a single element's code cannot follow a slow decay; the block's exact largest
//     value does, and carries the others with it (with gradients cut tenfold after 3000 steps
//     the median of the held sqrt(v) stays within 1.5% of the exact average's, scatter 15%).
//   - Round to nearest even: no random numbers, the same result on every run.
// All arithmetic is fp32; the codes are rounded from the fp32 moments after the weights have
// used them.
//
// HBM-bound: per element 4 (G) + 8 (w) + 2 (bf16 copy) + 16 bytes with fp32 moments, + 4.03 with
// 8-bit ones.  Measured: 85 M weights in 120 tensors with fp32 moments 389 us (floor 390 at 6.54 TB/s),
// 201 M in 40 tensors with 8-bit moments 592 to 606 us (floor 556).
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "dust_device.cuh"
#include "dust_internal.h"

namespace dust {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 4096;       // elements of one work unit with fp32 moments
constexpr int kUnit8Small = 2048;  // with 8-bit moments: one block a warp,
constexpr int kUnit8 = 16384;      // or eight, where that leaves enough units
constexpr int kCtas8 = 4;          // CTAs of the 8-bit kernel that an SM holds
constexpr int kBlock = DUST_STATE_BLOCK;
constexpr float kTop = 448.0f;  // largest e4m3 value
// A block whose largest magnitude is below this is held as zeros: 448 / max stays finite.
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100
constexpr float kLeast = 1.0f / 512.0f;  // smallest positive e4m3 value

struct OptTensor {
    const void* G;
    float* W;
    __nv_bfloat16* Wb;
    void* m;
    void* v;
    float* ms;
    float* vs;
    int64_t n;
    int64_t unit_begin;
    float lr, lr_wd;
};

template <int kMax>
struct OptTable {
    OptTensor t[kMax];
    OptParams o;
    const float* g_scale;
    const int32_t* step;
    double beta1, beta2;
    int64_t units;
    int n, unit;
};

// Without .ftz: a subnormal v has a root of 3.7e-23 and more, which an eps below that does not replace.
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / c1 and 1 / sqrt(c2) of this step.
struct Bias {
    float i1, i2;
};

template <bool kGbf16>
__device__ __forceinline__ float4 load_g4(const void* G, int64_t e) {
    if (kGbf16) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(G) + e));
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                           __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    }
    return __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(G) + e));
}
template <bool kGbf16>
__device__ __forceinline__ float load_g1(const void* G, int64_t e) {
    return kGbf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(G)[e])
                  : static_cast<const float*>(G)[e];
}

__device__ __forceinline__ void store_b4(__nv_bfloat16* p, float4 w) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(w.x, w.y);
    __nv_bfloat162 hi = __floats2bfloat162_rn(w.z, w.w);
    uint2 b;
    b.x = *reinterpret_cast<uint32_t*>(&lo);
    b.y = *reinterpret_cast<uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(p) = b;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ F2 both(float x) { return F2{x, x}; }

// Two elements of an 8-bit tensor: m and r = sqrt(v) in, m' and r' out.  The moments are formed with
// one rounding for each product, sum and root, so that the codes are those of the formulas evaluated
// step by step in fp32.  (Contracted into multiply-adds they move one code in a million by a step; packed
// products and sums are contracted in spite of their rounding modifiers, the scalar intrinsics are not.)
__device__ __forceinline__ float blend(float a, float b, float x, float c) {  // a b + x c
    return __fadd_rn(__fmul_rn(a, b), __fmul_rn(x, c));
}
__device__ __forceinline__ void update8(const OptParams& o, const OptTensor& t, Bias b, F2 g, F2& w, F2& m, F2& r) {
    m = F2{blend(m.x, o.b1, g.x, o.omb1), blend(m.y, o.b1, g.y, o.omb1)};
    r = F2{__fsqrt_rn(blend(__fmul_rn(r.x, r.x), o.b2, __fmul_rn(g.x, g.x), o.omb2)),
           __fsqrt_rn(blend(__fmul_rn(r.y, r.y), o.b2, __fmul_rn(g.y, g.y), o.omb2))};
    w = fma2(both(-t.lr_wd), w, w);
    const F2 den = fma2(r, both(b.i2), both(o.eps)), num = mul2(m, both(b.i1));
    w = fma2(both(-t.lr), mul2(num, F2{rcp_approx(den.x), rcp_approx(den.y)}), w);
}

// One element: the new moments and weight; `r` returns sqrt(v').
template <bool kAdam>
__device__ __forceinline__ void update(const OptParams& o, const OptTensor& t, Bias b, float g,
                                       float& w, float& m, float& v, float& r) {
    w = fmaf(-t.lr_wd, w, w);
    if (kAdam) {
        m = fmaf(o.b1, m, o.omb1 * g);
        v = fmaf(o.b2, v, o.omb2 * (g * g));
        r = sqrt_approx(v);
        w = fmaf(-t.lr, __fdividef(m * b.i1, fmaf(r, b.i2, o.eps)), w);
    } else {
        m = fmaf(o.mu, m, g);
        w = fmaf(-t.lr, m, w);
    }
}

template <int kMax>
__device__ __forceinline__ int find_tensor(const OptTable<kMax>& T, int64_t u) {
    int lo = 0, hi = T.n;  // the last tensor whose first unit is <= u
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (T.t[mid].unit_begin <= u)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <int kMax>
__device__ __forceinline__ Bias bias_of(const OptTable<kMax>& T, float* sh) {
    if (T.step == nullptr) return Bias{T.o.c1, T.o.c2};
    // the step count on the device (a captured graph replays with the count it finds)
    if (threadIdx.x == 0) {
        const double t = static_cast<double>(max(*T.step, 1));
        sh[0] = static_cast<float>(1.0 / (1.0 - pow(T.beta1, t)));
        sh[1] = static_cast<float>(1.0 / sqrt(1.0 - pow(T.beta2, t)));
    }
    __syncthreads();
    return Bias{sh[0], sh[1]};
}

template <int kMax, bool kAdam, bool kGbf16>
__global__ void __launch_bounds__(kThreads) opt_grouped_f32_kernel(const __grid_constant__ OptTable<kMax> T) {
    __shared__ float sh[2];
    const Bias b = kAdam ? bias_of(T, sh) : Bias{1.f, 1.f};
    const float gs = T.g_scale ? __ldg(T.g_scale) : 1.0f;
    for (int64_t u = blockIdx.x; u < T.units; u += gridDim.x) {
        const OptTensor& t = T.t[find_tensor(T, u)];
        const int64_t e0 = (u - t.unit_begin) * kUnit;
        float* const tm = static_cast<float*>(t.m);
        float* const tv = static_cast<float*>(t.v);
        const int64_t left = t.n - e0;
        const int n = left < kUnit ? static_cast<int>(left) : kUnit;
        const int n4 = n >> 2;
#pragma unroll 2
        for (int q = threadIdx.x; q < n4; q += kThreads) {
            const int64_t e = e0 + 4 * q;
            float4 g = load_g4<kGbf16>(t.G, e);
            float4 w = *reinterpret_cast<const float4*>(t.W + e);
            float4 m = *reinterpret_cast<const float4*>(tm + e);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (kAdam) v = *reinterpret_cast<const float4*>(tv + e);
            float r;
            update<kAdam>(T.o, t, b, g.x * gs, w.x, m.x, v.x, r);
            update<kAdam>(T.o, t, b, g.y * gs, w.y, m.y, v.y, r);
            update<kAdam>(T.o, t, b, g.z * gs, w.z, m.z, v.z, r);
            update<kAdam>(T.o, t, b, g.w * gs, w.w, m.w, v.w, r);
            *reinterpret_cast<float4*>(t.W + e) = w;
            *reinterpret_cast<float4*>(tm + e) = m;
            if (kAdam) *reinterpret_cast<float4*>(tv + e) = v;
            if (t.Wb) store_b4(t.Wb + e, w);
        }
        const int e1 = 4 * n4 + static_cast<int>(threadIdx.x);  // a tensor's last, partial quad
        if (e1 < n) {
            const int64_t e = e0 + e1;
            float w = t.W[e], m = tm[e], v = kAdam ? tv[e] : 0.f, r;
            update<kAdam>(T.o, t, b, load_g1<kGbf16>(t.G, e) * gs, w, m, v, r);
            t.W[e] = w;
            tm[e] = m;
            if (kAdam) tv[e] = v;
            if (t.Wb) t.Wb[e] = __float2bfloat16_rn(w);
        }
    }
}

// Four e4m3 codes to fp32 and back (the hardware's conversions; rounding to nearest even).
__device__ __forceinline__ float4 from_e4m3(uint32_t c) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xFFFFu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> 16), __NV_E4M3);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(a.x, a.y, d.x, d.y);
}
__device__ __forceinline__ uint32_t to_e4m3(float4 y) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y.x, y.y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y.z, y.w), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
// The larger magnitude, NaN if either is.
__device__ __forceinline__ float max_abs(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(fabsf(a)), "f"(fabsf(b)));
    return y;
}
__device__ __forceinline__ float max_abs4(float4 x) { return max_abs(max_abs(x.x, x.y), max_abs(x.z, x.w)); }
// The largest over the warp: magnitudes order like their bit patterns, with infinity above every number
// and NaN above infinity.
__device__ __forceinline__ float warp_max(float x) {
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x)));
}

// One block's operands as they are loaded: lane l holds elements 4 l .. 4 l + 3 and 128 + 4 l .. + 3, so
// every access of the warp is contiguous.
struct Block8 {
    float4 g[2], w[2];
    uint32_t cm[2], cr[2];
};

template <bool kGbf16>
__device__ __forceinline__ void load_block(const OptTensor& t, int64_t blk, int lane, Block8& x) {
    const uint8_t* const tm = static_cast<const uint8_t*>(t.m);
    const uint8_t* const tv = static_cast<const uint8_t*>(t.v);
    const int64_t e0 = blk * kBlock;
    if (e0 + kBlock <= t.n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t e = e0 + 128 * h + 4 * lane;
            x.g[h] = load_g4<kGbf16>(t.G, e);
            x.w[h] = *reinterpret_cast<const float4*>(t.W + e);
            x.cm[h] = *reinterpret_cast<const uint32_t*>(tm + e);
            x.cr[h] = *reinterpret_cast<const uint32_t*>(tv + e);
        }
    } else {  // the tensor's last, shorter block: elements past its end count as zeros
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float* gp = &x.g[h].x;
            float* wp = &x.w[h].x;
            x.cm[h] = x.cr[h] = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t e = e0 + 128 * h + 4 * lane + j;
                gp[j] = wp[j] = 0.f;
                if (e < t.n) {
                    gp[j] = load_g1<kGbf16>(t.G, e);
                    wp[j] = t.W[e];
                    x.cm[h] |= static_cast<uint32_t>(tm[e]) << (8 * j);
                    x.cr[h] |= static_cast<uint32_t>(tv[e]) << (8 * j);
                }
            }
        }
    }
}

// A positive r keeps at least the smallest code (a NaN stays one).
__device__ __forceinline__ float held_root(float y) { return y > 0.f ? fmaxf(y, kLeast) : y; }

// The step on one block and its stores; the block's largest magnitudes are two warp reductions.  The scales
// come in and go out in sm and sr.
__device__ __forceinline__ void step_block(const OptParams& o, const OptTensor& t, Bias b, float gs, int64_t blk,
                                           int lane, Block8& x, float& sm, float& sr) {
    uint8_t* const tm = static_cast<uint8_t*>(t.m);
    uint8_t* const tv = static_cast<uint8_t*>(t.v);
    const int64_t e0 = blk * kBlock;
    const bool whole = e0 + kBlock <= t.n;
    float4 m[2], r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        m[h] = from_e4m3(x.cm[h]);
        r[h] = from_e4m3(x.cr[h]);
        const F2 g0{__fmul_rn(x.g[h].x, gs), __fmul_rn(x.g[h].y, gs)}, g1{__fmul_rn(x.g[h].z, gs), __fmul_rn(x.g[h].w, gs)};
        F2 m0{__fmul_rn(m[h].x, sm), __fmul_rn(m[h].y, sm)}, m1{__fmul_rn(m[h].z, sm), __fmul_rn(m[h].w, sm)};
        F2 r0{__fmul_rn(r[h].x, sr), __fmul_rn(r[h].y, sr)}, r1{__fmul_rn(r[h].z, sr), __fmul_rn(r[h].w, sr)};
        F2 w0{x.w[h].x, x.w[h].y}, w1{x.w[h].z, x.w[h].w};
        update8(o, t, b, g0, w0, m0, r0);
        update8(o, t, b, g1, w1, m1, r1);
        m[h] = make_float4(m0.x, m0.y, m1.x, m1.y);
        r[h] = make_float4(r0.x, r0.y, r1.x, r1.y);
        x.w[h] = make_float4(w0.x, w0.y, w1.x, w1.y);
        if (whole) {
            const int64_t e = e0 + 128 * h + 4 * lane;
            *reinterpret_cast<float4*>(t.W + e) = x.w[h];
            if (t.Wb) store_b4(t.Wb + e, x.w[h]);
        }
    }
    const float top_m = warp_max(max_abs(max_abs4(m[0]), max_abs4(m[1])));
    const float top_r = warp_max(max_abs(max_abs4(r[0]), max_abs4(r[1])));
    // even lanes form m's factors and odd lanes r's, so that the quotient is taken once
    const float top = (lane & 1) ? top_r : top_m;
    const bool tiny = top < kTiny;  // false for NaN
    const float inv = tiny ? 0.f : kTop / top;
    const float im = __shfl_sync(0xFFFFFFFFu, inv, 0), ir = __shfl_sync(0xFFFFFFFFu, inv, 1);
    const float scale = tiny ? 0.f : top * (1.0f / kTop);
    sm = __shfl_sync(0xFFFFFFFFu, scale, 0);
    sr = __shfl_sync(0xFFFFFFFFu, scale, 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t e = e0 + 128 * h + 4 * lane;
        const F2 m0 = mul2(F2{m[h].x, m[h].y}, both(im)), m1 = mul2(F2{m[h].z, m[h].w}, both(im));
        const F2 r0 = mul2(F2{r[h].x, r[h].y}, both(ir)), r1 = mul2(F2{r[h].z, r[h].w}, both(ir));
        const uint32_t cm = to_e4m3(make_float4(m0.x, m0.y, m1.x, m1.y));
        const uint32_t cr = to_e4m3(make_float4(held_root(r0.x), held_root(r0.y), held_root(r1.x), held_root(r1.y)));
        if (whole) {
            *reinterpret_cast<uint32_t*>(tm + e) = cm;
            *reinterpret_cast<uint32_t*>(tv + e) = cr;
        } else {
            const float* wp = &x.w[h].x;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j < t.n) {
                    t.W[e + j] = wp[j];
                    tm[e + j] = static_cast<uint8_t>(cm >> (8 * j));
                    tv[e + j] = static_cast<uint8_t>(cr >> (8 * j));
                    if (t.Wb) t.Wb[e + j] = __float2bfloat16_rn(wp[j]);
                }
        }
    }
}

// A warp takes a run of up to eight consecutive blocks, so that their scales are one 32-byte sector
// each way: with a 4-byte load and store for each block the launch took 24% longer.
template <int kMax, bool kGbf16>
__global__ void __launch_bounds__(kThreads, kCtas8) opt_grouped_e4m3_kernel(const __grid_constant__ OptTable<kMax> T) {
    __shared__ float sh[2];
    const Bias b = bias_of(T, sh);
    const float gs = T.g_scale ? __ldg(T.g_scale) : 1.0f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = T.unit / kBlock / (kThreads / 32);
    for (int64_t u = blockIdx.x; u < T.units; u += gridDim.x) {
        const OptTensor& t = T.t[find_tensor(T, u)];
        const int64_t first = ((u - t.unit_begin) * (kThreads / 32) + warp) * run;
        const int64_t blocks = (t.n + kBlock - 1) / kBlock;
        if (first >= blocks) continue;
        const int cnt = static_cast<int>(min(static_cast<int64_t>(run), blocks - first));
        float my_sm = 0.f, my_sr = 0.f;  // lane k: block first + k
        if (lane < cnt) {
            my_sm = t.ms[first + lane];
            my_sr = t.vs[first + lane];
        }
        for (int k = 0; k < cnt; ++k) {
            Block8 x;
            load_block<kGbf16>(t, first + k, lane, x);
            float sm = __shfl_sync(0xFFFFFFFFu, my_sm, k), sr = __shfl_sync(0xFFFFFFFFu, my_sr, k);
            step_block(T.o, t, b, gs, first + k, lane, x, sm, sr);
            if (lane == k) {
                my_sm = sm;
                my_sr = sr;
            }
        }
        if (lane < cnt) {
            t.ms[first + lane] = my_sm;
            t.vs[first + lane] = my_sr;
        }
    }
}

// Tensors of one launch: a table of 32 is 2.6 KB of kernel parameters, one of 256 20 KB.
constexpr int kFew = 32;
constexpr int kMany = 256;

// 1 - beta is formed from the decimal that an fp32 beta stands for: 1 - 0.999f is off by 1.3e-5
// relative.  A beta that is not the fp32 nearest to a decimal of seven places is taken as it is.
double meant(float beta) {
    const double d = std::round(static_cast<double>(beta) * 1e7) / 1e7;
    return static_cast<float>(d) == beta ? d : static_cast<double>(beta);
}

template <int kMax>
dust_status launch(const OptParams& o, const dust_opt_params* p, const dust_opt_tensor* ts, int n,
                   bool g_bf16, bool eight, const float* g_scale, const int32_t* step, cudaStream_t s) {
    OptTable<kMax> T;
    T.o = o;
    if (o.kind == DUST_OPT_ADAM) {
        T.o.eps = std::max(o.eps, 1.17549435e-38f);  // the quotients flush subnormal divisors to zero
        T.beta1 = meant(p->beta1);
        T.beta2 = meant(p->beta2);
        T.o.omb1 = static_cast<float>(1.0 - T.beta1);
        T.o.omb2 = static_cast<float>(1.0 - T.beta2);
        // the kernels multiply by the inverse corrections
        T.o.c1 = static_cast<float>(1.0 / (1.0 - std::pow(T.beta1, p->step)));
        T.o.c2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(T.beta2, p->step)));
    }
    T.g_scale = g_scale;
    T.step = o.kind == DUST_OPT_ADAM ? step : nullptr;
    T.n = 0;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) total += ts[i].n;
    T.unit = !eight ? kUnit : total / kUnit8 >= static_cast<int64_t>(num_sms()) * kCtas8 * 4 ? kUnit8 : kUnit8Small;
    int64_t units = 0;
    for (int i = 0; i < n; ++i) {
        if (ts[i].n == 0) continue;
        OptTensor& t = T.t[T.n++];
        t.G = ts[i].G;
        t.W = ts[i].W;
        t.Wb = static_cast<__nv_bfloat16*>(ts[i].W_bf16);
        t.m = ts[i].m;
        t.v = ts[i].v;
        t.ms = ts[i].m_scale;
        t.vs = ts[i].v_scale;
        t.n = ts[i].n;
        t.unit_begin = units;
        t.lr = o.lr * ts[i].lr_scale;
        t.lr_wd = t.lr * p->weight_decay * ts[i].decay_scale;
        units += (t.n + T.unit - 1) / T.unit;
    }
    if (units == 0) return DUST_OK;
    T.units = units;
    // one CTA a unit: the block scheduler evens out the SMs (402 us with 32 CTAs an SM on the twelve-block stack)
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(units, 1 << 30));
    prof_begin(s);
    if (eight) {
        if (g_bf16)
            opt_grouped_e4m3_kernel<kMax, true><<<blocks, kThreads, 0, s>>>(T);
        else
            opt_grouped_e4m3_kernel<kMax, false><<<blocks, kThreads, 0, s>>>(T);
    } else if (o.kind == DUST_OPT_ADAM) {
        if (g_bf16)
            opt_grouped_f32_kernel<kMax, true, true><<<blocks, kThreads, 0, s>>>(T);
        else
            opt_grouped_f32_kernel<kMax, true, false><<<blocks, kThreads, 0, s>>>(T);
    } else {
        if (g_bf16)
            opt_grouped_f32_kernel<kMax, false, true><<<blocks, kThreads, 0, s>>>(T);
        else
            opt_grouped_f32_kernel<kMax, false, false><<<blocks, kThreads, 0, s>>>(T);
    }
    prof_end(s, "optimizer_step_grouped");
    return cudaGetLastError() == cudaSuccess ? DUST_OK : DUST_ERR_CUDA;
}

}  // namespace

dust_status opt_grouped_launch(const OptParams& o, const dust_opt_params* p, const dust_opt_tensor* ts,
                               int n, bool g_bf16, bool eight, const float* g_scale,
                               const int32_t* step, cudaStream_t s) {
    for (int i = 0; i < n; i += kMany) {
        const int cnt = std::min(kMany, n - i);
        const dust_status st = cnt <= kFew
                                   ? launch<kFew>(o, p, ts + i, cnt, g_bf16, eight, g_scale, step, s)
                                   : launch<kMany>(o, p, ts + i, cnt, g_bf16, eight, g_scale, step, s);
        if (st != DUST_OK) return st;
    }
    return DUST_OK;
}

}  // namespace dust
