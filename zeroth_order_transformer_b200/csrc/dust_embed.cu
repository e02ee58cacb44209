// Token embedding: the lookup with its scaling, and the gradient of the table.
//
//   out_t = scale E[ids_t]                 (a zero row for ids_t < 0, a NaN row for ids_t >= V)
//   G[v] (+)= scale sum_{t: ids_t = v} g_t (tokens with ids outside [0, V) add nothing)
//
// The lookup is one pass: a thread moves eight elements of a row, two such items at a time (65536 tokens of
// 2048 from fp32 to bf16 76 us; one item 91, four 82, eight 99).
//
// The gradient is a sum over the tokens of each row, and the tokens of a row are scattered over
// the batch.  They are brought together by a stable radix sort of the token indices by id
// (least significant digit first, up to nine bits a pass: a vocabulary of 2^18 takes two), which
// moves 8 bytes a token where a row is hundreds to thousands; up to 16384 tokens are sorted by one cluster in
// one launch.  The sorted positions are cut into chunks of equal length; one warp sums a chunk's rows over 128 (fp32) or 256 (bf16) columns,
// sixteen bytes a lane, eight rows in flight, and writes a table row whenever the id changes.  An id
// that crosses a chunk border leaves partial sums, which a last kernel adds in chunk order: no
// sum depends on the order of atomics, and every run gives the same result.  Rows that no token names are
// cleared in the same launch by CTAs that look for their ids in the sorted list, so every row is written once.
//
// Up to 4096 tokens take one launch instead: each CTA picks the tokens whose id falls to its share of the
// table (id mod the number of shares), sorts those few in shared memory and sums them.
//
// Both are HBM-bound: the rows read and written once.  Measured: the lookup above 5.3 TB/s of the bytes it cannot do
// without (every row is read from L2, 537 MB, where 137 MB of them differ); the gradient of 65536 tokens onto
// 65536 x 2048 152 us, 800 MB and so 5.3 TB/s with the sort, its sums alone 126 us.  Clearing in the sort's launches
// instead, which leave HBM idle, took 203 us: writes alone run at about half the rate of reads and writes together.
#include <algorithm>

#include "dust_device.cuh"
#include "dust_internal.h"

namespace dust {
namespace {

// ------------------------------------------------------------------ rows of eight elements
struct V8 {
    float v[8];
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Elements [0, n) of the eight at p (16-byte aligned); the others are 0.
__device__ __forceinline__ V8 load8(const float* p, int n) {
    V8 r;
    if (n >= 8) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        const float4 b = reinterpret_cast<const float4*>(p)[1];
        r = V8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = j < n ? p[j] : 0.f;
    }
    return r;
}
__device__ __forceinline__ V8 load8(const __nv_bfloat16* p, int n) {
    V8 r;
    if (n >= 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        r = V8{{bf_lo(a.x), bf_hi(a.x), bf_lo(a.y), bf_hi(a.y), bf_lo(a.z), bf_hi(a.z), bf_lo(a.w),
                bf_hi(a.w)}};
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = j < n ? __bfloat162float(p[j]) : 0.f;
    }
    return r;
}
__device__ __forceinline__ void store8(float* p, const V8& r, int n) {
    if (n >= 8) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(r.v[0], r.v[1], r.v[2], r.v[3]));
        __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(r.v[4], r.v[5], r.v[6], r.v[7]));
    } else {
        for (int j = 0; j < n; ++j) p[j] = r.v[j];
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const V8& r, int n) {
    if (n >= 8) {
        uint4 w;
        uint32_t* wp = &w.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(r.v[2 * j], r.v[2 * j + 1]);
            wp[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        __stcs(reinterpret_cast<uint4*>(p), w);
    } else {
        for (int j = 0; j < n; ++j) p[j] = __float2bfloat16_rn(r.v[j]);
    }
}

// ------------------------------------------------------------------ the lookup
constexpr int kFThreads = 256;
constexpr int kFItems = 2;  // items of eight elements a thread holds at once

template <typename TE, typename TO>
__global__ void __launch_bounds__(kFThreads) embedding_kernel(const int32_t* ids, const TE* E,
                                                              int64_t ld_E, int64_t N, int32_t V, int32_t d, int32_t nv,
                                                              uint64_t nv_magic, float scale, TO* out,
                                                              int64_t ld_out) {
    pdl_trigger();
    pdl_wait();
    const int64_t total = N * nv;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * (kFThreads * kFItems) + threadIdx.x;
    V8 r[kFItems];
    int64_t at[kFItems];
    int left[kFItems];
    float by[kFItems];
#pragma unroll
    for (int j = 0; j < kFItems; ++j) {
        const int64_t f = base + j * kFThreads;
        left[j] = 0;
        if (f < total) {
            const int64_t t = div_by_magic(f, nv, nv_magic);
            const int c = 8 * static_cast<int>(f - t * nv);
            const int32_t id = ids[t];
            left[j] = d - c;
            at[j] = t * ld_out + c;
            by[j] = 1.0f;
            if (id >= 0 && id < V) {
                by[j] = scale;
                r[j] = load8(E + static_cast<int64_t>(id) * ld_E + c, left[j]);
            } else {
                const float fill = id < 0 ? 0.f : __uint_as_float(0x7FC00000u);
#pragma unroll
                for (int k = 0; k < 8; ++k) r[j].v[k] = fill;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kFItems; ++j)
        if (left[j] > 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) r[j].v[k] *= by[j];
            store8(out + at[j], r[j], left[j]);
        }
}

// ------------------------------------------------------------------ stable radix sort by id
constexpr int kBinBits = 9;
constexpr int kBins = 1 << kBinBits;
constexpr int kSThreads = 512;  // one thread per bin in the prefix sums
constexpr int kSWarps = kSThreads / 32;
static_assert(kSThreads == kBins, "one thread per bin");
// Keys per lane: a tile is 512 of each.  Small tiles spread a sort over more SMs, large ones shorten the
// sums over the tiles' counts, which every CTA takes itself.
constexpr int kFewRounds = 2, kManyRounds = 8;
constexpr int64_t kManyTokens = 1 << 18;

__device__ __forceinline__ uint32_t key_of(int32_t id, int32_t V) {
    return id >= 0 && id < V ? static_cast<uint32_t>(id) : static_cast<uint32_t>(V);  // no row: last
}

// Digit counts of each tile: hist[tile][bin].
template <int kSRounds>
__global__ void __launch_bounds__(kSThreads) embed_hist_kernel(const int32_t* ids, const uint32_t* keys,
                                                               int64_t N, int32_t V, int shift, uint32_t mask,
                                                               int32_t* hist) {
    __shared__ int32_t cnt[kBins];
    pdl_trigger();
    pdl_wait();
    cnt[threadIdx.x] = 0;
    __syncthreads();
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * (kSThreads * kSRounds);
#pragma unroll
    for (int r = 0; r < kSRounds; ++r) {
        const int64_t p = p0 + r * kSThreads + threadIdx.x;
        if (p < N) {
            const uint32_t k = ids ? key_of(ids[p], V) : keys[p];
            atomicAdd(&cnt[(k >> shift) & mask], 1);
        }
    }
    __syncthreads();
    hist[static_cast<int64_t>(blockIdx.x) * kBins + threadIdx.x] = cnt[threadIdx.x];
}

// Where each of this thread's keys goes within a stable order of the tile by digit, on top of
// base[bin].  Keys are taken warp by warp, round by round, lane by lane: their order in the tile.
// `n` keys are valid.  All threads of the CTA call it; wh [kSWarps][kBins] is scratch.
template <int kSRounds>
__device__ __forceinline__ void tile_ranks(const uint32_t (&digit)[kSRounds], int n, int32_t base,
                                           int32_t (*wh)[kBins], int32_t (&pos)[kSRounds]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int w = 0; w < kSWarps; ++w) wh[w][threadIdx.x] = 0;
    __syncthreads();
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int r = 0; r < kSRounds; ++r) {
        const int at = (warp * kSRounds + r) * 32 + lane;
        const uint32_t dg = at < n ? digit[r] : 0xFFFFFFFFu;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, dg);
        int before = 0;
        if (at < n) before = wh[warp][dg];
        __syncwarp();
        pos[r] = before + __popc(same & below);
        if (at < n && (same & below) == 0) wh[warp][dg] = before + __popc(same);
        __syncwarp();
    }
    __syncthreads();
    int32_t run = base;  // of bin threadIdx.x
    for (int w = 0; w < kSWarps; ++w) {
        const int32_t c = wh[w][threadIdx.x];
        wh[w][threadIdx.x] = run;
        run += c;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSRounds; ++r) {
        const int at = (warp * kSRounds + r) * 32 + lane;
        if (at < n) pos[r] += wh[warp][digit[r]];
    }
    __syncthreads();
}

// Exclusive prefix sum over the CTA's 32 kWarps threads.
template <int kWarps>
__device__ __forceinline__ int32_t scan_bins(int32_t x, int32_t* sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += y;
    }
    if (lane == 31) sh[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int32_t w = lane < kWarps ? sh[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += y;
        }
        if (lane < kWarps) sh[lane] = w;
    }
    __syncthreads();
    const int32_t r = s - x + (warp > 0 ? sh[warp - 1] : 0);
    __syncthreads();
    return r;
}

// One pass over a tile: reads its keys (ids in the first pass), writes keys and token indices in
// the order of the pass's digit.  Each CTA sums the other tiles' counts itself.
template <int kSRounds>
__global__ void __launch_bounds__(kSThreads) embed_scatter_kernel(
    const int32_t* ids, const uint32_t* keys, const int32_t* idx,
    int64_t N, int32_t V, int shift, uint32_t mask, const int32_t* hist, int tiles,
    uint32_t* keys_out, int32_t* idx_out) {
    __shared__ int32_t wh[kSWarps][kBins];
    __shared__ int32_t sh[32];
    pdl_trigger();
    pdl_wait();
    int32_t all = 0, earlier = 0;
    const int tile = blockIdx.x;
#pragma unroll 8
    for (int t = 0; t < tiles; ++t) {
        const int32_t c = hist[static_cast<int64_t>(t) * kBins + threadIdx.x];
        all += c;
        if (t < tile) earlier += c;
    }
    const int32_t base = scan_bins<kSWarps>(all, sh) + earlier;
    constexpr int kTile = kSThreads * kSRounds;
    const int64_t p0 = static_cast<int64_t>(tile) * kTile;
    const int n = static_cast<int>(min(static_cast<int64_t>(kTile), N - p0));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t key[kSRounds], digit[kSRounds];
    int32_t val[kSRounds], pos[kSRounds];
#pragma unroll
    for (int r = 0; r < kSRounds; ++r) {
        const int at = (warp * kSRounds + r) * 32 + lane;
        key[r] = 0;
        val[r] = 0;
        if (at < n) {
            key[r] = ids ? key_of(ids[p0 + at], V) : keys[p0 + at];
            val[r] = ids ? static_cast<int32_t>(p0 + at) : idx[p0 + at];
        }
        digit[r] = (key[r] >> shift) & mask;
    }
    tile_ranks<kSRounds>(digit, n, base, wh, pos);
#pragma unroll
    for (int r = 0; r < kSRounds; ++r) {
        const int at = (warp * kSRounds + r) * 32 + lane;
        if (at < n) {
            keys_out[pos[r]] = key[r];
            idx_out[pos[r]] = val[r];
        }
    }
}

// The same sort of up to kClusterTokens tokens in one launch: a cluster of eight CTAs, each with an eighth of the list
// in shared memory.  A pass counts, exchanges the counts, and sends each key to its place in the CTA that holds it.
// (8000 tokens onto 4096 x 768, added: 2.4 us less than with the launches above, 16000 1.8; 32000, eight keys a thread,
// 3.4 more.)
constexpr int kCCtas = 8, kCThreads = kBins, kCWarps = kCThreads / 32;  // a thread for each bin
constexpr int kCMost = 4;  // keys of a thread
constexpr int64_t kClusterTokens = static_cast<int64_t>(kCCtas) * kCThreads * kCMost;
template <int kKeys>
constexpr size_t cluster_smem() {
    return kCWarps * kBins * 4 + kBins * 4 + 2ull * kCThreads * kKeys * 8;
}

template <int kKeys>
__global__ void __launch_bounds__(kCThreads) embed_sort_kernel(const int32_t* ids, int32_t N, int32_t V, int bits,
                                                               int passes, uint32_t* keys_out, int32_t* idx_out) {
    extern __shared__ uint64_t csm[];
    constexpr int kTile = kCThreads * kKeys;
    uint64_t* list = csm;  // [2][kTile] key and token
    int32_t(*wh)[kBins] = reinterpret_cast<int32_t(*)[kBins]>(csm + 2 * kTile);
    int32_t* count = reinterpret_cast<int32_t*>(wh + kCWarps);
    __shared__ int32_t sh[32];
    pdl_trigger();
    pdl_wait();
    const int rank = static_cast<int>(blockIdx.x), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t mask = (1u << bits) - 1u, below = (1u << lane) - 1u;
    const int n = max(0, min(kTile, N - rank * kTile));  // of this CTA's part
    for (int pass = 0; pass < passes; ++pass) {
        uint64_t item[kKeys];
        int32_t digit[kKeys], pos[kKeys];
#pragma unroll
        for (int r = 0; r < kKeys; ++r) {
            const int at = (warp * kKeys + r) * 32 + lane;
            item[r] = 0;
            if (at < n) {
                const int32_t t = rank * kTile + at;
                item[r] = pass == 0 ? static_cast<uint64_t>(key_of(ids[t], V)) << 32 | static_cast<uint32_t>(t)
                                    : list[(pass & 1) * kTile + at];
            }
            digit[r] = static_cast<int32_t>(static_cast<uint32_t>(item[r] >> 32) >> (pass * bits) & mask);
        }
        // each key's place among its warp's keys of its digit
#pragma unroll
        for (int w = 0; w < kCWarps; ++w) wh[w][threadIdx.x] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kKeys; ++r) {
            const bool mine = (warp * kKeys + r) * 32 + lane < n;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, mine ? digit[r] : -1);
            int before = 0;
            if (mine) before = wh[warp][digit[r]];
            __syncwarp();
            pos[r] = before + __popc(same & below);
            if (mine && (same & below) == 0) wh[warp][digit[r]] = before + __popc(same);
            __syncwarp();
        }
        __syncthreads();
        const int bin = threadIdx.x;
        int32_t have[kCWarps], all = 0, earlier = 0;
#pragma unroll
        for (int w = 0; w < kCWarps; ++w) have[w] = wh[w][bin];
#pragma unroll
        for (int w = 0; w < kCWarps; ++w) all += have[w];
        count[bin] = all;
        cluster_arrive();
        cluster_wait();
        int32_t c[kCCtas];
#pragma unroll
        for (int k = 0; k < kCCtas; ++k) {
            uint32_t from;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(smem_u32(count + bin)), "r"(k));
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c[k]) : "r"(from) : "memory");
        }
        all = 0;
#pragma unroll
        for (int k = 0; k < kCCtas; ++k) {
            all += c[k];
            if (k < rank) earlier += c[k];
        }
        int32_t run = scan_bins<kCWarps>(all, sh) + earlier;
#pragma unroll
        for (int w = 0; w < kCWarps; ++w) {
            wh[w][bin] = run;
            run += have[w];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kKeys; ++r) {
            if ((warp * kKeys + r) * 32 + lane >= n) continue;
            const int32_t to = pos[r] + wh[warp][digit[r]];
            if (pass + 1 == passes) {
                keys_out[to] = static_cast<uint32_t>(item[r] >> 32);
                idx_out[to] = static_cast<int32_t>(static_cast<uint32_t>(item[r]));
            } else {
                uint32_t there;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(there)
                             : "r"(smem_u32(list + ((pass + 1) & 1) * kTile + to % kTile)), "r"(to / kTile));
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(there), "l"(item[r]) : "memory");
            }
        }
        // the keys are in place, and the counts have been read
        cluster_arrive();
        cluster_wait();
    }
}

template <int kKeys>
bool launch_cluster_sort(const int32_t* ids, int64_t N, int32_t V, int bits, int passes, uint32_t* keys, int32_t* idx,
                         cudaStream_t s) {
    static PerContextOnce attr;
    if (!attr.run([] {
            return cudaFuncSetAttribute(embed_sort_kernel<kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(cluster_smem<kKeys>())) == cudaSuccess;
        }))
        return false;
    return dependent_launch(embed_sort_kernel<kKeys>, dim3(kCCtas), kCThreads, cluster_smem<kKeys>(), s, kCCtas, ids,
                            static_cast<int32_t>(N), V, bits, passes, keys, idx);
}

// ------------------------------------------------------------------ the sums
constexpr int kGThreads = 256;
constexpr int kGWarps = kGThreads / 32;
constexpr int kZeroRows = 16;  // table rows that one clearing CTA looks after (8: 171 us in place of 155, 64: 166)

struct GradArgs {
    const uint32_t* key;  // sorted
    const int32_t* idx;
    const void* g;
    float* G;
    float* head;  // [chunks, dpad]: sums of ids that began in an earlier chunk
    float* tail;  // [chunks, dpad]: sums of ids that begin in the chunk and go on past its end
    int64_t ld_g, ld_G, N, units;
    int32_t V, d, dpad, slabs, chunk, chunks, accumulate;
    float scale;
};

template <typename T>
struct Lane;  // what one lane sums: 16 bytes of a row
template <>
struct Lane<float> {
    static constexpr int kN = 4;
    using Raw = float4;
    static __device__ __forceinline__ Raw raw(const uint4& w) {
        return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ void add(float (&a)[4], const Raw& r) {
        a[0] += r.x;
        a[1] += r.y;
        a[2] += r.z;
        a[3] += r.w;
    }
    static __device__ __forceinline__ Raw tail(const float* p, int n) {
        return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, 0.f);
    }
};
template <>
struct Lane<__nv_bfloat16> {
    static constexpr int kN = 8;
    using Raw = uint4;
    static __device__ __forceinline__ Raw raw(const uint4& w) { return w; }
    static __device__ __forceinline__ void add(float (&a)[8], const Raw& r) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[2 * j] += bf_lo(w[j]);
            a[2 * j + 1] += bf_hi(w[j]);
        }
    }
    static __device__ __forceinline__ Raw tail(const __nv_bfloat16* p, int n) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n) w[j >> 1] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[j])) << (16 * (j & 1));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Writes or adds a finished row piece.  Each element gets one addition in the whole call, so the
// reductions (which the warp does not wait for, unlike a load of the old row) leave no order open.  They take values
// and results below 2^-126 as zero, which a load and a store would not, in up to 1.4 times the time (2000 tokens
// onto 4096 x 768 11.5 us from 9.1, 65536 of fp32 onto 65536 x 2048 232 from 162).
template <int kN>
__device__ __forceinline__ void put_row(float* row, const float (&a)[kN], int n, float scale, bool accumulate) {
    if (n >= kN) {
#pragma unroll
        for (int j = 0; j < kN; j += 4) {
            const float4 w = make_float4(a[j] * scale, a[j + 1] * scale, a[j + 2] * scale, a[j + 3] * scale);
            if (accumulate)
                asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(row + j), "f"(w.x), "f"(w.y),
                             "f"(w.z), "f"(w.w)
                             : "memory");
            else
                *reinterpret_cast<float4*>(row + j) = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kN; ++j)
            if (j < n) row[j] = accumulate ? row[j] + a[j] * scale : a[j] * scale;
    }
}
template <int kN>
__device__ __forceinline__ void put_partial(float* row, const float (&a)[kN]) {
#pragma unroll
    for (int j = 0; j < kN / 4; ++j)
        reinterpret_cast<float4*>(row)[j] = make_float4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]);
}

// The pieces of the rows of eight tokens, n columns of them left.  No condition stands around the loads of whole pieces:
// with one around each they waited for one another (65536 tokens onto 4096 x 768 61.5 us, then 64.0).
template <typename T>
__device__ __forceinline__ void load_rows(typename Lane<T>::Raw (&raw)[8], const T* g, const int32_t (&t)[8], int64_t ld, int n) {
    if (n >= Lane<T>::kN) {
#pragma unroll
        for (int j = 0; j < 8; ++j) raw[j] = Lane<T>::raw(load_once(g + t[j] * ld));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) raw[j] = n > 0 ? Lane<T>::tail(g + t[j] * ld, n) : typename Lane<T>::Raw{};
    }
}

template <typename T>
__global__ void __launch_bounds__(kGThreads) embed_grad_kernel(const __grid_constant__ GradArgs A) {
    constexpr int kN = Lane<T>::kN;
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t sum_blocks = (A.units + kGWarps - 1) / kGWarps;
    if (static_cast<int64_t>(blockIdx.x) >= sum_blocks) {
        // clear the rows of [r0, r0 + kZeroRows) that no token names
        __shared__ bool absent[kZeroRows];
        const int64_t r0 = (static_cast<int64_t>(blockIdx.x) - sum_blocks) * kZeroRows;
        if (threadIdx.x < kZeroRows) {
            const uint32_t v = static_cast<uint32_t>(r0 + threadIdx.x);
            int64_t lo = 0, hi = A.N;  // first position whose key is >= v
            while (lo < hi) {
                const int64_t mid = (lo + hi) >> 1;
                if (A.key[mid] < v)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            absent[threadIdx.x] = r0 + threadIdx.x < A.V && (lo == A.N || A.key[lo] != v);
        }
        __syncthreads();
        for (int r = warp; r < kZeroRows; r += kGWarps) {
            if (!absent[r]) continue;
            float* row = A.G + (r0 + r) * A.ld_G;
            for (int c = 4 * lane; c < A.d; c += 128) {
                if (c + 4 <= A.d)
                    *reinterpret_cast<float4*>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
                else
                    for (int j = c; j < A.d; ++j) row[j] = 0.f;
            }
        }
        return;
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kGWarps + warp;
    if (unit >= A.units) return;
    const int64_t c = unit / A.slabs;
    const int col = static_cast<int>(unit - c * A.slabs) * (32 * kN) + kN * lane;
    const int n = A.d - col;  // columns left, this lane's own among them
    const int64_t p0 = c * A.chunk, p1 = min(A.N, p0 + A.chunk);
    const uint32_t none = static_cast<uint32_t>(A.V);
    uint32_t cur = A.key[p0];
    bool began_before = p0 > 0 && A.key[p0 - 1] == cur;
    const T* g = static_cast<const T*>(A.g) + col;
    float acc[kN] = {};
    for (int64_t q = p0; q < p1 && cur != none; q += 32) {
        const int cnt = static_cast<int>(min(static_cast<int64_t>(32), p1 - q));
        uint32_t my_key = none;
        int32_t my_idx = 0;
        if (lane < cnt) {
            my_key = A.key[q + lane];
            my_idx = A.idx[q + lane];
        }
        for (int b = 0; b < cnt; b += 8) {
            typename Lane<T>::Raw raw[8];
            int32_t t[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = __shfl_sync(0xFFFFFFFFu, my_idx, b + j);
            load_rows<T>(raw, g, t, A.ld_g, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t k = __shfl_sync(0xFFFFFFFFu, my_key, b + j);
                if (b + j >= cnt || cur == none) break;  // uniform over the warp
                if (k != cur) {
                    if (n > 0) {
                        if (began_before)
                            put_partial(A.head + c * A.dpad + col, acc);
                        else
                            put_row(A.G + static_cast<int64_t>(cur) * A.ld_G + col, acc, n, A.scale, A.accumulate != 0);
                    }
                    began_before = false;
                    cur = k;
#pragma unroll
                    for (int i = 0; i < kN; ++i) acc[i] = 0.f;
                    if (cur == none) break;
                }
                Lane<T>::add(acc, raw[j]);
            }
        }
    }
    if (cur == none || n <= 0) return;
    const bool goes_on = p1 < A.N && A.key[p1] == cur;
    if (began_before)
        put_partial(A.head + c * A.dpad + col, acc);
    else if (goes_on)
        put_partial(A.tail + c * A.dpad + col, acc);
    else
        put_row(A.G + static_cast<int64_t>(cur) * A.ld_G + col, acc, n, A.scale, A.accumulate != 0);
}

// CTA (chunk, kJoinCols columns): if an id begins in the chunk and goes on past its end, adds its partial
// sums.  Four groups of the CTA's threads take consecutive runs of chunks, each summed in order
// (32000 tokens onto 4096 x 768 40.3 us; two groups, of twice the columns, 42.4).
constexpr int kJoinCols = 256;
constexpr int kJoinThreads = kJoinCols / 4, kJoinGroups = kGThreads / kJoinThreads;
__global__ void __launch_bounds__(kGThreads) embed_join_kernel(const __grid_constant__ GradArgs A, int32_t slabs) {
    pdl_trigger();
    pdl_wait();
    const int64_t c = blockIdx.x / slabs;
    const int64_t p0 = c * A.chunk, p1 = p0 + A.chunk;
    if (p1 >= A.N) return;
    const uint32_t cur = A.key[p1 - 1], after = A.key[p1];
    const uint32_t before = p0 > 0 ? A.key[p0 - 1] : ~cur;
    if (cur == static_cast<uint32_t>(A.V) || after != cur || before == cur) return;
    __shared__ float4 part[kGThreads];
    const int group = threadIdx.x / kJoinThreads, at = threadIdx.x % kJoinThreads;
    const int col = static_cast<int>(blockIdx.x - c * slabs) * kJoinCols + 4 * at;
    // chunks c + 1 .. lo - 1 begin with this id
    int64_t lo = c + 1;
    for (int more = kGThreads; more == kGThreads; lo += more) {
        const int64_t k = lo + threadIdx.x;
        more = __syncthreads_count(k < A.chunks && A.key[k * A.chunk] == cur);
    }
    const int64_t per = (lo - c - 1 + kJoinGroups - 1) / kJoinGroups, from = c + 1 + group * per;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < A.dpad) {
        if (group == 0) s = *reinterpret_cast<const float4*>(A.tail + c * A.dpad + col);
#pragma unroll 8
        for (int64_t k = from; k < min(lo, from + per); ++k) {
            const float4 h = *reinterpret_cast<const float4*>(A.head + k * A.dpad + col);
            s = make_float4(s.x + h.x, s.y + h.y, s.z + h.z, s.w + h.w);
        }
    }
    part[threadIdx.x] = s;
    __syncthreads();
    if (group == 0 && col < A.d) {
        float acc[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int g = 1; g < kJoinGroups; ++g) {
            const float4 h = part[g * kJoinThreads + at];
            acc[0] += h.x, acc[1] += h.y, acc[2] += h.z, acc[3] += h.w;
        }
        put_row(A.G + static_cast<int64_t>(cur) * A.ld_G + col, acc, A.d - col, A.scale, A.accumulate != 0);
    }
}

// ------------------------------------------------------------------ small batches in one launch
constexpr int kSmallTokens = DUST_EMBEDDING_SMALL;
constexpr int kRankTokens = 512;  // up to which a share is sorted by rank (2000 tokens 9.1 us in a graph, bitonic 11.5)

struct SmallArgs {
    const int32_t* ids;
    const void* g;
    float* G;
    int64_t ld_g, ld_G;
    int32_t N, V, d, shares, accumulate;  // shares: a power of two
    float scale;
};

// CTA (share, 32 kN columns).  Keys are (id, token), all different, so that sorting them orders each id's
// tokens; the eight warps sum consecutive runs of the sorted list and join the ids that cross runs.
template <typename T>
__global__ void __launch_bounds__(kGThreads) embed_grad_small_kernel(const __grid_constant__ SmallArgs A) {
    constexpr int kN = Lane<T>::kN;
    extern __shared__ uint64_t list[];  // [kSmallTokens]
    __shared__ float first[kGWarps][32 * kN], last[kGWarps][32 * kN];
    int32_t* count = reinterpret_cast<int32_t*>(first);  // until the list is complete
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t share = static_cast<int32_t>(blockIdx.x);
    pdl_trigger();
    pdl_wait();

    // this share's tokens, in any order: the sort puts them right
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
    for (int t0 = 0; t0 < A.N; t0 += 4 * kGThreads) {
        int32_t id[4];  // on their way together (2000 tokens 9.2 us in a graph, one at a time 10.2)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + j * kGThreads + threadIdx.x;
            id[j] = t < A.N ? A.ids[t] : -1;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool mine = id[j] >= 0 && id[j] < A.V && (id[j] & (A.shares - 1)) == share;
            const uint32_t vote = __ballot_sync(0xFFFFFFFFu, mine);
            if (vote == 0) continue;  // uniform over the warp
            int at = 0;
            if (lane == 0) at = atomicAdd(count, __popc(vote));
            at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(vote & ((1u << lane) - 1u));
            if (mine)
                list[at] = (static_cast<uint64_t>(id[j]) << 32) | static_cast<uint32_t>(t0 + j * kGThreads + threadIdx.x);
        }
    }
    __syncthreads();
    const int n = *count;
    __syncthreads();  // count's memory is used again
    const uint64_t* sorted = list;
    if (n <= kRankTokens) {
        // few keys: each one's place is the number of smaller ones
        uint64_t* to = list + kSmallTokens / 2;
        static_assert(kRankTokens == 2 * kGThreads, "up to two keys a thread");
        const int i = threadIdx.x, i2 = i + kGThreads;
        const uint64_t k = i < n ? list[i] : 0, k2 = i2 < n ? list[i2] : 0;
        int place = 0, place2 = 0;
        if (n <= kGThreads) {
#pragma unroll 8
            for (int j = 0; j < n; ++j) place += list[j] < k;
        } else {  // both in one go (3000 tokens 15.0 us, one after the other 16.6)
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                const uint64_t other = list[j];
                place += other < k;
                place2 += other < k2;
            }
        }
        if (i < n) to[place] = k;
        if (i2 < n) to[place2] = k2;
        sorted = to;
        __syncthreads();
    } else {  // bitonic
        int size = 1;
        while (size < n) size <<= 1;
        for (int i = n + threadIdx.x; i < size; i += kGThreads) list[i] = ~0ull;  // sorts behind all
        __syncthreads();
        for (int k = 2; k <= size; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
                for (int i = threadIdx.x; i < size / 2; i += kGThreads) {
                    const int a = 2 * i - (i & (j - 1)), b = a + j;
                    const uint64_t x = list[a], y = list[b];
                    if ((x > y) == ((a & k) == 0)) {
                        list[a] = y;
                        list[b] = x;
                    }
                }
                __syncthreads();
            }
    }

    const int col = static_cast<int>(blockIdx.y) * (32 * kN) + kN * lane;
    const int left = A.d - col;
    const T* g = static_cast<const T*>(A.g) + col;
    // warp w: positions [p0, p1) of the list
    const int per = (n + kGWarps - 1) / kGWarps;
    const int p0 = min(n, warp * per), p1 = min(n, p0 + per);
    auto key = [&](int p) { return static_cast<int32_t>(sorted[p] >> 32); };
    if (p0 < p1) {
        int32_t cur = key(p0);
        bool began_before = p0 > 0 && key(p0 - 1) == cur;
        float acc[kN] = {};
        for (int p = p0; p < p1; p += 8) {
            typename Lane<T>::Raw raw[8];
            int32_t t[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = static_cast<int32_t>(static_cast<uint32_t>(sorted[min(p + j, p1 - 1)]));
            load_rows<T>(raw, g, t, A.ld_g, left);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (p + j >= p1) break;
                const int32_t k = key(p + j);
                if (k != cur) {
                    if (began_before) {
#pragma unroll
                        for (int i = 0; i < kN; ++i) first[warp][kN * lane + i] = acc[i];
                    } else if (left > 0) {
                        put_row(A.G + static_cast<int64_t>(cur) * A.ld_G + col, acc, left, A.scale, A.accumulate != 0);
                    }
                    began_before = false;
                    cur = k;
#pragma unroll
                    for (int i = 0; i < kN; ++i) acc[i] = 0.f;
                }
                Lane<T>::add(acc, raw[j]);
            }
        }
        const bool goes_on = p1 < n && key(p1) == cur;
        if (began_before) {
#pragma unroll
            for (int i = 0; i < kN; ++i) first[warp][kN * lane + i] = acc[i];
        } else if (goes_on) {
#pragma unroll
            for (int i = 0; i < kN; ++i) last[warp][kN * lane + i] = acc[i];
        } else if (left > 0) {
            put_row(A.G + static_cast<int64_t>(cur) * A.ld_G + col, acc, left, A.scale, A.accumulate != 0);
        }
    }
    __syncthreads();
    // the warp in whose run an id begins that goes on past it adds the later runs' shares in order
    if (p0 < p1 && p1 < n) {
        const int32_t cur = key(p1 - 1);
        if (key(p1) == cur && !(p0 > 0 && key(p0 - 1) == cur) && left > 0) {
            float acc[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) acc[i] = last[warp][kN * lane + i];
            for (int w = warp + 1; w < kGWarps && w * per < n && key(w * per) == cur; ++w)
#pragma unroll
                for (int i = 0; i < kN; ++i) acc[i] += first[w][kN * lane + i];
            put_row(A.G + static_cast<int64_t>(cur) * A.ld_G + col, acc, left, A.scale, A.accumulate != 0);
        }
    }
    if (A.accumulate) return;
    // clear this share's rows that no token names: each lane looks for one row, the warp clears them
    const int64_t rows = (static_cast<int64_t>(A.V) - share + A.shares - 1) / A.shares;  // share + k shares < V
    for (int64_t k0 = 32 * warp; k0 < rows; k0 += 32 * kGWarps) {
        const int64_t k = k0 + lane;
        bool absent = false;
        if (k < rows) {
            const uint64_t v = static_cast<uint64_t>(share + k * A.shares) << 32;
            int lo = 0, hi = n;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sorted[mid] < v)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            absent = lo == n || (sorted[lo] >> 32) != (v >> 32);
        }
        uint32_t todo = __ballot_sync(0xFFFFFFFFu, absent);
        const float zero[kN] = {};
        while (todo) {
            const int b = __ffs(todo) - 1;
            todo &= todo - 1;
            if (left > 0) put_row(A.G + (share + (k0 + b) * A.shares) * A.ld_G + col, zero, left, 1.0f, false);
        }
    }
}

template <typename T>
dust_status launch_small(const SmallArgs& A, int slabs, cudaStream_t s) {
    return dependent_launch(embed_grad_small_kernel<T>, dim3(static_cast<unsigned>(A.shares), static_cast<unsigned>(slabs)),
                            kGThreads, kSmallTokens * 8, s, 1, A)
               ? DUST_OK
               : DUST_ERR_CUDA;
}

struct GradPlan {
    int64_t N;
    int slabs, chunk, chunks, tiles, dpad, passes, bits;
    size_t keys, hist, part;  // bytes of one array of each kind
};

// Chunk length: about 24 warps for each SM, between 32 and 1024 positions; 16 while those leave no more than 36 warps for
// each SM (8000 tokens onto 4096 x 768, added: 20.7 us in a graph, with 32 23.2; 16000 30.9 and 29.1).
GradPlan grad_plan(dust_dtype dt, int64_t N, int32_t V, int32_t d) {
    GradPlan p{};
    p.N = N;
    const int cols = dt == DUST_BF16 ? 256 : 128;
    p.slabs = (d + cols - 1) / cols;
    const int64_t want = std::max<int64_t>(1, static_cast<int64_t>(num_sms()) * 24 / p.slabs);
    int64_t c = N <= 24 * want ? 16 : 32;
    while (c < 1024 && N / (2 * c) >= want) c *= 2;
    p.chunk = static_cast<int>(c);
    p.chunks = static_cast<int>((N + c - 1) / c);
    const int tile = kSThreads * (N < kManyTokens ? kFewRounds : kManyRounds);
    p.tiles = static_cast<int>((N + tile - 1) / tile);
    p.dpad = (d + 7) / 8 * 8;
    int bits = 1;  // of the keys 0 .. V
    while (bits < 31 && (static_cast<int64_t>(V) >> bits) != 0) ++bits;
    p.passes = (bits + kBinBits - 1) / kBinBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.keys = align_up(static_cast<size_t>(N) * 4, 256);
    p.hist = align_up(static_cast<size_t>(p.tiles) * kBins * 4, 256);
    p.part = align_up(static_cast<size_t>(p.chunks) * p.dpad * 4, 256);
    return p;
}

template <typename TE, typename TO>
bool launch_lookup(const int32_t* ids, const void* E, int64_t ld_E, int64_t N, int32_t V, int32_t d, float scale,
                   void* out, int64_t ld_out, unsigned blocks, int32_t nv, cudaStream_t s) {
    return dependent_launch(embedding_kernel<TE, TO>, dim3(blocks), kFThreads, 0, s, 1, ids, static_cast<const TE*>(E), ld_E,
                            N, V, d, nv, div_magic(nv), scale, static_cast<TO*>(out), ld_out);
}

}  // namespace

dust_status embedding_launch(const int32_t* ids, const void* E, dust_dtype dt, int64_t ld_E, int64_t N, int32_t V,
                             int32_t d, float scale, void* out, dust_dtype out_dt, int64_t ld_out,
                             cudaStream_t s) {
    const int32_t nv = (d + 7) / 8;
    const int64_t blocks = (N * nv + kFThreads * kFItems - 1) / (kFThreads * kFItems);
    if (blocks > 2147483647LL) return DUST_ERR_UNSUPPORTED;
    const unsigned nb = static_cast<unsigned>(blocks);
    prof_begin(s);
    using bf16 = __nv_bfloat16;
    const bool ok =
        dt == DUST_BF16
            ? (out_dt == DUST_BF16 ? launch_lookup<bf16, bf16>(ids, E, ld_E, N, V, d, scale, out, ld_out, nb, nv, s)
                                   : launch_lookup<bf16, float>(ids, E, ld_E, N, V, d, scale, out, ld_out, nb, nv, s))
            : (out_dt == DUST_BF16 ? launch_lookup<float, bf16>(ids, E, ld_E, N, V, d, scale, out, ld_out, nb, nv, s)
                                   : launch_lookup<float, float>(ids, E, ld_E, N, V, d, scale, out, ld_out, nb, nv, s));
    prof_end(s, "embedding");
    return ok ? DUST_OK : DUST_ERR_CUDA;
}

size_t embedding_grad_workspace_bytes(dust_dtype dt, int64_t N, int32_t V, int32_t d) {
    if (N <= kSmallTokens) return 0;
    const GradPlan p = grad_plan(dt, N, V, d);
    return 4 * p.keys + p.hist + 2 * p.part;
}

dust_status embedding_grad_launch(const int32_t* ids, const void* g, dust_dtype dt, int64_t ld_g, int64_t N,
                                  int32_t V, int32_t d, float scale, float* G, int64_t ld_G, int accumulate,
                                  void* ws, cudaStream_t s) {
    const GradPlan p = grad_plan(dt, N, V, d);
    if (N <= kSmallTokens) {
        // two to four CTAs an SM: more look through the ids once more each, fewer leave an SM's loads waiting (2000
        // tokens onto 4096 x 768, added: 8.9 us, one to two 9.1, five to ten 9.7; 4000 tokens 17.6, 19.2 and 18.5)
        int shares = 1;
        while (shares < 512 && static_cast<int64_t>(shares) * p.slabs < static_cast<int64_t>(num_sms()) * 2) shares *= 2;
        const SmallArgs A{ids, g, G, ld_g, ld_G, static_cast<int32_t>(N), V, d, shares, accumulate, scale};
        if (p.slabs > 65535) return DUST_ERR_UNSUPPORTED;
        prof_begin(s);
        const dust_status st = dt == DUST_BF16 ? launch_small<__nv_bfloat16>(A, p.slabs, s)
                                               : launch_small<float>(A, p.slabs, s);
        prof_end(s, "embedding_grad_small");
        return st;
    }
    char* w = static_cast<char*>(ws);
    uint32_t* key[2] = {reinterpret_cast<uint32_t*>(w), reinterpret_cast<uint32_t*>(w + p.keys)};
    int32_t* idx[2] = {reinterpret_cast<int32_t*>(w + 2 * p.keys), reinterpret_cast<int32_t*>(w + 3 * p.keys)};
    int32_t* hist = reinterpret_cast<int32_t*>(w + 4 * p.keys);
    float* head = reinterpret_cast<float*>(w + 4 * p.keys + p.hist);
    float* tail = reinterpret_cast<float*>(w + 4 * p.keys + p.hist + p.part);
    const uint32_t mask = (1u << p.bits) - 1u;
    int at = 1;  // where the sorted list ends up
    if (N <= kClusterTokens) {
        const int per = kCCtas * kCThreads;
        prof_begin(s);
        const bool ok = N <= 2 * per ? launch_cluster_sort<2>(ids, N, V, p.bits, p.passes, key[at], idx[at], s)
                                     : launch_cluster_sort<kCMost>(ids, N, V, p.bits, p.passes, key[at], idx[at], s);
        prof_end(s, "embedding_sort");
        if (!ok) return DUST_ERR_CUDA;
    }
    for (int pass = 0; N > kClusterTokens && pass < p.passes; ++pass) {
        const int32_t* first = pass == 0 ? ids : nullptr;
        const int to = at ^ 1, shift = pass * p.bits;
        const bool few = N < kManyTokens;
        const uint32_t* key_in = key[at];
        const int32_t *idx_in = idx[at], *hist_in = hist;
        prof_begin(s);
        bool ok = dependent_launch(few ? embed_hist_kernel<kFewRounds> : embed_hist_kernel<kManyRounds>, dim3(p.tiles),
                                   kSThreads, 0, s, 1, first, key_in, N, V, shift, mask, hist);
        prof_end(s, "embedding_sort_count");
        prof_begin(s);
        ok = ok && dependent_launch(few ? embed_scatter_kernel<kFewRounds> : embed_scatter_kernel<kManyRounds>,
                                    dim3(p.tiles), kSThreads, 0, s, 1, first, key_in, idx_in, N, V, shift, mask, hist_in,
                                    p.tiles, key[to], idx[to]);
        prof_end(s, "embedding_sort");
        if (!ok) return DUST_ERR_CUDA;
        at = to;
    }
    GradArgs A{};
    A.key = key[at];
    A.idx = idx[at];
    A.g = g;
    A.G = G;
    A.head = head;
    A.tail = tail;
    A.ld_g = ld_g;
    A.ld_G = ld_G;
    A.N = N;
    A.V = V;
    A.d = d;
    A.dpad = p.dpad;
    A.slabs = p.slabs;
    A.chunk = p.chunk;
    A.chunks = p.chunks;
    A.units = static_cast<int64_t>(p.chunks) * p.slabs;
    A.accumulate = accumulate;
    A.scale = scale;
    const int64_t zero_blocks = accumulate ? 0 : (static_cast<int64_t>(V) + kZeroRows - 1) / kZeroRows;
    const int64_t blocks = (A.units + kGWarps - 1) / kGWarps + zero_blocks;
    const int join_slabs = (d + kJoinCols - 1) / kJoinCols;
    if (blocks > 2147483647LL || static_cast<int64_t>(p.chunks) * join_slabs > 2147483647LL)
        return DUST_ERR_UNSUPPORTED;
    prof_begin(s);
    bool ok = dependent_launch(dt == DUST_BF16 ? embed_grad_kernel<__nv_bfloat16> : embed_grad_kernel<float>,
                               dim3(static_cast<unsigned>(blocks)), kGThreads, 0, s, 1, A);
    prof_end(s, "embedding_grad");
    if (ok && p.chunks > 1) {
        prof_begin(s);
        ok = dependent_launch(embed_join_kernel, dim3(static_cast<unsigned>(p.chunks * join_slabs)), kGThreads, 0, s, 1, A,
                              join_slabs);
        prof_end(s, "embedding_grad_join");
    }
    return ok ? DUST_OK : DUST_ERR_CUDA;
}

}  // namespace dust
