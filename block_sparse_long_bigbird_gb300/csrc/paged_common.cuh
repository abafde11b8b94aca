// What the kernels of the paged attention share: the plan (how a call's
// sweeps are cut into units), the walk over a unit's 64-key blocks, the mask
// of a row against a block, and an exact path for rows that ordinary
// arithmetic spoils.
//
// A unit is one tile of query rows (a few tokens times the query heads of one
// key head) against one stretch of the 64-key blocks that any of its rows may
// see. The lengths live on the device, so no host code can cut the sweeps:
// every CTA reads them (at most kPagedMaxBatch) and computes the same plan in
// shared memory. That costs about a microsecond, where a planning kernel of
// its own would cost a launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"
#include "paged.h"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

// Lets a kernel use up to the largest dynamic shared memory, once per device.
template <typename K>
inline cudaError_t allow_smem(K kern, std::atomic<bool> (&done)[64], size_t bytes) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

constexpr unsigned kAllLanes = 0xffffffffu;

__device__ __forceinline__ uint64_t low_bits(int c) {  // bits [0, c), c clamped to [0, 64]
    return c <= 0 ? 0ull : (c >= 64 ? ~0ull : ((1ull << c) - 1ull));
}

__device__ __forceinline__ bool not_finite(float x) { return !(fabsf(x) <= 3.402823466e38f); }

// The plan in shared memory. Arrays over sequences, then the global list.
struct Plan {
    int *q, *s;        // [B] new tokens and tokens in the cache (q = 0 for a refused sequence)
    int *ns;           // [B] splits of each of the sequence's sweeps
    int *ubase;        // [B + 1] first unit
    int *sbase;        // [B + 1] first partial-result slot
    int *gpos;         // [ng] global positions
    int *gblk;         // [ngb] 64-key blocks that hold one, ascending
    uint64_t *gbit;    // [ngb] which of their keys
    int *misc;         // [0] ngb, [1] longest stride of a dilated head, [2] longest sweep, [4 + 2 k] costs of kCuts
    int ngb, max_stride;
};

// Splits tried for the longest sweep.
constexpr int kCuts = 16;
__device__ __forceinline__ int cut_of(int k) {
    return k < 6 ? k + 1 : k < 9 ? 2 * k - 4 : k < 10 ? 16 : k < 11 ? 24 : k < 12 ? 32 : k < 13 ? 48 : k < 14 ? 64 : k < 15 ? 96 : 128;
}

__host__ __device__ inline size_t plan_bytes(int B, int ng) {
    const size_t ints = 5 * (size_t)B + 2 + 2 * (size_t)ng + 4 + kCuts;
    return ((ints * 4 + 15) & ~(size_t)15) + (size_t)ng * 8;
}

__device__ __forceinline__ Plan plan_at(void *smem, int B, int ng) {
    Plan P;
    P.gbit = reinterpret_cast<uint64_t *>(smem);
    int *w = reinterpret_cast<int *>(P.gbit + ng);
    P.q = w;
    P.s = w + B;
    P.ns = w + 2 * B;
    P.ubase = w + 3 * B;
    P.sbase = w + 4 * B + 1;
    P.gpos = w + 5 * B + 2;
    P.gblk = P.gpos + ng;
    P.misc = P.gblk + ng;
    P.ngb = 0;
    P.max_stride = 1;
    return P;
}

// Stride of a query head (dilation + 1); out-of-range entries count as 1.
__device__ __forceinline__ int head_stride(const PagedProblem &p, int h) {
    if (!p.dilation) return 1;
    const int v = __ldg(p.dilation + h);
    if (v < 0 || v > kMaxDilation) {
        atomicOr(p.status, kDevBadIndex);
        return 1;
    }
    return v + 1;
}

// Keys before the query that a head's window reaches.
__device__ __forceinline__ int head_reach(const PagedProblem &p, int stride) {
    const long long r = (long long)p.half * stride;
    return r > kPagedMaxLen ? (int)kPagedMaxLen : (int)r;
}

// First entry of the ascending list a[0..n) that is >= v.
__device__ __forceinline__ int lower_bound(const int *a, int n, int v) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] < v) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// Upper estimate of the 64-key blocks that one tile of a sequence walks.
__device__ __forceinline__ int estimate_blocks(const PagedProblem &p, const Plan &P, int q, int s) {
    if (q == 0) return 0;
    const int all = (s + 63) >> 6;
    const long long span = (long long)head_reach(p, P.max_stride) + min(q, p.tpt);
    const long long band = (span >> 6) + 2 + P.ngb;
    return band < all ? (int)band : all;
}

// Computed by the whole CTA. Ends with a barrier.
__device__ inline void make_plan(const PagedProblem &p, Plan &P) {
    const int tid = threadIdx.x, lane = tid & 31, nthr = blockDim.x;
    for (int b = tid; b < p.B; b += nthr) {
        int q = p.qlens ? __ldg(p.qlens + b) : p.m, s = __ldg(p.lens + b);
        if (q < 0 || q > p.m || s < q || (long long)s > ((long long)p.max_pages << p.log_page)) {
            atomicOr(p.status, kDevBadIndex);
            q = s = 0;
        }
        P.q[b] = q;
        P.s[b] = s;
    }
    // the global list: a block starts where the block number changes; entries
    // that break the order are skipped (the call's result is then unspecified)
    for (int i = tid; i < p.ng; i += nthr) {
        int v = __ldg(p.gidx + i);
        if (v < 0 || v >= kPagedMaxLen || (i > 0 && __ldg(p.gidx + i - 1) >= v)) {
            atomicOr(p.status, kDevBadIndex);
            v = -1;
        }
        P.gpos[i] = v;
    }
    if (tid == 0) {
        P.misc[1] = 1;
        P.misc[2] = 0;
    }
    __syncthreads();
    if (p.dilation)
        for (int h = tid; h < p.Hq; h += nthr) atomicMax(&P.misc[1], head_stride(p, h));
    if (tid < 32) {
        int n = 0, kept = 0, last = -1;  // blocks and entries so far, the last entry's block
        for (int i0 = 0; i0 < p.ng; i0 += 32) {
            const int v = i0 + lane < p.ng ? P.gpos[i0 + lane] : -1;
            const unsigned good = __ballot_sync(kAllLanes, v >= 0), below = (1u << lane) - 1u;
            const int blk = v >> 6, src = good & below ? 31 - __clz(good & below) : -1;
            const int before = __shfl_sync(kAllLanes, blk, src < 0 ? 0 : src);
            const bool head = v >= 0 && blk != (src < 0 ? last : before);
            const unsigned heads = __ballot_sync(kAllLanes, head);
            const int at = n + __popc(heads & (below | (1u << lane))) - 1;
            if (head) {
                P.gblk[at] = blk;
                P.gbit[at] = 0ull;
            }
            __syncwarp();
            if (v >= 0) {
                P.gpos[kept + __popc(good & below)] = v;
                atomicOr(reinterpret_cast<unsigned long long *>(P.gbit + at), 1ull << (v & 63));
            }
            __syncwarp();
            if (good) last = __shfl_sync(kAllLanes, blk, 31 - __clz(good));
            n += __popc(heads);
            kept += __popc(good);
        }
        for (int i = kept + lane; i < p.ng; i += 32) P.gpos[i] = 0x7fffffff;
        if (lane == 0) P.misc[0] = n;
    }
    __syncthreads();
    P.ngb = P.misc[0];
    P.max_stride = P.misc[1];
    // The longest sweep, then what each way of cutting it (and the others into
    // pieces as long) would cost: rounds of `slots` units of mean length, and a
    // last round as long as the longest piece. A split unit costs more, as it
    // writes partial results that are read again.
    int len = 0x3fffffff;
    if (p.cut) {
        const int warp = tid >> 5, nwarps = nthr >> 5;
        if (tid < p.B) {
            int e = 0;
            for (int b = tid; b < p.B; b += nthr) e = max(e, estimate_blocks(p, P, P.q[b], P.s[b]));
            atomicMax(&P.misc[2], e);
        }
        __syncthreads();
        const int longest = P.misc[2];
        for (int k = warp; k < kCuts; k += nwarps) {
            const int piece = (longest + cut_of(k) - 1) / cut_of(k);
            int units = 0, parts = 0;
            long long total = 0;
            for (int b = lane; b < p.B; b += 32) {
                const int n = (P.q[b] + p.tpt - 1) / p.tpt * p.Hkv;
                const int e = estimate_blocks(p, P, P.q[b], P.s[b]);
                const int ns = piece > 0 && e > piece ? (e + piece - 1) / piece : 1;
                units += n * ns;
                parts += ns > 1 ? n * ns : 0;
                total += (long long)n * e;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                units += __shfl_xor_sync(kAllLanes, units, o);
                parts += __shfl_xor_sync(kAllLanes, parts, o);
                total += __shfl_xor_sync(kAllLanes, total, o);
            }
            if (lane == 0) {
                // in 1/16 blocks; a cut that is too short or needs too much scratch is out
                const long long own = 16 * total + 16ll * (units - parts) * p.cost_plain + 16ll * parts * p.cost_split;
                const int u = max(units, 1);
                const long long mean = own / u;
                long long cost = (long long)((u + p.slots - 1) / p.slots) * mean + 16ll * piece - 16 * total / u;
                if (k > 0 && (piece < p.min_split || parts > p.max_parts)) cost = 0x7fffffff;
                P.misc[4 + k] = (int)(cost > 0x7fffffff ? 0x7fffffff : cost);
            }
        }
        __syncthreads();
        int best = 0;
        for (int k = 1; k < kCuts; ++k)
            if (P.misc[4 + k] < P.misc[4 + best]) best = k;
        len = max(1, (longest + cut_of(best) - 1) / cut_of(best));
    }
    if (tid < 32) {
        const int all_tiles = (p.m + p.tpt - 1) / p.tpt;
        int ubase = 0, sbase = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            int nu = 0, nslot = 0, ns = 1;
            if (b < p.B) {
                const int tiles = (P.q[b] + p.tpt - 1) / p.tpt;
                const int est = p.cut ? estimate_blocks(p, P, P.q[b], P.s[b]) : 0;
                ns = est > len ? (est + len - 1) / len : 1;
                nu = p.Hkv * (tiles * ns + all_tiles - tiles);
                nslot = ns > 1 ? p.Hkv * tiles * ns : 0;
                P.ns[b] = ns;
            }
            int iu = nu, is = nslot;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(kAllLanes, iu, o), c = __shfl_up_sync(kAllLanes, is, o);
                if (lane >= o) {
                    iu += a;
                    is += c;
                }
            }
            if (b < p.B) {
                P.ubase[b] = ubase + iu - nu;
                P.sbase[b] = sbase + is - nslot;
            }
            ubase += __shfl_sync(kAllLanes, iu, 31);
            sbase += __shfl_sync(kAllLanes, is, 31);
        }
        if (lane == 0) {
            P.ubase[p.B] = ubase;
            P.sbase[p.B] = sbase;
        }
    }
    __syncthreads();
}

// One unit: `live` false means rows that are only zeroed (past q of their sequence).
struct Unit {
    int b, hk, t0, split, ns, slot;  // slot: partial-result slot (ns > 1)
    int q, s;
    bool live;
    int lo_blk, n_glob, e0, e1;      // entries [e0, e1): first the global blocks before lo_blk, then lo_blk ...
};

// Is a position among the global ones?
__device__ __forceinline__ bool is_global(const Plan &P, const PagedProblem &p, int pos) {
    if (p.ng == 0) return false;
    const int i = lower_bound(P.gpos, p.ng, pos);
    return i < p.ng && P.gpos[i] == pos;
}

__device__ __forceinline__ Unit decode_unit(const PagedProblem &p, const Plan &P, int u) {
    Unit U;
    int lo = 0, hi = p.B;  // last b with ubase[b] <= u
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (P.ubase[mid] <= u) lo = mid; else hi = mid;
    }
    U.b = lo;
    U.q = P.q[lo];
    U.s = P.s[lo];
    U.ns = P.ns[lo];
    int r = u - P.ubase[lo];
    const int tiles = (U.q + p.tpt - 1) / p.tpt;
    const int n_live = p.Hkv * tiles * U.ns;
    U.slot = 0;
    U.lo_blk = U.n_glob = U.e0 = U.e1 = 0;
    if (r >= n_live) {
        r -= n_live;
        const int pad = (p.m + p.tpt - 1) / p.tpt - tiles;
        U.live = false;
        U.split = 0;
        U.ns = 1;
        U.hk = r / pad;
        U.t0 = (tiles + r % pad) * p.tpt;
        return U;
    }
    U.live = true;
    U.slot = P.sbase[lo] + r;
    U.split = r % U.ns;
    r /= U.ns;
    U.hk = r / tiles;
    U.t0 = (tiles - 1 - r % tiles) * p.tpt;  // the longest sweeps first
    const int p0 = U.s - U.q + U.t0, p1 = U.s - U.q + min(U.t0 + p.tpt, U.q) - 1;
    int stride = 1;
    if (p.dilation)
        for (int g = 0; g < p.group; ++g) stride = max(stride, head_stride(p, U.hk * p.group + g));
    int first = max(0, p0 - head_reach(p, stride));
    if (p.ng) {  // a global row sees everything before it
        const int i = lower_bound(P.gpos, p.ng, p0);
        if (i < p.ng && P.gpos[i] <= p1) first = 0;
    }
    U.lo_blk = first >> 6;
    U.n_glob = p.ng ? lower_bound(P.gblk, P.ngb, U.lo_blk) : 0;
    const int n = U.n_glob + (p1 >> 6) - U.lo_blk + 1;
    U.e0 = (int)((long long)n * U.split / U.ns);
    U.e1 = (int)((long long)n * (U.split + 1) / U.ns);
    return U;
}

__device__ __forceinline__ int entry_block(const Plan &P, const Unit &U, int e) {
    return e < U.n_glob ? P.gblk[e] : U.lo_blk + e - U.n_glob;
}

// Which keys of a block are global.
__device__ __forceinline__ uint64_t global_bits(const Plan &P, const PagedProblem &p, int blk) {
    if (p.ng == 0) return 0ull;
    const int i = lower_bound(P.gblk, P.ngb, blk);
    return i < P.ngb && P.gblk[i] == blk ? P.gbit[i] : 0ull;
}

// Page number that holds token position `pos`, or -1.
__device__ __forceinline__ int page_of(const PagedProblem &p, int b, int pos) {
    const int c = pos >> p.log_page;
    if (c >= p.max_pages) return -1;
    const int v = __ldg(p.table + (size_t)b * p.max_pages + c);
    if (v >= p.num_pages || v < -1) {
        atomicOr(p.status, kDevBadIndex);
        return -1;
    }
    return v;
}

// What a row needs to mask a block.
struct Row {
    int pos;       // token position
    int stride;
    int reach;     // half * stride
    uint64_t pat;  // bits 0, stride, 2 stride, ...
    bool glob, valid;
};

__device__ __forceinline__ Row make_row(const PagedProblem &p, const Plan &P, const Unit &U, int head, int t) {
    Row r;
    r.valid = U.live && t < U.q;
    r.pos = U.s - U.q + t;
    r.stride = head_stride(p, head);
    r.reach = head_reach(p, r.stride);
    r.pat = ~0ull;
    if (r.stride > 1) {
        r.pat = 0ull;
        for (int i = 0; i < 64; i += r.stride) r.pat |= 1ull << i;
    }
    r.glob = r.valid && is_global(P, p, r.pos);
    return r;
}

// Keys of block `blk` that the row sees: before it, in its window (every
// stride-th key back to `reach`), or global. `gbits`, the block's global keys;
// `present`, the keys whose page is there.
__device__ __forceinline__ uint64_t row_mask(const Row &r, int blk, uint64_t gbits, uint64_t present) {
    const int rel = r.pos - (blk << 6);
    if (!r.valid || rel < 0) return 0ull;
    uint64_t band = ~0ull;
    if (!r.glob) {
        if (r.stride > 1) band = r.pat << (rel % r.stride);
        band &= ~low_bits(rel - r.reach);
    }
    return (band | gbits) & low_bits(rel + 1) & present;
}

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Row `row` of a unit: which token and head it is. Rows go head by head, so
// that one tensor copy fetches a tile's queries.
__device__ __forceinline__ void row_token(const PagedProblem &p, const Unit &U, int row, int tpt, int &t, int &head) {
    const int g = row / tpt;
    t = U.t0 + row - g * tpt;
    head = U.hk * p.group + g;
}

// One row of a unit by the definition, the whole warp together: only the keys
// that the row sees are read, so what masked places hold (unwritten memory,
// infinities, NaN) cannot reach the result. The tiled kernels multiply masked
// values by zero instead and call this for rows whose sums came out infinite
// or NaN, which ordinary inputs never cause. Returns the running maximum and
// sum, and in `acc` the lane's D / 32 sums.
template <typename T, int D>
__device__ __noinline__ float2 exact_row(const PagedProblem &p, const Plan &P, const Unit &U, int t, int head,
                                         float (&acc)[D / 32]) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const T *Q = static_cast<const T *>(p.Q) + (((size_t)U.b * p.Hq + head) * p.m + t) * D + lane * E;
    float q[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = to_float<T>(Q[i]) * p.scale_log2;
        acc[i] = 0.f;
    }
    const Row r = make_row(p, P, U, head, t);
    float m = -CUDART_INF_F, l = 0.f;
    for (int e = U.e0; e < U.e1; ++e) {
        const int blk = entry_block(P, U, e);
        uint64_t w = row_mask(r, blk, global_bits(P, p, blk), ~0ull);
        while (w) {
            const int i = __ffsll((long long)w) - 1;
            w &= w - 1;
            const int j = (blk << 6) + i;
            const int pg = page_of(p, U.b, j);
            if (pg < 0) continue;
            const size_t at = (((size_t)pg * p.Hkv + U.hk) << p.log_page) + (j & (p.page - 1));
            const T *k = static_cast<const T *>(p.K) + at * D + lane * E;
            float s = 0.f;
#pragma unroll
            for (int x = 0; x < E; ++x) s = fmaf(q[x], to_float<T>(k[x]), s);
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kAllLanes, s, o);
            if (s == -CUDART_INF_F) continue;  // weight 0 whatever the maximum
            if (not_finite(s)) {  // +inf or NaN: so is every element of the row
#pragma unroll
                for (int x = 0; x < E; ++x) acc[x] = CUDART_NAN_F;
                return make_float2(0.f, CUDART_NAN_F);
            }
            const float mn = fmaxf(m, s);
            const float f = m == -CUDART_INF_F ? 0.f : ptx::ex2(m - mn), w1 = ptx::ex2(s - mn);
            l = l * f + w1;
            const T *v = static_cast<const T *>(p.V) + at * D + lane * E;
#pragma unroll
            for (int x = 0; x < E; ++x) acc[x] = fmaf(w1, to_float<T>(v[x]), acc[x] * f);
            m = mn;
        }
    }
    return make_float2(m, l);
}

// Stores what exact_row returned: the finished row, or its split's partial.
template <typename T, int D>
__device__ __forceinline__ void store_exact_row(const PagedProblem &p, const Unit &U, int t, int head, int row,
                                                float2 ml, const float (&acc)[D / 32]) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    if (U.ns > 1) {
        const size_t at = (size_t)U.slot * p.rows + row;
#pragma unroll
        for (int i = 0; i < E; ++i) p.part_o[at * D + lane * E + i] = acc[i];
        if (lane == 0) p.part_ml[at] = ml;
    } else {
        T *O = static_cast<T *>(p.O) + (((size_t)U.b * p.Hq + head) * p.m + t) * D + lane * E;
        const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
#pragma unroll
        for (int i = 0; i < E; ++i) O[i] = from_float<T>(acc[i] * inv);
    }
}

}  // namespace
}  // namespace sa
