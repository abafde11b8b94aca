// What the kernels of the paged attention share: the plan (how a call's
// sweeps are cut into units), the walk over a unit's 64-key blocks, the mask
// of a row against a block, and a pass by the definition over rows that ordinary
// arithmetic spoils.
//
// A tile is a few tokens times the query heads of one key head; it walks the
// 64-key blocks that any of its rows may see. All tiles' blocks (and a constant
// for what a tile costs besides) are laid end to end, and CTA c of n takes the
// stretch [T c / n, T (c + 1) / n): every CTA gets the same amount of work
// whatever the lengths of the sequences, and a tile is split only where a
// boundary falls into it, so there are fewer than 2 n partial results. The part
// of a tile that one CTA takes is a unit. Where splitting would add more than
// it evens out, CTAs take whole tiles in turn. The lengths live on the device, so no
// host code can do this: every CTA reads them (at most kPagedMaxBatch) and
// computes the same plan in shared memory, which costs one or two microseconds
// where a planning kernel would cost a launch.
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
    long long *vbase;  // [B + 1] where a sequence's tiles begin on the common axis, then the share
    uint64_t *gbit;    // [ngb] global keys of those blocks
    int *q, *s;        // [B] new tokens and tokens in the cache (q = 0 for a refused sequence)
    int *gpos;         // [ng] global positions
    int *gblk;         // [ngb] 64-key blocks that hold one, ascending
    int *far;          // [B] what global positions add to the length of a sequence's tiles (far_blocks)
    int *hstride;      // [Hkv] longest stride of a key head's query heads (with dilation)
    int *misc;         // [4] [0] ngb, [1] CTAs (0: whole tiles in turn), [2] remainder of the shares
    int ngb;
    int ctas;          // CTAs that share the axis
    long long share;   // its length divided by them: share * ctas + rest
    int rest;
    bool cut;          // whether tiles are split
};

__host__ __device__ constexpr size_t plan_bytes(int B, int ng, int Hkv) {
    return 8 * (size_t)(B + 2 + ng) + (((2 * (size_t)B + 2 * (size_t)ng + (ng > 0 ? B : 0) + Hkv + 4) * 4 + 15) & ~(size_t)15);
}

__device__ __forceinline__ Plan plan_at(void *smem, int B, int ng, int Hkv) {
    Plan P;
    P.vbase = reinterpret_cast<long long *>(smem);
    P.gbit = reinterpret_cast<uint64_t *>(P.vbase + B + 2);
    P.q = reinterpret_cast<int *>(P.gbit + ng);
    P.s = P.q + B;
    P.gpos = P.s + B;
    P.gblk = P.gpos + ng;
    P.far = P.gblk + ng;
    P.hstride = P.far + (ng > 0 ? B : 0);
    P.misc = P.hstride + Hkv;
    P.ngb = 0;
    P.ctas = 1;
    P.share = 0;
    P.rest = 0;
    P.cut = false;
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

// a / b for numbers that mostly fit 32 bits.
__device__ __forceinline__ long long divide(long long a, long long b) {
    if (((unsigned long long)a | (unsigned long long)b) >> 32) return a / b;
    return (long long)((uint32_t)a / (uint32_t)b);
}

// Length on the common axis of one tile of a sequence for a key head of that
// stride: an estimate of the blocks it walks, and its fixed cost. `far`: what
// global positions add to the window (far_blocks).
// It decides how evenly the work is spread, nothing else.
__device__ __forceinline__ int tile_length(const PagedProblem &p, int q, int s, int stride, int far) {
    const int all = (s + 63) >> 6;
    const long long span = (long long)head_reach(p, stride) + min(q, p.tpt);
    const long long band = (span >> 6) + 2 + far;
    return (band < all ? (int)band : all) + p.cost;
}

// Blocks that a sequence's tiles walk because of global positions: those before the
// last tile's window that hold one (or, listed, the global keys there, 64 to an
// entry); any number, if a new token is global and sees its whole sequence. (Then its
// tile is the only long one, but the axis has one length per sequence and head.)
__device__ inline int far_blocks(const PagedProblem &p, const Plan &P, int q, int s) {
    const int i = lower_bound(P.gpos, p.ng, s - q);
    if (i < p.ng && P.gpos[i] < s) return (int)(kPagedMaxLen >> 6);
    const long long window = (long long)s - head_reach(p, 1) - min(q, p.tpt);  // where it begins
    const int first = window > 0 ? (int)(window >> 6) : 0;
    return p.listed ? (lower_bound(P.gpos, p.ng, first << 6) + 63) >> 6 : lower_bound(P.gblk, P.ngb, first);
}

// New tokens and tokens in the cache of a sequence; none of either if they break
// the contract.
__device__ __forceinline__ void lengths(const PagedProblem &p, int q, int s, int &q_out, int &s_out) {
    const bool bad = q < 0 || q > p.m || s < q || (long long)s > ((long long)p.max_pages << p.log_page);
    if (bad) atomicOr(p.status, kDevBadIndex);
    q_out = bad ? 0 : q;
    s_out = bad ? 0 : s;
}

// What make_plan left in shared memory, where it had anything to plan.
__device__ __forceinline__ void take_plan(const PagedProblem &p, Plan &P) {
    P.ngb = p.ng > 0 ? P.misc[0] : 0;
    if (!p.cut) return;
    P.cut = P.misc[1] > 0;
    P.ctas = P.cut ? P.misc[1] : 1;
    P.rest = P.misc[2];
    P.share = P.vbase[p.B + 1];
}

// Marks (-1) the entries of a[0..n) that are not above every one kept before
// them, so that what the walks search is ascending whatever a list held. One
// warp; out of line, as lists are hardly ever out of order.
__device__ __noinline__ void keep_ascending(int *a, int n) {
    const int lane = threadIdx.x & 31;
    int top = -1;  // the largest entry so far
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int v = i0 + lane < n ? a[i0 + lane] : -1;
        int most = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) most = max(most, __shfl_up_sync(kAllLanes, most, o));
        const int prior = __shfl_up_sync(kAllLanes, most, 1);
        if (i0 + lane < n && v <= (lane == 0 ? top : max(top, prior))) a[i0 + lane] = -1;
        top = max(top, __shfl_sync(kAllLanes, most, 31));
    }
    __syncwarp();
}

// Computed by the whole CTA. Ends with a barrier where there is anything to plan;
// where there is not it returns at once, and what the caller has set up in shared
// memory needs a barrier of its own. All loads are issued before the first is
// used, and warp 0 does what follows on its own: the plan stands before every
// call's first load of a key, so its latency counts.
__device__ inline void make_plan(const PagedProblem &p, Plan &P) {
    const int tid = threadIdx.x, lane = tid & 31, nthr = blockDim.x;
    int q0 = p.m, s0 = 0, g0 = -1, g1 = -1;
    if (!p.cut && p.ng == 0 && !p.dilation) return;  // whole tiles in turn: nothing to plan
    if (p.cut && tid < p.B) {
        if (p.qlens) q0 = __ldg(p.qlens + tid);
        s0 = __ldg(p.lens + tid);
    }
    if (tid < p.ng) {
        g0 = __ldg(p.gidx + tid);
        if (tid > 0) g1 = __ldg(p.gidx + tid - 1);
    }
    for (int b = tid; p.cut && b < p.B; b += nthr) {
        int q = q0, s = s0;
        if (b != tid) {
            q = p.qlens ? __ldg(p.qlens + b) : p.m;
            s = __ldg(p.lens + b);
        }
        lengths(p, q, s, P.q[b], P.s[b]);
    }
    // the global list: entries out of range or order are latched and do not count
    bool unsorted = false;
    for (int i = tid; i < p.ng; i += nthr) {
        const int v = i == tid ? g0 : __ldg(p.gidx + i);
        const int before = i == tid ? g1 : __ldg(p.gidx + i - 1);
        if (v < 0 || v >= kPagedMaxLen || (i > 0 && before >= v)) {
            atomicOr(p.status, kDevBadIndex);
            unsorted = true;
        }
        P.gpos[i] = v >= kPagedMaxLen ? -1 : v;
    }
    if (p.dilation)
        for (int h = tid; h < p.Hkv; h += nthr) {
            int st = 1;
            for (int g = 0; g < p.group; ++g) st = max(st, head_stride(p, h * p.group + g));
            P.hstride[h] = st;
        }
    unsorted = __syncthreads_or(unsorted);
    const int all_tiles = (p.m + p.tpt - 1) / p.tpt;
    // the last warp: the blocks of the global list; one starts where the block number changes
    if (p.ng > 0 && tid >= nthr - 32) {
        if (unsorted) keep_ascending(P.gpos, p.ng);
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
    if (p.cut && p.ng > 0) {  // the lengths below go by the list
        __syncthreads();
        P.ngb = P.misc[0];
    }
    if (p.cut && p.ng > 0) {  // the lengths below go by the list
        __syncthreads();
        P.ngb = P.misc[0];
    }
    if (p.cut && tid < 32) {
        long long base = 0;
        int longest = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {  // each sequence's length on the axis, summed up
            const int b = b0 + lane;
            long long v = 0;
            if (b < p.B) {
                const int q = P.q[b], s = P.s[b], tiles = (q + p.tpt - 1) / p.tpt;
                const int far = p.ng > 0 && tiles > 0 ? far_blocks(p, P, q, s) : 0;
                if (p.ng > 0) P.far[b] = far;
                v = (long long)p.Hkv * (all_tiles - tiles) * p.cost;  // tiles without tokens
                if (!p.dilation) {
                    const int len = tiles > 0 ? tile_length(p, q, s, 1, far) : 0;
                    v += (long long)p.Hkv * tiles * len;
                    longest = max(longest, len);
                } else if (tiles > 0) {
                    for (int h = 0; h < p.Hkv; ++h) {
                        const int len = tile_length(p, q, s, P.hstride[h], far);
                        v += (long long)tiles * len;
                        longest = max(longest, len);
                    }
                }
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long a = __shfl_up_sync(kAllLanes, v, o);
                if (lane >= o) v += a;
            }
            if (b < p.B) P.vbase[b + 1] = base + v;
            base += __shfl_sync(kAllLanes, v, 31);
        }
        longest = __reduce_max_sync(kAllLanes, longest);
        if (lane == 0) {
            P.vbase[0] = 0;
            // as many CTAs as there are tiles, or pieces worth having
            const long long tiles = (long long)p.B * p.Hkv * all_tiles;
            const long long pieces = p.cut ? divide(base, p.min_piece) : 0;
            const long long want = pieces > tiles ? pieces : tiles;
            const int ctas = want < p.slots ? (int)want : p.slots;
            const long long share = divide(base, ctas);
            // what the last CTA would walk beyond an even share with whole tiles
            const long long over = divide(tiles + p.slots - 1, p.slots) * longest - share;
            P.misc[1] = over > p.whole ? ctas : 0;
            P.misc[2] = (int)(base - share * ctas);
            P.vbase[p.B + 1] = share;
        }
    }
    __syncthreads();
    take_plan(p, P);
}

// Where CTA c's stretch begins: floor(length * c / ctas).
__device__ __forceinline__ long long cta_begin(const Plan &P, int c) {
    return P.share * c + (long long)((uint32_t)(c * P.rest) / (uint32_t)P.ctas);
}
// The CTA whose stretch holds x, at or after CTA c.
__device__ __forceinline__ int cta_of(const Plan &P, long long x, int c) {
    const long long guess = divide(x, P.share + 1);  // no stretch is longer
    if (guess > c) c = (int)guess;
    while (c + 1 < P.ctas && cta_begin(P, c + 1) <= x) ++c;
    return c;
}

// A tile on the axis, and how to get to the next one. `live` false: its rows are
// only zeroed (past q of their sequence).
struct Tile {
    int b, hk, t0;
    int q, s;
    int tiles, i, len;  // the sequence's tiles, this one's number (of the padding, once past them), length
    bool live;
    long long begin, end;

    __device__ __forceinline__ void place(const PagedProblem &p) {
        live = hk < p.Hkv;
        end = begin + (live ? len : p.cost);
        // the longest sweeps first
        t0 = (live ? tiles - 1 - i : tiles + i % ((p.m + p.tpt - 1) / p.tpt - tiles)) * p.tpt;
    }
    __device__ __forceinline__ int length(const PagedProblem &p, const Plan &P, int stride) const {
        return tile_length(p, q, s, stride, p.ng > 0 ? P.far[b] : 0);
    }
    __device__ __forceinline__ int head(const PagedProblem &p) const {  // key head
        return live ? hk : i / ((p.m + p.tpt - 1) / p.tpt - tiles);
    }
    __device__ __forceinline__ void start(const PagedProblem &p, const Plan &P, int seq) {
        b = seq;
        q = P.q[b];
        s = P.s[b];
        begin = P.vbase[b];
        tiles = (q + p.tpt - 1) / p.tpt;
        i = 0;
        hk = tiles > 0 ? 0 : p.Hkv;
        if (tiles > 0) len = length(p, P, p.dilation ? P.hstride[0] : 1);
    }
    __device__ __forceinline__ void advance(const PagedProblem &p, const Plan &P) {
        begin = end;
        if (begin == P.vbase[b + 1]) {
            if (b + 1 < p.B) start(p, P, b + 1);
        } else if (++i == tiles && live) {
            i = 0;
            if (++hk < p.Hkv && p.dilation) len = length(p, P, P.hstride[hk]);
        }
        place(p);
    }
};

__device__ __forceinline__ Tile find_tile(const PagedProblem &p, const Plan &P, long long x) {
    Tile T;
    int lo = 0, hi = p.B;  // last b with vbase[b] <= x; every sequence has a length
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (P.vbase[mid] <= x) lo = mid; else hi = mid;
    }
    T.len = 0;
    T.start(p, P, lo);
    long long off = x - T.begin;
    if (T.tiles > 0) {
        if (!p.dilation) {
            const long long per = (long long)T.len * T.tiles;
            T.hk = (int)min(divide(off, per), (long long)p.Hkv);
            T.begin += T.hk * per;
            off -= T.hk * per;
        } else {
            for (; T.hk < p.Hkv; ++T.hk) {
                T.len = T.length(p, P, P.hstride[T.hk]);
                const long long per = (long long)T.len * T.tiles;
                if (off < per) break;
                T.begin += per;
                off -= per;
            }
        }
    }
    const int len = T.hk < p.Hkv ? T.len : p.cost;
    T.i = (int)divide(off, len);
    T.begin += (long long)T.i * len;
    T.place(p);
    return T;
}

// One CTA's part of a tile.
struct Unit {
    int b, hk, t0;
    int q, s;
    bool live, split;
    int slot;                    // partial-result slot (split)
    // entries [e0, e1): first the global blocks before lo_blk (or, listed, the global
    // keys before it, 64 to an entry), then lo_blk ...
    int lo_blk, n_glob, e0, e1;
};

// Is a position among the global ones?
__device__ __forceinline__ bool is_global(const Plan &P, const PagedProblem &p, int pos) {
    if (p.ng == 0) return false;
    const int i = lower_bound(P.gpos, p.ng, pos);
    return i < p.ng && P.gpos[i] == pos;
}

// Global positions before a unit's first block.
__device__ __forceinline__ int far_globals(const PagedProblem &p, const Plan &P, const Unit &U) {
    return p.ng ? lower_bound(P.gpos, p.ng, U.lo_blk << 6) : 0;
}

// The units of a CTA, in order: next() fills the following one and returns
// whether there is one.
struct Units {
    Tile T;
    long long v, end;
    int c;
    __device__ __forceinline__ void begin(const PagedProblem &p, const Plan &P, int cta) {
        c = cta;
        v = end = 0;
        if (!P.cut) {
            v = cta;
            end = (long long)p.B * p.Hkv * ((p.m + p.tpt - 1) / p.tpt);
        } else if (cta < P.ctas) {
            v = cta_begin(P, cta);
            end = cta_begin(P, cta + 1);
            T = find_tile(p, P, v);
        }
    }
    __device__ __forceinline__ bool next(const PagedProblem &p, const Plan &P, Unit &U) {
        U.b = U.hk = U.t0 = U.q = U.s = U.slot = U.lo_blk = U.n_glob = U.e0 = U.e1 = 0;
        U.live = U.split = false;
        if (v >= end) return false;
        long long from = 0, stop = 0;
        if (!P.cut) {
            const int all_tiles = (p.m + p.tpt - 1) / p.tpt;
            const int u = (int)v, i = u % all_tiles, bh = u / all_tiles;
            T.b = bh / p.Hkv;
            T.hk = bh - T.b * p.Hkv;
            lengths(p, p.qlens ? __ldg(p.qlens + T.b) : p.m, __ldg(p.lens + T.b), T.q, T.s);
            T.tiles = (T.q + p.tpt - 1) / p.tpt;
            T.live = i < T.tiles;
            T.t0 = i * p.tpt;
            v += gridDim.x;
            U.hk = T.hk;
            U.split = false;
            U.slot = 0;
        } else {
            if (v == T.end) T.advance(p, P);
            from = v;
            stop = T.end > end ? end : T.end;
            U.hk = T.head(p);
            U.split = T.live && (from > T.begin || stop < T.end);
            U.slot = 2 * c + (from == T.begin);
            v = stop;
        }
        U.b = T.b;
        U.t0 = T.t0;
        U.q = T.q;
        U.s = T.s;
        U.live = T.live;
        U.lo_blk = U.n_glob = U.e0 = U.e1 = 0;
        if (!T.live) return true;
        const int p0 = U.s - U.q + U.t0, p1 = U.s - U.q + min(U.t0 + p.tpt, U.q) - 1;
        int first = max(0, p0 - head_reach(p, p.dilation ? P.hstride[U.hk] : 1));
        if (p.ng) {  // a global row sees everything before it
            const int i = lower_bound(P.gpos, p.ng, p0);
            if (i < p.ng && P.gpos[i] <= p1) first = 0;
        }
        U.lo_blk = first >> 6;
        U.n_glob = !p.ng ? 0 : p.listed ? (far_globals(p, P, U) + 63) >> 6 : lower_bound(P.gblk, P.ngb, U.lo_blk);
        const int n = U.n_glob + (p1 >> 6) - U.lo_blk + 1;
        U.e1 = n;
        if (U.split) {
            const long long len = T.end - T.begin;
            U.e0 = (int)divide(n * (from - T.begin), len);
            U.e1 = (int)divide(n * (stop - T.begin), len);
        }
        return true;
    }
};

// The units of a CTA that works on one at a time: thread 0 finds the next one
// while the others work and leaves it in shared memory, where it costs no
// registers. Two rooms: the one being filled is not the one being read.
struct alignas(16) UnitRoom {
    Units units;
    Unit U[2];
    int more[2];
};

__device__ __forceinline__ void fill_room(const PagedProblem &p, const Plan &P, UnitRoom *room, int k) {
    Units u = room->units;  // in registers: what follows would be a chain of shared-memory accesses
    Unit next;
    const bool more = u.next(p, P, next);
    room->units = u;
    room->U[k] = next;
    room->more[k] = more;
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

// Element x of a 16-byte piece, as fp32 (exact). x is a constant wherever this is
// used. By bits, not through a pointer of another type.
template <typename T>
__device__ __forceinline__ float element(const uint4 &v, int x) {
    constexpr bool half = sizeof(T) == 2;
    const int i = half ? x >> 1 : x;
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    if (!half) return __uint_as_float(w);
    return __uint_as_float(x & 1 ? w & 0xffff0000u : w << 16);
}

// Two values rounded to bf16 (to nearest, ties to even), a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Sixteen consecutive elements, rounded and written (16-byte aligned).
template <typename T>
__device__ __forceinline__ void store16(T *at, const float (&v)[16]) {
    uint4 *out = reinterpret_cast<uint4 *>(at);
    if (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            out[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                __float_as_uint(v[4 * i + 3]));
    }
}

// Row `row` of a unit: which token and head it is. Rows go head by head, so
// that one tensor copy fetches a tile's queries.
__device__ __forceinline__ void row_token(const PagedProblem &p, const Unit &U, int row, int tpt, int &t, int &head) {
    const int g = tpt == 1 ? row : row / tpt;
    t = U.t0 + row - g * tpt;
    head = U.hk * p.group + g;
}

// Where elements [4 k, 4 k + 4) of a row's partial sums lie: rows side by side, so
// that threads that hold a row each write whole lines.
template <int D>
__device__ __forceinline__ size_t part_at(const PagedProblem &p, int slot, int k, int row) {
    return (((size_t)slot * (D / 4) + k) * p.rows + row) * 4;
}

// Rows [at0, at0 + R) of a unit by the definition, those of them whose results hold an
// infinity or NaN, the whole warp together: a key counts for the rows that see it and
// for no others. 32 keys at a time, a lane each for the scores, then eight values in
// flight; the rows share what is loaded. (33000 rows that all see an infinity among
// 16000 keys, d = 64: 66 ms; key by key with the whole warp, a row at a time, 770.)
template <typename T, int D, int R>
__device__ __forceinline__ void exact_rows(const PagedProblem &p, const Plan &P, const Unit &U, int at0) {
    constexpr int E = D / 32, VE = 16 / sizeof(T), AHEAD = 8;
    struct alignas(E * sizeof(T)) Piece {
        T x[E];
    };
    const int lane = threadIdx.x & 31, half_rows = p.tpt_half * p.group;
    size_t base[R];  // where the row is in Q and O
    Row row[R];
    float acc[R][E], m[R], l[R];
    unsigned again = 0u, spoiled = 0u;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int at = min(at0 + r, p.rows - 1), x = at / half_rows;  // the halves of a unit hold different tokens
        const int k = at - x * half_rows, g = k / p.tpt_half, head = U.hk * p.group + g;
        const int t = U.t0 + x * p.tpt_half + k - g * p.tpt_half;
        base[r] = (((size_t)U.b * p.Hq + head) * p.m + t) * D;
        row[r] = make_row(p, P, U, head, t);
        row[r].valid = row[r].valid && at0 + r < p.rows;
        bool bad = false;
        if (row[r].valid && U.split) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                bad |= not_finite(p.part_o[part_at<D>(p, U.slot, (lane * E + i) >> 2, at) + ((lane * E + i) & 3)]);
            bad |= not_finite(p.part_ml[(size_t)U.slot * p.rows + at].y);
        } else if (row[r].valid) {
            const Piece o = *reinterpret_cast<const Piece *>(static_cast<const T *>(p.O) + base[r] + lane * E);
#pragma unroll
            for (int i = 0; i < E; ++i) bad |= not_finite(to_float<T>(o.x[i]));
        }
        if (__any_sync(kAllLanes, bad)) again |= 1u << r;
        m[r] = -CUDART_INF_F;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[r][i] = 0.f;
    }
    if (!again) return;
    const int far = p.listed ? far_globals(p, P, U) : 0;
    for (int e = U.e0; e < U.e1; ++e) {
        const bool listed = p.listed && e < U.n_glob;
        const int blk = listed ? 0 : entry_block(P, U, e);
        const uint64_t gbits = listed ? 0ull : global_bits(P, p, blk);
        uint64_t w[R], any = 0ull;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w[r] = 0ull;
            if (((again & ~spoiled) >> r) & 1u) w[r] = listed ? low_bits(far - 64 * e) : row_mask(row[r], blk, gbits, ~0ull);
            any |= w[r];
        }
#pragma unroll 1
        for (int i0 = 0; i0 < 64; i0 += 32) {
            const uint32_t seen = (uint32_t)(any >> i0);
            if (!seen) continue;
            float s[R];  // of the lane's key
            size_t at = 0;
            bool there = false;
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = 0.f;
            if ((seen >> lane) & 1u) {
                const int j = listed ? P.gpos[64 * e + i0 + lane] : (blk << 6) + i0 + lane;
                const int pg = page_of(p, U.b, j);
                there = pg >= 0;
                if (there) {
                    at = ((((size_t)pg * p.Hkv + U.hk) << p.log_page) + (j & (p.page - 1))) * D;
                    const uint4 *k = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.K) + at);
#pragma unroll 4
                    for (int c = 0; c < D / VE; ++c) {
                        const uint4 kw = __ldg(k + c);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            if (!((again >> r) & 1u)) continue;
                            const uint4 qw = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.Q) + base[r]) + c);
#pragma unroll
                            for (int x = 0; x < VE; ++x)
                                s[r] = fmaf(element<T>(qw, x) * p.scale_log2, element<T>(kw, x), s[r]);
                        }
                    }
                }
            }
            unsigned on[R], all_on = 0u;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (!there || !((uint32_t)(w[r] >> (i0 + lane)) & 1u)) s[r] = -CUDART_INF_F;
                on[r] = __ballot_sync(kAllLanes, s[r] != -CUDART_INF_F);  // a score of -inf has weight 0 whatever the maximum
                all_on |= on[r];
                // +inf or NaN: so is every element of the row
                if (__any_sync(kAllLanes, !(s[r] <= 3.402823466e38f))) spoiled |= 1u << r;
                if (!on[r]) continue;
                float mn = s[r];
#pragma unroll
                for (int o = 16; o; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(kAllLanes, mn, o));
                mn = fmaxf(m[r], mn);
                const float f = ptx::ex2(m[r] - mn);  // 0 from the initial -inf
                s[r] = ptx::ex2(s[r] - mn);
                float sum = s[r];
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAllLanes, sum, o);
                l[r] = l[r] * f + sum;
                m[r] = mn;
#pragma unroll
                for (int i = 0; i < E; ++i) acc[r][i] *= f;
            }
#pragma unroll 1
            for (int k0 = 0; k0 < 32; k0 += AHEAD) {
                Piece v[AHEAD];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const size_t from = __shfl_sync(kAllLanes, (unsigned long long)at, k0 + k);
                    if ((all_on >> (k0 + k)) & 1u)
                        v[k] = *reinterpret_cast<const Piece *>(static_cast<const T *>(p.V) + from + lane * E);
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k) {
                        const float wk = __shfl_sync(kAllLanes, s[r], k0 + k);
                        if ((on[r] >> (k0 + k)) & 1u) {
#pragma unroll
                            for (int i = 0; i < E; ++i) acc[r][i] = fmaf(wk, to_float<T>(v[k].x[i]), acc[r][i]);
                        }
                    }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (!((again >> r) & 1u)) continue;
        if ((spoiled >> r) & 1u) {
            m[r] = 0.f;
            l[r] = CUDART_NAN_F;
#pragma unroll
            for (int i = 0; i < E; ++i) acc[r][i] = CUDART_NAN_F;
        }
        if (U.split) {  // the split's partial result
#pragma unroll
            for (int i = 0; i < E; ++i)
                p.part_o[part_at<D>(p, U.slot, (lane * E + i) >> 2, at0 + r) + ((lane * E + i) & 3)] = acc[r][i];
            if (lane == 0) p.part_ml[(size_t)U.slot * p.rows + at0 + r] = make_float2(m[r], l[r]);
        } else {
            const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
            T *O = static_cast<T *>(p.O) + base[r] + lane * E;
#pragma unroll
            for (int i = 0; i < E; ++i) O[i] = from_float<T>(acc[r][i] * inv);
        }
    }
}

// The tiled kernels multiply masked values by zero, so an infinity or NaN at a key
// that a row does not see spoils the row's sums; ordinary inputs never do that.
// A CTA that met such a row goes over its units once more when it is through
// with them, and takes the rows whose results are not finite again by the
// definition. (Not between its units: no other warp may wait for rows that
// take as long as their keys are many.) Called by `warps` whole warps after a
// barrier; the results are read back from where they were written. (Nothing of the
// caller's but where its plan lies, which would otherwise have to be in memory.)
template <typename T, int D, int R>
__device__ __noinline__ void rows_again(const PagedProblem &p, void *plan, int warp, int warps) {
    Plan P = plan_at(plan, p.B, p.ng, p.Hkv);
    take_plan(p, P);
    Units units;
    units.begin(p, P, blockIdx.x);
    Unit U;
    while (units.next(p, P, U))
        if (U.live)
            for (int at = R * warp; at < p.rows; at += R * warps) exact_rows<T, D, R>(p, P, U, at);
}

}  // namespace
}  // namespace sa
