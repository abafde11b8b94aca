// Writing and moving the pages of a key/value cache. All of it is bounded by
// the memory: the data kernels move 16 bytes per thread and load several
// vectors before storing any; the bookkeeping (tables of pages, reference
// counts) is done in one or two small launches and every choice it makes
// (which free page comes next, where a page moves) depends on the inputs alone,
// so equal inputs give equal tables.
//
// Measured: 4096 new tokens in each of 4 sequences, 8 heads of 128, bf16: 18.4 us, 5.5
// TB/s; a single token in each of 64 sequences 3.9 us (launch); 12 layers' last pages
// of 32 forked rows (151 MB moved) 27 us, of which the plan takes 5; a pool of 4096 pages
// in 4 layers compacted (490 MB moved) 84 us, 5.8 TB/s.
//
// The bookkeeping calls read `*_in` and write `*_out`, which may be the same
// arrays: a kernel reads what it needs of an array before any thread writes
// what another still has to read.
#include "internal.h"
#include "paged.h"

namespace sa {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kBookThreads = 1024;

// ------------------------------------------------------------------ append
// New token t of sequence b goes to position lens[b] - q[b] + t. blockIdx.y is
// one (sequence, key head); a thread moves up to kAppendVecs 16-byte pieces of
// K rows and the same pieces of V rows, all requested before the first is
// stored. Consecutive threads take consecutive pieces, and the rows of a page
// follow one another on both sides, so reads and writes are whole lines.
constexpr int kAppendThreads = 256, kAppendVecs = 4;

__global__ void __launch_bounds__(kAppendThreads) cache_append(const AppendProblem p, int log_ppr) {
    for (long long bh = blockIdx.y; bh < (long long)p.B * p.Hkv; bh += gridDim.y) {
        const int h = (int)(bh % p.Hkv), b = (int)(bh / p.Hkv);
        const int q = p.qlens ? __ldg(p.qlens + b) : p.m, s = __ldg(p.lens + b);
        if (q < 0 || q > p.m || s < q || (long long)s > ((long long)p.max_pages << p.log_page)) {
            if (threadIdx.x == 0) atomicOr(p.status, kDevBadIndex);
            continue;
        }
        const long long pieces = (long long)q << log_ppr;
        const int32_t *row = p.table + (size_t)b * p.max_pages;
        for (long long i0 = (long long)blockIdx.x * (kAppendThreads * kAppendVecs) + threadIdx.x; i0 < pieces;
             i0 += (long long)gridDim.x * (kAppendThreads * kAppendVecs)) {
            uint4 k[kAppendVecs], v[kAppendVecs];
            int pg[kAppendVecs];
#pragma unroll
            for (int x = 0; x < kAppendVecs; ++x) {
                const long long i = i0 + x * kAppendThreads;
                pg[x] = -1;
                if (i < pieces) {
                    const size_t src = ((size_t)bh * p.m << log_ppr) + (size_t)i;
                    k[x] = __ldcs(static_cast<const uint4 *>(p.Kn) + src);
                    v[x] = __ldcs(static_cast<const uint4 *>(p.Vn) + src);
                    pg[x] = __ldg(row + ((s - q + (int)(i >> log_ppr)) >> p.log_page));
                    if (pg[x] < 0 || pg[x] >= p.num_pages) {  // nowhere to write the token
                        atomicOr(p.status, kDevBadIndex);
                        pg[x] = -1;
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < kAppendVecs; ++x) {
                const long long i = i0 + x * kAppendThreads;
                if (pg[x] < 0) continue;
                const int pos = s - q + (int)(i >> log_ppr);
                const size_t dst = ((((((size_t)pg[x] * p.Hkv + h) << p.log_page) + (pos & (p.page - 1)))) << log_ppr) +
                                   (size_t)(i & ((1 << log_ppr) - 1));
                static_cast<uint4 *>(p.K)[dst] = k[x];
                static_cast<uint4 *>(p.V)[dst] = v[x];
            }
        }
    }
}

// ------------------------------------------------------------------ moving pages
// Pages src[i] -> dst[i], i < *n, of every layer of both pools. A CTA takes
// chunks of one page of one layer; the page numbers are the same for its whole
// chunk.
constexpr int kMoveThreads = 256, kMoveVecs = 8;
constexpr int kMoveChunk = kMoveThreads * kMoveVecs * 16;  // 32 KB

__device__ __forceinline__ void move_pages(const PoolProblem &p, const int32_t *src, const int32_t *dst, int n,
                                           int first_cta, int ctas) {
    const long long chunks = (long long)((p.page_bytes + kMoveChunk - 1) / kMoveChunk);
    const long long total = 2ll * p.layers * n * chunks;
    for (long long w = first_cta; w < total; w += ctas) {
        const int c = (int)(w % chunks);
        long long r = w / chunks;
        const int i = (int)(r % n);
        r /= n;
        const int layer = (int)(r >> 1);
        const int a = __ldg(src + i), b = __ldg(dst + i);
        if (a < 0 || a >= p.num_pages || b < 0 || b >= p.num_pages) {
            if (threadIdx.x == 0 && c == 0) atomicOr(p.status, kDevBadIndex);
            continue;
        }
        uint8_t *pool = (r & 1) ? p.V : p.K;
        const size_t base = (size_t)layer * p.num_pages;
        const uint8_t *from = pool + (base + a) * p.page_bytes;
        uint8_t *to = pool + (base + b) * p.page_bytes;
        const size_t at = (size_t)c * kMoveChunk + (size_t)threadIdx.x * 16;
        uint4 v[kMoveVecs];
#pragma unroll
        for (int k = 0; k < kMoveVecs; ++k) {
            const size_t o = at + (size_t)k * kMoveThreads * 16;
            if (o < p.page_bytes) v[k] = __ldcs(reinterpret_cast<const uint4 *>(from + o));
        }
#pragma unroll
        for (int k = 0; k < kMoveVecs; ++k) {
            const size_t o = at + (size_t)k * kMoveThreads * 16;
            if (o < p.page_bytes) __stcs(reinterpret_cast<uint4 *>(to + o), v[k]);
        }
    }
}

__global__ void __launch_bounds__(kMoveThreads) cache_move(const PoolProblem p) {
    move_pages(p, p.src, p.dst, p.n, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------------ bookkeeping helpers
// Exclusive prefix sum over the 32 warps of a CTA of kBookThreads; returns the
// sum before this warp and leaves the total in `total`. `sh`: 33 ints.
__device__ __forceinline__ int warp_prefix(int mine, int *sh, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) sh[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        int v = sh[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += a;
        }
        sh[lane + 1] = v;  // the lanes have read sh before any of them writes
        if (lane == 0) sh[0] = 0;
    }
    __syncthreads();
    total = sh[32];
    return sh[warp];
}

// Each warp owns a contiguous stretch of the pages, a multiple of 32 long.
__device__ __forceinline__ void warp_stretch(int n, int &lo, int &hi) {
    const int per = (((n + 31) / 32) + 31) & ~31;
    const long long a = (long long)(threadIdx.x >> 5) * per;
    lo = a < n ? (int)a : n;
    hi = a + per < n ? (int)(a + per) : n;
}

// Calls f(i, counts[i]) for i in [lo, hi), the whole warp together, 32 at a
// time in order; past the end f gets `none`. Eight loads are in flight at once.
template <typename F>
__device__ __forceinline__ void for_counts(const int32_t *counts, int lo, int hi, int none, F f) {
    const int lane = threadIdx.x & 31;
    for (int i0 = lo; i0 < hi; i0 += 256) {
        int v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + 32 * k + lane;
            v[k] = i < hi ? counts[i] : none;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) f(i0 + 32 * k + lane, v[k]);
    }
}

// Lowest `want` free pages (count 0), in order, to list[]; returns how many
// there are in all. Copies refs_in to refs_out on the way.
__device__ inline int list_free_pages(const PoolProblem &p, int32_t *list, int want, int *sh) {
    const int lane = threadIdx.x & 31;
    int lo, hi, total;
    warp_stretch(p.num_pages, lo, hi);
    int n = 0;
    for_counts(p.refs_in, lo, hi, 1, [&](int i, int v) {
        if (i < hi && p.refs_out != p.refs_in) p.refs_out[i] = v;
        n += __popc(__ballot_sync(kAll, v == 0));
    });
    int at = warp_prefix(n, sh, total);
    if (at < want)
        for_counts(p.refs_in, lo, hi, 1, [&](int i, int v) {
            const unsigned free = __ballot_sync(kAll, v == 0);
            const int k = at + __popc(free & ((1u << lane) - 1u));
            if (v == 0 && k < want) list[k] = i;
            at += __popc(free);
        });
    __syncthreads();
    return total;
}

// Scratch of fork and reserve: what each row gets.
__host__ __device__ inline int up32(int x) { return (x + 31) & ~31; }

// The page that a table entry names, or -1; entries outside [-1, num_pages) count
// as -1 and are latched.
__device__ __forceinline__ int page_in(const PoolProblem &p, int v) {
    if (v < -1 || v >= p.num_pages) {
        atomicOr(p.status, kDevBadIndex);
        return -1;
    }
    return v;
}

// One holder of page v lets go of it.
__device__ __forceinline__ void drop_page(const PoolProblem &p, int v) {
    if (atomicSub(p.refs_out + v, 1) <= 0) {  // the table names a page that nobody holds
        atomicAdd(p.refs_out + v, 1);
        atomicOr(p.status, kDevBadIndex);
    }
}

// ------------------------------------------------------------------ fork
// ws: row_src[B] (source row, or -1: not forked), row_new[B] (own last page, or
// -1), then move_src[B], move_dst[B] and the number of moves.
__global__ void __launch_bounds__(kBookThreads, 1) fork_plan(const PoolProblem p) {
    __shared__ int sh[33];
    __shared__ int s_bad;
    extern __shared__ int dyn[];  // first[B]: the first fork that names the row as destination
    int32_t *row_src = p.ws, *row_new = row_src + up32(p.B), *mv_src = row_new + up32(p.B),
            *mv_dst = mv_src + up32(p.B), *n_mv = mv_dst + up32(p.B), *list = n_mv + 32;
    int *first = dyn;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) s_bad = 0;
    for (int b = tid; b < p.B; b += kBookThreads) {
        first[b] = 0x7fffffff;
        row_src[b] = row_new[b] = -1;
        const int len = p.lens_in[b];
        if (p.lens_out != p.lens_in) p.lens_out[b] = len;
    }
    __syncthreads();
    for (int i = tid; i < p.n; i += kBookThreads) {
        const int d = p.dst[i];
        if (d >= 0 && d < p.B) atomicMin(first + d, i);
    }
    __syncthreads();
    // a fork holds if its rows are in range, its destination is empty and named
    // by no earlier fork, and its source is no fork's destination
    int need = 0;  // forks of this warp's stretch that need a page of their own
    int lo, hi, total;
    warp_stretch(p.n, lo, hi);
    auto fork_of = [&](int i, int &s, int &d, int &len) -> bool {
        s = p.src[i];
        d = p.dst[i];
        if (s < 0 || s >= p.B || d < 0 || d >= p.B || first[d] != i || first[s] != 0x7fffffff) return false;
        len = p.lens_in[s];
        return len >= 0 && (long long)len <= ((long long)p.max_pages << p.log_page) && p.lens_in[d] == 0;
    };
    auto needs_page = [&](int s, int len) -> bool {
        if (!(len & (p.page - 1))) return false;
        const int v = p.table_in[(size_t)s * p.max_pages + (len >> p.log_page)];
        return v >= 0 && v < p.num_pages;
    };
    for (int i = lo + lane; i - lane < hi; i += 32) {
        int s, d, len;
        const bool ok = i < hi && fork_of(i, s, d, len);
        if (i < hi && !ok) s_bad = 1;
        need += __popc(__ballot_sync(kAll, ok && needs_page(s, len)));
    }
    int at = warp_prefix(need, sh, total);
    const int have = list_free_pages(p, list, total, sh);
    if (total > have && tid == 0) atomicOr(p.status, kDevNoPages);
    if (s_bad && tid == 0) atomicOr(p.status, kDevBadIndex);
    for (int i = lo + lane; i - lane < hi; i += 32) {
        int s, d, len;
        const bool ok = i < hi && fork_of(i, s, d, len);
        const bool own = ok && needs_page(s, len);
        const unsigned m = __ballot_sync(kAll, own);
        const int k = at + __popc(m & ((1u << lane) - 1u));
        at += __popc(m);
        if (!ok || (own && k >= have)) continue;  // no page left: the destination stays empty
        row_src[d] = s;
        if (own) {
            const int pg = list[k];
            row_new[d] = pg;
            mv_src[k] = p.table_in[(size_t)s * p.max_pages + (len >> p.log_page)];
            mv_dst[k] = pg;
            p.refs_out[pg] = 1;
        }
    }
    if (tid == 0) *n_mv = total < have ? total : have;
    __syncthreads();
    // lengths last: sources and destinations are told apart by lens_in above,
    // which may be the same array
    for (int b = tid; b < p.B; b += kBookThreads)
        if (row_src[b] >= 0) p.lens_out[b] = p.lens_in[row_src[b]];
}

// Tables and reference counts of the forked rows, and their last pages' data.
__global__ void __launch_bounds__(kMoveThreads) fork_apply(const PoolProblem p) {
    const int32_t *row_src = p.ws, *row_new = row_src + up32(p.B), *mv_src = row_new + up32(p.B),
                  *mv_dst = mv_src + up32(p.B), *n_mv = mv_dst + up32(p.B);
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const int s = row_src[b];
        if (s < 0) {
            if (p.table_out != p.table_in)
                for (int c = threadIdx.x; c < p.max_pages; c += blockDim.x)
                    p.table_out[(size_t)b * p.max_pages + c] = p.table_in[(size_t)b * p.max_pages + c];
            continue;
        }
        const int len = p.lens_out[b], full = len >> p.log_page;
        for (int c = threadIdx.x; c < p.max_pages; c += blockDim.x) {
            // pages that the empty row had in reserve go back
            const int old = page_in(p, p.table_in[(size_t)b * p.max_pages + c]);
            if (old >= 0) drop_page(p, old);
            int v = -1;
            if (c < full || (c == full && (len & (p.page - 1)))) {
                v = page_in(p, p.table_in[(size_t)s * p.max_pages + c]);
                if (c == full) v = row_new[b];
                else if (v >= 0) atomicAdd(p.refs_out + v, 1);
            }
            p.table_out[(size_t)b * p.max_pages + c] = v;
        }
    }
    move_pages(p, mv_src, mv_dst, *n_mv, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------------ free, trim
// Rows named in src[0..n) give up their pages. A row named twice gives them up
// once.
__global__ void __launch_bounds__(256) free_rows(const PoolProblem p) {
    __shared__ int s_gone;
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        __syncthreads();
        if (threadIdx.x == 0) s_gone = 0;
        __syncthreads();
        bool mine = false;
        for (int i = threadIdx.x; i < p.n; i += blockDim.x) {
            const int r = p.src[i];
            mine |= r == b;
            if (b == 0 && (r < 0 || r >= p.B)) atomicOr(p.status, kDevBadIndex);
        }
        if (mine) s_gone = 1;
        __syncthreads();
        const bool gone = s_gone != 0;
        for (int c = threadIdx.x; c < p.max_pages; c += blockDim.x) {
            const size_t at = (size_t)b * p.max_pages + c;
            const int v = p.table_in[at];
            if (gone) {
                if (page_in(p, v) >= 0) drop_page(p, v);
                p.table_out[at] = -1;
            } else if (p.table_out != p.table_in) {
                p.table_out[at] = v;
            }
        }
        if (threadIdx.x == 0) p.lens_out[b] = gone ? 0 : p.lens_in[b];
    }
}

// Pages that no later token can see: all their tokens lie more than `reach`
// before the next one, and none of them is global. A global position still to
// come will see everything, so its sequence keeps every page. So does a sequence
// whose length breaks the contract, and every one if the list does: pages given
// up do not come back.
__global__ void __launch_bounds__(256) trim_rows(const PoolProblem p) {
    bool unsorted = false;
    for (int i = threadIdx.x; i < p.ng; i += blockDim.x)
        unsorted |= __ldg(p.gidx + i) <= (i == 0 ? -1 : __ldg(p.gidx + i - 1));
    unsorted = __syncthreads_or(unsorted);
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const int len = p.lens_in[b];
        const bool bad = unsorted || len < 0 || (long long)len > ((long long)p.max_pages << p.log_page);
        if (bad && threadIdx.x == 0) atomicOr(p.status, kDevBadIndex);
        const bool keep_all = bad || (p.ng > 0 && __ldg(p.gidx + p.ng - 1) >= len);
        const long long lowest = (long long)len - p.reach;  // first position the next token's window holds
        for (int c = threadIdx.x; c < p.max_pages; c += blockDim.x) {
            const size_t at = (size_t)b * p.max_pages + c;
            int v = p.table_in[at];
            const long long end = ((long long)c + 1) << p.log_page;
            if (page_in(p, v) >= 0 && !keep_all && end <= lowest) {
                int lo = 0, hi = p.ng;  // first global position in or after the page
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (__ldg(p.gidx + mid) < end - p.page) lo = mid + 1; else hi = mid;
                }
                if (lo >= p.ng || __ldg(p.gidx + lo) >= end) {
                    drop_page(p, v);
                    v = -1;
                }
            }
            if (v != p.table_in[at] || p.table_out != p.table_in) p.table_out[at] = v;
        }
    }
}

// ------------------------------------------------------------------ reserve
// Pages for tokens [lens - q, lens) of every row: slots from the first one past
// the old tokens' last page to the new last page, where the table has none yet.
// ws: base[B] (a row's first page in the list), have, then the list.
__device__ __forceinline__ bool reserve_range(const PoolProblem &p, int b, int &c0, int &c1) {
    const int s = p.lens_in[b], q = p.qlens[b];
    c0 = c1 = 0;
    if (q < 0 || s < q || (long long)s > ((long long)p.max_pages << p.log_page)) return false;
    c0 = (s - q + p.page - 1) >> p.log_page;
    c1 = (s + p.page - 1) >> p.log_page;
    return true;
}

__global__ void __launch_bounds__(kBookThreads, 1) reserve_plan(const PoolProblem p) {
    __shared__ int sh[33];
    int32_t *base = p.ws, *have = base + up32(p.B), *list = have + 32;
    const int lane = threadIdx.x & 31;
    int total = 0;
    for (int b = threadIdx.x >> 5; b < p.B; b += 32) {  // a warp per row
        int c0, c1, n = 0;
        if (!reserve_range(p, b, c0, c1) && lane == 0) atomicOr(p.status, kDevBadIndex);
        for (int c = c0 + lane; c - lane < c1; c += 32)
            n += __popc(__ballot_sync(kAll, c < c1 && page_in(p, p.table_in[(size_t)b * p.max_pages + c]) < 0));
        if (lane == 0) base[b] = n;
    }
    __syncthreads();
    for (int b0 = 0; b0 < p.B; b0 += kBookThreads) {  // counts to first places, in row order
        const int b = b0 + threadIdx.x, n = b < p.B ? base[b] : 0;
        int v = n, sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += a;
        }
        const int before = warp_prefix(__shfl_sync(kAll, v, 31), sh, sum);
        if (b < p.B) base[b] = total + before + v - n;
        total += sum;
    }
    const int free = list_free_pages(p, list, total < p.num_pages ? total : p.num_pages, sh);
    if (threadIdx.x == 0) {
        *have = total < free ? total : free;
        if (total > free) atomicOr(p.status, kDevNoPages);
    }
}

__global__ void __launch_bounds__(256) reserve_apply(const PoolProblem p) {
    const int32_t *base = p.ws, *have = base + up32(p.B), *list = have + 32;
    const int lane = threadIdx.x & 31;
    const int n_have = *have;
    for (int b = blockIdx.x * 8 + (threadIdx.x >> 5); b < p.B; b += gridDim.x * 8) {
        int c0, c1, at = base[b];
        reserve_range(p, b, c0, c1);
        for (int c = lane; c - lane < p.max_pages; c += 32) {
            const size_t i = (size_t)b * p.max_pages + c;
            int v = c < p.max_pages ? p.table_in[i] : 0;
            const bool want = c < p.max_pages && c >= c0 && c < c1 && (v < 0 || v >= p.num_pages);
            const unsigned m = __ballot_sync(kAll, want);
            const int k = at + __popc(m & ((1u << lane) - 1u));
            at += __popc(m);
            if (want && k < n_have) {
                v = list[k];
                p.refs_out[v] = 1;
            }
            if (c < p.max_pages && (want || p.table_out != p.table_in)) p.table_out[i] = v;
        }
    }
}

// ------------------------------------------------------------------ compact
// With L live pages, those numbered L and up move to the free ones below L
// (there are as many): the fewest moves that leave pages [0, L) live. The k-th
// such page, in order, goes to the k-th hole, so no page is both source and
// destination. ws: n_moves, L, then movers[], holes[], to[num_pages].
__global__ void __launch_bounds__(kBookThreads, 1) compact_plan(const PoolProblem p) {
    __shared__ int sh[33];
    int32_t *n_mv = p.ws, *movers = p.ws + 32, *holes = movers + up32(p.num_pages), *to = holes + up32(p.num_pages);
    const int lane = threadIdx.x & 31;
    int lo, hi, live, n = 0;
    warp_stretch(p.num_pages, lo, hi);
    bool negative = false;
    for_counts(p.refs_in, lo, hi, 0, [&](int, int v) {
        n += __popc(__ballot_sync(kAll, v > 0));
        negative |= v < 0;
    });
    if (negative) atomicOr(p.status, kDevBadIndex);
    const int live_before = warp_prefix(n, sh, live);
    // rank of a hole i < L: free pages before it; of a mover i >= L: live pages
    // before it, less the live ones below L
    int rank = live_before, below = 0;
    for_counts(p.refs_in, lo, hi, 0, [&](int i, int v) {
        const unsigned m = __ballot_sync(kAll, v > 0);
        if (i < live && i < hi && v <= 0) holes[i - rank - __popc(m & ((1u << lane) - 1u))] = i;
        below += __popc(__ballot_sync(kAll, v > 0 && i < live));
        rank += __popc(m);
    });
    int live_below;
    warp_prefix(below, sh, live_below);
    rank = live_before - live_below;
    for_counts(p.refs_in, lo, hi, 0, [&](int i, int v) {
        const unsigned m = __ballot_sync(kAll, v > 0);
        if (v > 0 && i >= live) movers[rank + __popc(m & ((1u << lane) - 1u))] = i;
        rank += __popc(m);
        if (i < hi) to[i] = v > 0 ? i : -1;  // what is free has no place
    });
    __syncthreads();
    const int moves = live - live_below;
    for (int k = threadIdx.x; k < moves; k += kBookThreads) to[movers[k]] = holes[k];
    // counts: a hole takes its mover's, what lies past L becomes free
    if (p.refs_out != p.refs_in)
        for (int i = threadIdx.x; i < live; i += kBookThreads) p.refs_out[i] = p.refs_in[i];
    __syncthreads();
    for (int k = threadIdx.x; k < moves; k += kBookThreads) p.refs_out[holes[k]] = p.refs_in[movers[k]];
    __syncthreads();
    for (int i = live + threadIdx.x; i < p.num_pages; i += kBookThreads) p.refs_out[i] = 0;
    if (threadIdx.x == 0) *n_mv = moves;
}

__global__ void __launch_bounds__(kMoveThreads) compact_apply(const PoolProblem p) {
    const int32_t *n_mv = p.ws, *movers = p.ws + 32, *holes = movers + up32(p.num_pages),
                  *to = holes + up32(p.num_pages);
    const long long cells = (long long)p.B * p.max_pages;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < cells;
         i += (long long)gridDim.x * blockDim.x) {
        int v = page_in(p, p.table_in[i]);
        if (v >= 0) {
            v = to[v];
            if (v < 0) atomicOr(p.status, kDevBadIndex);  // the table names a page that nobody holds
        }
        p.table_out[i] = v;
    }
    move_pages(p, movers, holes, *n_mv, blockIdx.x, gridDim.x);
}

cudaError_t copy_refs(const PoolProblem &p, cudaStream_t stream) {
    if (p.refs_out == p.refs_in) return cudaSuccess;
    return cudaMemcpyAsync(p.refs_out, p.refs_in, (size_t)p.num_pages * 4, cudaMemcpyDeviceToDevice, stream);
}

int clamp_grid(long long want, long long most) { return (int)(want < 1 ? 1 : want > most ? most : want); }

// CTAs for moving up to n pages (and at least `other` for the bookkeeping).
int move_grid(const PoolProblem &p, long long n, long long other, int num_sms) {
    const long long chunks = (long long)((p.page_bytes + kMoveChunk - 1) / kMoveChunk);
    const long long work = 2ll * p.layers * n * chunks;
    return clamp_grid(work > other ? work : other, 6ll * num_sms);
}

}  // namespace

size_t cache_workspace_words(int num_pages, int B) {
    const size_t fork = 4 * (size_t)up32(B) + 32 + up32(B < num_pages ? B : num_pages);
    const size_t reserve = (size_t)up32(B) + 32 + up32(num_pages);
    const size_t compact = 32 + 3 * (size_t)up32(num_pages);
    const size_t a = fork > reserve ? fork : reserve;
    return a > compact ? a : compact;
}

cudaError_t launch_cache_append(const AppendProblem &p, int num_sms, cudaStream_t stream) {
    const int log_ppr = p.row_bytes == 128 ? 3 : p.row_bytes == 256 ? 4 : 5;
    const long long per_head = (((long long)p.m << log_ppr) + kAppendThreads * kAppendVecs - 1) / (kAppendThreads * kAppendVecs);
    const long long heads = (long long)p.B * p.Hkv;
    const dim3 grid(clamp_grid(per_head, 1 << 20), clamp_grid(heads, 65535));
    cache_append<<<grid, kAppendThreads, 0, stream>>>(p, log_ppr);
    return cudaGetLastError();
}

cudaError_t launch_cache_copy(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches) {
    *launches = 0;
    if (p.n == 0) return cudaSuccess;
    cache_move<<<move_grid(p, p.n, 1, num_sms), kMoveThreads, 0, stream>>>(p);
    *launches = 1;
    return cudaGetLastError();
}

cudaError_t launch_cache_fork(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches) {
    fork_plan<<<1, kBookThreads, (size_t)p.B * 4, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    fork_apply<<<move_grid(p, p.n < p.B ? p.n : p.B, p.B, num_sms), kMoveThreads, 0, stream>>>(p);
    *launches = 2;
    return cudaGetLastError();
}

cudaError_t launch_cache_free(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches) {
    cudaError_t e = copy_refs(p, stream);
    if (e != cudaSuccess) return e;
    free_rows<<<clamp_grid(p.B, 8ll * num_sms), 256, 0, stream>>>(p);
    *launches = 1;
    return cudaGetLastError();
}

cudaError_t launch_cache_trim(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches) {
    cudaError_t e = copy_refs(p, stream);
    if (e != cudaSuccess) return e;
    trim_rows<<<clamp_grid(p.B, 8ll * num_sms), 256, 0, stream>>>(p);
    *launches = 1;
    return cudaGetLastError();
}

cudaError_t launch_cache_reserve(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches) {
    reserve_plan<<<1, kBookThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    reserve_apply<<<clamp_grid((p.B + 7) / 8, 8ll * num_sms), 256, 0, stream>>>(p);
    *launches = 2;
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches) {
    compact_plan<<<1, kBookThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long cells = ((long long)p.B * p.max_pages + kMoveThreads - 1) / kMoveThreads;
    compact_apply<<<move_grid(p, p.num_pages / 2, cells, num_sms), kMoveThreads, 0, stream>>>(p);
    *launches = 2;
    return cudaGetLastError();
}

}  // namespace sa
