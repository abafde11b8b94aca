// Host side of the paged cache's entry points: argument checks, the choice of
// kernel, scratch sizes and launches. Nothing is kept between calls.
#include <cuda_runtime.h>
#include <math.h>

#include "internal.h"
#include "paged.h"

namespace sa {

// The most query rows per key head of the kernels that stream the cache. On the
// ordinary units: one in bf16 (from two on the matrix instructions of paged_few
// are ahead: 64 sequences of 4096 tokens, 8 key heads, d = 64, take 96 us for one
// row on either, 102 against 96 us for two, 174 against 97 us for three), and
// eight in fp32. With warp-level matrix instructions up to 24 rows, 128-row tiles
// beyond: the same batch with 24 rows takes 137 against 168 us, 16 sequences of
// 32768 tokens 237 against 241 us (d = 128: 341 and 358); 32 rows would take 160
// and 167, 271 and 240, 481 and 356 us.
constexpr int kRowsBf16 = 1, kRowsFp32 = 8, kFewRows = 24;

// ns: the longest walk of a global token that is left to one CTA (paged_shape).
constexpr long long kGlobalWalk = 200000;

PagedKernel paged_shape(PagedProblem &p, sa_dtype dtype, bool force_simt, int num_sms) {
    p.group = p.Hq / p.Hkv;
    p.log_page = p.page == 16 ? 4 : p.page == 32 ? 5 : p.page == 64 ? 6 : 7;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)p.d);
    const long long rows = (long long)p.m * p.group;
    PagedKernel kind;
    int per_sm = 1;
    // ns: a 64-key block in a CTA that has the SM to itself (or its usual share),
    // and what splitting tiles adds to a call (more units, and the join)
    int block_ns, split_ns = 12000;
    if (rows <= (dtype == SA_FP32 ? kRowsFp32 : kRowsBf16)) {
        kind = kPagedRows;
        p.tpt = p.tpt_half = p.m;
        p.rows = (int)rows;
        per_sm = paged_rows_ctas(p.rows);
        p.min_piece = 4;
        p.cost = 4;
        block_ns = dtype == SA_FP32 ? p.d / 64 * (450 + 130 * p.rows) : p.d == 64 ? 450 : 550;
    } else if (dtype == SA_BF16 && !force_simt && rows <= kFewRows) {
        kind = kPagedFew;
        p.tpt = p.tpt_half = p.m;
        p.rows = (int)rows;
        // CTAs of four warps where there are tiles for all of them, so that others stream
        // while one starts or joins its unit, and of as many as registers allow else: 64
        // sequences of 900 tokens, 8 key heads, 4 rows, d = 128, take 50 us, 58 with eight
        // warps; one sequence 17.8 and 15.1.
        p.warps = (long long)p.B * p.Hkv >= 2ll * num_sms ? 4 : p.d == 64 && rows > 16 ? 12 : 8;
        per_sm = paged_few_ctas(p.d, p.rows, p.warps);
        p.min_piece = 4;
        p.cost = 4;
        block_ns = p.d == 64 ? 450 : 650;
        split_ns = 14000;
    } else if (dtype == SA_BF16 && !force_simt) {
        kind = kPagedTc;
        const int most = 128 / p.group;
        p.tpt_half = p.m < most ? p.m : most;
        const int halves = p.m > p.tpt_half ? 2 : 1;
        p.tpt = halves * p.tpt_half;
        p.rows = halves * p.tpt_half * p.group;
        p.min_piece = 8;
        p.cost = 3;
        block_ns = halves == 2 ? 1000 : 550;
        split_ns = 28000;
    } else {
        kind = kPagedTile;
        const int most = 64 / p.group;
        p.tpt = p.tpt_half = p.m < most ? p.m : most;
        p.rows = p.tpt * p.group;
        per_sm = p.d == 64 ? 4 : 2;
        p.min_piece = 2;
        p.cost = 1;
        p.listed = 1;
        block_ns = p.d == 64 ? 7200 : 13000;
        split_ns = 20000;
    }
    // Whole tiles take as many rounds of the GPU's CTAs as there are tiles to a CTA,
    // rounded up; split ones share the blocks evenly, also with CTAs that had no
    // tile. One token, 8 key heads, d = 128, one sequence: 900 keys take 15.4 us whole
    // and 15.6 split, 4000 keys 46 and 18; 8 sequences of 900 keys 15.8 and 20; in
    // fp32 with four rows 900 keys 34 and 21. 1000 tokens with a window of 512 over
    // 8192 keys, 12 heads, four sequences: 34 and 62.
    // The device decides by the lengths. The host leaves plan and join out where
    // splitting would not pay if every tile took the longest walk, and that is not so
    // long that uneven lengths would make up for it. No tile walks more than its table
    // row or, without dilation, its window and a block per global position (listed
    // ones 64 to an entry); but one with a global token, which only the device can tell,
    // walks its whole sequence. Such tokens are few, and plan and join cost every call (a
    // step of one sequence, window 512, 16 global: 10.0 us with, 7.8 without), so they
    // come in for it where its walk would take kGlobalWalk in one CTA: a global token at
    // the end of 65536 keys, 12 heads of 64, takes 60 us with them and 536 without.
    p.whole = split_ns / block_ns;
    const long long tiles = (long long)p.B * p.Hkv * ((p.m + p.tpt - 1) / p.tpt);
    const long long row = (((long long)p.max_pages << p.log_page) + 63) >> 6;
    long long longest = row;
    if (!p.dilation && p.half < longest << 6) {
        const long long band = (((long long)p.half + p.tpt) >> 6) + 2 + (p.listed ? (p.ng + 63) >> 6 : p.ng);
        longest = band < longest ? band : longest;
    }
    longest += p.cost;
    const long long ctas = (long long)num_sms * per_sm;
    auto share = [&](long long walk) {  // CTAs that get a piece each
        const long long pieces = tiles * (walk / p.min_piece + 1);
        return pieces < ctas ? pieces : ctas;
    };
    p.cut = (tiles + ctas - 1) / ctas * longest - tiles * longest / share(longest) > p.whole || longest > 2ll * p.whole ||
            (p.ng > 0 && row * block_ns > kGlobalWalk);
    // A global token's walk may be shared by a CTA per SM; more of them, idle on most
    // calls, would cost those (5 tokens of 8 sequences in fp32: 36 us, 42 with 4 per SM).
    long long slots = p.cut ? share(longest) : tiles < ctas ? tiles : ctas;
    if (p.cut && p.ng > 0 && slots < num_sms) slots = share(row + p.cost) < num_sms ? share(row + p.cost) : num_sms;
    p.slots = (int)slots;
    return kind;
}

size_t paged_workspace_bytes(const PagedProblem &p) {
    return p.cut ? 2 * (size_t)p.slots * p.rows * (p.d + 2) * sizeof(float) : 0;
}

}  // namespace sa

namespace {

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// Sizes of the attention and the append; the limits come after the contract.
sa_status sizes_ok(int B, int Hkv, int m, int d, int page, int num_pages, int max_pages) {
    if (B < 1 || Hkv < 1 || m < 1 || num_pages < 1 || max_pages < 1) return SA_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || !page_ok(page)) return SA_ERR_INVALID_ARG;
    if (B > sa::kPagedMaxBatch || (long long)max_pages * page > sa::kPagedMaxLen) return SA_ERR_UNSUPPORTED;
    if ((long long)num_pages * Hkv > 0x7fffffffll || (long long)B * Hkv * m > 0x3fffffffll) return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

sa_status finish(cudaError_t e, int launches) {
    if (e == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return SA_ERR_CUDA;
    sa::api_set_launches(launches);
    return SA_OK;
}

// Sizes and pointers that the bookkeeping calls share.
sa_status pool_ok(const void *K, const void *V, int layers, int num_pages, size_t page_bytes) {
    if (!K || !V || K == V || !al16(K) || !al16(V)) return SA_ERR_INVALID_ARG;
    if (layers < 1 || num_pages < 1 || page_bytes == 0 || (page_bytes & 15u)) return SA_ERR_INVALID_ARG;
    if (page_bytes > (1ull << 40) / (size_t)num_pages || layers > (1 << 16)) return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

sa_status tables_ok(int B, int max_pages, int num_pages, const void *a, const void *b, const void *c, const void *d) {
    if (B < 1 || max_pages < 1 || num_pages < 1) return SA_ERR_INVALID_ARG;
    if (!a || !b || !c || !d || !al4(a) || !al4(b) || !al4(c) || !al4(d)) return SA_ERR_INVALID_ARG;
    if (B > sa::kPagedMaxBatch) return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

sa_status ws_ok(const void *ws, size_t bytes, size_t need) {
    return ws && al16(ws) && bytes >= need ? SA_OK : SA_ERR_INVALID_ARG;
}

int log2_page(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

}  // namespace

extern "C" {

sa_status longformer_attn_paged_fwd(const void *Q, const void *K_pages, const void *V_pages, void *O, int B, int Hq,
                                    int Hkv, int m, int d, int page, int num_pages, int max_pages,
                                    const int32_t *block_table, const int32_t *seq_lens, const int32_t *q_lens,
                                    int window, const int32_t *dilation, const int32_t *global_idx, int n_global,
                                    void *workspace, size_t workspace_bytes, sa_dtype dtype, sa_stream_t stream) {
    if (dtype != SA_BF16 && dtype != SA_FP32) return SA_ERR_INVALID_ARG;
    if (!Q || !K_pages || !V_pages || !O || !al16(Q) || !al16(K_pages) || !al16(V_pages) || !al16(O))
        return SA_ERR_INVALID_ARG;
    if (O == Q || O == K_pages || O == V_pages) return SA_ERR_INVALID_ARG;
    if (!block_table || !seq_lens || !al4(block_table) || !al4(seq_lens) || !al4(q_lens) || !al4(dilation) ||
        !al4(global_idx))
        return SA_ERR_INVALID_ARG;
    if (window < 0 || (window & 1) || n_global < 0 || (n_global > 0 && !global_idx)) return SA_ERR_INVALID_ARG;
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return SA_ERR_INVALID_ARG;
    sa_status s = sizes_ok(B, Hkv, m, d, page, num_pages, max_pages);
    if (s != SA_OK) return s;
    if (Hq / Hkv > sa::kPagedMaxGroup || Hkv > sa::kPagedMaxHeads || n_global > sa::kPagedMaxGlobal || (long long)B * Hq > (1ll << 30))
        return SA_ERR_UNSUPPORTED;
    sa::PagedProblem p = {};
    int sms = 0;
    s = sa::api_device(&p.status, &sms);
    if (s != SA_OK) return s;
    p.Q = Q; p.K = K_pages; p.V = V_pages; p.O = O;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.m = m; p.d = d;
    p.page = page; p.num_pages = num_pages; p.max_pages = max_pages;
    p.table = block_table; p.lens = seq_lens; p.qlens = q_lens;
    p.half = window / 2;
    p.dilation = dilation;
    p.gidx = n_global > 0 ? global_idx : nullptr;
    p.ng = n_global;
    p.wait_ns = sa::api_wait_ns();
    // the scratch that any window needs, then what this one makes of it (not more)
    sa::PagedProblem any = p;
    any.half = (int)sa::kPagedMaxLen;
    sa::paged_shape(any, dtype, sa::api_force_simt(), sms);
    const size_t room = sa::paged_workspace_bytes(any);
    if (room && ws_ok(workspace, workspace_bytes, room) != SA_OK) return SA_ERR_INVALID_ARG;
    const sa::PagedKernel kind = sa::paged_shape(p, dtype, sa::api_force_simt(), sms);
    const size_t need = sa::paged_workspace_bytes(p);
    if (need) {
        if (ws_ok(workspace, workspace_bytes, need) != SA_OK) return SA_ERR_INVALID_ARG;
        p.part_o = static_cast<float *>(workspace);
        p.part_ml = reinterpret_cast<float2 *>(p.part_o + 2 * (size_t)p.slots * p.rows * p.d);
    }
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = kind == sa::kPagedRows ? sa::launch_paged_rows(p, dtype, cs)
                    : kind == sa::kPagedFew ? sa::launch_paged_few(p, cs)
                    : kind == sa::kPagedTc ? sa::launch_paged_tc(p, cs)
                                           : sa::launch_paged_tile(p, dtype, cs);
    if (e == cudaSuccess && need) e = sa::launch_paged_merge(p, dtype, sms, cs);
    return finish(e, need ? 2 : 1);
}

size_t sa_longformer_paged_workspace_bytes(int B, int Hq, int Hkv, int m, int d, int page, int max_pages,
                                           sa_dtype dtype) {
    if ((dtype != SA_BF16 && dtype != SA_FP32) || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 ||
        Hq / Hkv > sa::kPagedMaxGroup || Hkv > sa::kPagedMaxHeads || sizes_ok(B, Hkv, m, d, page, 1, max_pages) != SA_OK)
        return 0;
    unsigned *status = nullptr;
    int sms = 0;
    if (sa::api_device(&status, &sms) != SA_OK) return 0;
    sa::PagedProblem p = {};
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.m = m; p.d = d; p.page = page; p.max_pages = max_pages;
    p.half = (int)sa::kPagedMaxLen;
    size_t most = 0;  // whichever kernel SA_OPT_FORCE_SIMT chooses by then
    for (int simt = 0; simt < 2; ++simt) {
        sa::paged_shape(p, dtype, simt != 0, sms);
        const size_t n = sa::paged_workspace_bytes(p);
        most = n > most ? n : most;
    }
    return most;
}

sa_status sa_cache_append(const void *K_new, const void *V_new, void *K_pages, void *V_pages, int B, int Hkv, int m,
                          int d, int page, int num_pages, int max_pages, const int32_t *block_table,
                          const int32_t *seq_lens, const int32_t *q_lens, sa_dtype dtype, sa_stream_t stream) {
    if (dtype != SA_BF16 && dtype != SA_FP32) return SA_ERR_INVALID_ARG;
    const void *t[4] = {K_new, V_new, K_pages, V_pages};
    for (int i = 0; i < 4; ++i) {
        if (!t[i] || !al16(t[i])) return SA_ERR_INVALID_ARG;
        for (int j = 2; j < i; ++j)
            if (t[i] == t[j]) return SA_ERR_INVALID_ARG;
    }
    if (K_new == K_pages || K_new == V_pages || V_new == K_pages || V_new == V_pages) return SA_ERR_INVALID_ARG;
    if (!block_table || !seq_lens || !al4(block_table) || !al4(seq_lens) || !al4(q_lens)) return SA_ERR_INVALID_ARG;
    sa_status s = sizes_ok(B, Hkv, m, d, page, num_pages, max_pages);
    if (s != SA_OK) return s;
    sa::AppendProblem p = {};
    int sms = 0;
    s = sa::api_device(&p.status, &sms);
    if (s != SA_OK) return s;
    p.Kn = K_new; p.Vn = V_new; p.K = K_pages; p.V = V_pages;
    p.B = B; p.Hkv = Hkv; p.m = m;
    p.row_bytes = d * (dtype == SA_FP32 ? 4 : 2);
    p.page = page; p.log_page = log2_page(page); p.num_pages = num_pages; p.max_pages = max_pages;
    p.table = block_table; p.lens = seq_lens; p.qlens = q_lens;
    return finish(sa::launch_cache_append(p, sms, reinterpret_cast<cudaStream_t>(stream)), 1);
}

size_t sa_cache_workspace_bytes(int num_pages, int B) {
    if (num_pages < 1 || B < 1 || B > sa::kPagedMaxBatch) return 0;
    return 4 * sa::cache_workspace_words(num_pages, B);
}

sa_status sa_cache_copy_pages(void *K_pages, void *V_pages, int layers, int num_pages, size_t page_bytes,
                              const int32_t *src, const int32_t *dst, int count, sa_stream_t stream) {
    sa_status s = pool_ok(K_pages, V_pages, layers, num_pages, page_bytes);
    if (s != SA_OK) return s;
    if (count < 0 || (count > 0 && (!src || !dst || !al4(src) || !al4(dst)))) return SA_ERR_INVALID_ARG;
    sa::PoolProblem p = {};
    int sms = 0, launches = 0;
    s = sa::api_device(&p.status, &sms);
    if (s != SA_OK) return s;
    p.K = static_cast<uint8_t *>(K_pages);
    p.V = static_cast<uint8_t *>(V_pages);
    p.layers = layers; p.num_pages = num_pages; p.page_bytes = page_bytes;
    p.src = src; p.dst = dst; p.n = count;
    const cudaError_t e = sa::launch_cache_copy(p, sms, reinterpret_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

sa_status sa_cache_fork(void *K_pages, void *V_pages, int layers, int num_pages, size_t page_bytes, int page, int B,
                        int max_pages, const int32_t *src, const int32_t *dst, int count, const int32_t *table_in,
                        const int32_t *lens_in, const int32_t *ref_in, int32_t *table_out, int32_t *lens_out,
                        int32_t *ref_out, void *workspace, size_t workspace_bytes, sa_stream_t stream) {
    sa_status s = pool_ok(K_pages, V_pages, layers, num_pages, page_bytes);
    if (s != SA_OK) return s;
    if (!page_ok(page) || count < 0 || (count > 0 && (!src || !dst || !al4(src) || !al4(dst)))) return SA_ERR_INVALID_ARG;
    if ((s = tables_ok(B, max_pages, num_pages, table_in, ref_in, table_out, ref_out)) != SA_OK) return s;
    if (!lens_in || !lens_out || !al4(lens_in) || !al4(lens_out)) return SA_ERR_INVALID_ARG;
    if ((long long)max_pages * page > sa::kPagedMaxLen) return SA_ERR_UNSUPPORTED;
    if ((s = ws_ok(workspace, workspace_bytes, sa_cache_workspace_bytes(num_pages, B))) != SA_OK) return s;
    sa::PoolProblem p = {};
    int sms = 0, launches = 0;
    s = sa::api_device(&p.status, &sms);
    if (s != SA_OK) return s;
    p.K = static_cast<uint8_t *>(K_pages);
    p.V = static_cast<uint8_t *>(V_pages);
    p.layers = layers; p.num_pages = num_pages; p.page_bytes = page_bytes;
    p.page = page; p.log_page = log2_page(page); p.B = B; p.max_pages = max_pages;
    p.src = src; p.dst = dst; p.n = count;
    p.table_in = table_in; p.lens_in = lens_in; p.refs_in = ref_in;
    p.table_out = table_out; p.lens_out = lens_out; p.refs_out = ref_out;
    p.ws = static_cast<int32_t *>(workspace);
    const cudaError_t e = sa::launch_cache_fork(p, sms, reinterpret_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

sa_status sa_cache_free(int num_pages, int B, int max_pages, const int32_t *rows, int count, const int32_t *table_in,
                        const int32_t *lens_in, const int32_t *ref_in, int32_t *table_out, int32_t *lens_out,
                        int32_t *ref_out, sa_stream_t stream) {
    sa_status s = tables_ok(B, max_pages, num_pages, table_in, ref_in, table_out, ref_out);
    if (s != SA_OK) return s;
    if (!lens_in || !lens_out || !al4(lens_in) || !al4(lens_out)) return SA_ERR_INVALID_ARG;
    if (count < 0 || (count > 0 && (!rows || !al4(rows)))) return SA_ERR_INVALID_ARG;
    sa::PoolProblem p = {};
    int sms = 0, launches = 0;
    s = sa::api_device(&p.status, &sms);
    if (s != SA_OK) return s;
    p.num_pages = num_pages; p.B = B; p.max_pages = max_pages;
    p.src = rows; p.n = count;
    p.table_in = table_in; p.lens_in = lens_in; p.refs_in = ref_in;
    p.table_out = table_out; p.lens_out = lens_out; p.refs_out = ref_out;
    const cudaError_t e = sa::launch_cache_free(p, sms, reinterpret_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

sa_status sa_cache_trim(int num_pages, int page, int B, int max_pages, int reach, const int32_t *global_idx,
                        int n_global, const int32_t *table_in, const int32_t *seq_lens, const int32_t *ref_in,
                        int32_t *table_out, int32_t *ref_out, sa_stream_t stream) {
    sa_status s = tables_ok(B, max_pages, num_pages, table_in, ref_in, table_out, ref_out);
    if (s != SA_OK) return s;
    if (!page_ok(page) || reach < 0 || !seq_lens || !al4(seq_lens)) return SA_ERR_INVALID_ARG;
    if (n_global < 0 || (n_global > 0 && (!global_idx || !al4(global_idx)))) return SA_ERR_INVALID_ARG;
    sa::PoolProblem p = {};
    int sms = 0, launches = 0;
    s = sa::api_device(&p.status, &sms);
    if (s != SA_OK) return s;
    p.num_pages = num_pages; p.page = page; p.log_page = log2_page(page); p.B = B; p.max_pages = max_pages;
    p.reach = reach;
    p.gidx = global_idx; p.ng = n_global;
    p.table_in = table_in; p.lens_in = seq_lens; p.refs_in = ref_in;
    p.table_out = table_out; p.refs_out = ref_out;
    const cudaError_t e = sa::launch_cache_trim(p, sms, reinterpret_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

sa_status sa_cache_reserve(int num_pages, int page, int B, int max_pages, const int32_t *seq_lens,
                           const int32_t *q_lens, const int32_t *table_in, const int32_t *ref_in, int32_t *table_out,
                           int32_t *ref_out, void *workspace, size_t workspace_bytes, sa_stream_t stream) {
    sa_status s = tables_ok(B, max_pages, num_pages, table_in, ref_in, table_out, ref_out);
    if (s != SA_OK) return s;
    if (!page_ok(page) || !seq_lens || !q_lens || !al4(seq_lens) || !al4(q_lens)) return SA_ERR_INVALID_ARG;
    if ((long long)max_pages * page > sa::kPagedMaxLen) return SA_ERR_UNSUPPORTED;
    if ((long long)B * max_pages > 0x7fffffffll) return SA_ERR_UNSUPPORTED;  // the pages asked for are counted in 32 bits
    if ((s = ws_ok(workspace, workspace_bytes, sa_cache_workspace_bytes(num_pages, B))) != SA_OK) return s;
    sa::PoolProblem p = {};
    int sms = 0, launches = 0;
    s = sa::api_device(&p.status, &sms);
    if (s != SA_OK) return s;
    p.num_pages = num_pages; p.page = page; p.log_page = log2_page(page); p.B = B; p.max_pages = max_pages;
    p.qlens = q_lens;
    p.table_in = table_in; p.lens_in = seq_lens; p.refs_in = ref_in;
    p.table_out = table_out; p.refs_out = ref_out;
    p.ws = static_cast<int32_t *>(workspace);
    const cudaError_t e = sa::launch_cache_reserve(p, sms, reinterpret_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

sa_status sa_cache_compact(void *K_pages, void *V_pages, int layers, int num_pages, size_t page_bytes, int B,
                           int max_pages, const int32_t *table_in, const int32_t *ref_in, int32_t *table_out,
                           int32_t *ref_out, void *workspace, size_t workspace_bytes, sa_stream_t stream) {
    sa_status s = pool_ok(K_pages, V_pages, layers, num_pages, page_bytes);
    if (s != SA_OK) return s;
    if ((s = tables_ok(B, max_pages, num_pages, table_in, ref_in, table_out, ref_out)) != SA_OK) return s;
    if ((s = ws_ok(workspace, workspace_bytes, sa_cache_workspace_bytes(num_pages, B))) != SA_OK) return s;
    sa::PoolProblem p = {};
    int sms = 0, launches = 0;
    s = sa::api_device(&p.status, &sms);
    if (s != SA_OK) return s;
    p.K = static_cast<uint8_t *>(K_pages);
    p.V = static_cast<uint8_t *>(V_pages);
    p.layers = layers; p.num_pages = num_pages; p.page_bytes = page_bytes;
    p.B = B; p.max_pages = max_pages;
    p.table_in = table_in; p.refs_in = ref_in; p.table_out = table_out; p.refs_out = ref_out;
    p.ws = static_cast<int32_t *>(workspace);
    const cudaError_t e = sa::launch_cache_compact(p, sms, reinterpret_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

}  // extern "C"
