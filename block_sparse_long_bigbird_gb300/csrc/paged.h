// Internal declarations of the paged key/value cache: the attention of new
// tokens over it and the kernels that write and move its pages.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sparse_attn.h"

namespace sa {

constexpr int kPagedMaxBatch = 1024;   // sequences per call: every CTA plans over them in shared memory
constexpr int kPagedMaxGlobal = 512;   // global positions per call: kept in shared memory
constexpr int kPagedMaxGroup = 64;     // query heads per key head: one token's group fits any row tile
constexpr int kPagedMaxHeads = 256;    // key heads per call: their strides are kept in shared memory
constexpr long long kPagedMaxLen = 1ll << 30;  // tokens per sequence (positions are 32-bit)

// One attention call over a paged cache, as validated by the host API.
struct PagedProblem {
    const void *Q;        // [B][Hq][m][d]
    const void *K, *V;    // [num_pages][Hkv][page][d]
    void *O;              // [B][Hq][m][d]
    int B, Hq, Hkv, m, d;
    int page, num_pages, max_pages;
    const int32_t *table;  // [B][max_pages], -1: no page
    const int32_t *lens;   // [B] tokens in the cache, the new ones included
    const int32_t *qlens;  // [B] new tokens, or NULL (m each)
    int half;              // window / 2: keys seen before the query
    const int32_t *dilation;  // [Hq] or NULL
    const int32_t *gidx;
    int ng;
    unsigned *status;
    // set by the launcher
    int group;       // Hq / Hkv
    int log_page;
    int tpt;         // tokens per unit
    int tpt_half;    // tokens per half of a unit (tpt: units of one half)
    int rows;        // rows per unit: tpt * group
    int cut;         // whether tiles may be split (then there is a plan, and paged_merge is launched)
    int slots;       // CTAs that share the work
    int min_piece;   // fewest 64-key blocks worth a CTA of their own
    int cost;        // what a tile costs beside its blocks, in blocks
    int listed;      // whether a tile's far global keys are walked side by side, 64 to an entry (paged_tile)
    int warps;       // warps of a CTA (paged_few)
    int whole;       // blocks that a CTA may walk beyond an even share before splitting tiles pays
    float scale_log2;
    unsigned long long wait_ns;
    float *part_o;   // [2 slots][d / 4][rows][4] partial sums of split tiles
    float2 *part_ml; // [2 slots][rows] (running maximum, sum)
};

// Which kernel serves a call: few rows per key head on the ordinary units or, in
// bf16, on warp-level matrix instructions; many rows in bf16 on the tensor cores;
// many rows on the ordinary units.
enum PagedKernel { kPagedRows = 0, kPagedFew = 1, kPagedTc = 2, kPagedTile = 3 };

// Fills the launcher's fields of `p` and says which kernel runs it.
PagedKernel paged_shape(PagedProblem &p, sa_dtype dtype, bool force_simt, int num_sms);
// CTAs of the streaming kernels that fit an SM, by the rows of a unit.
constexpr int paged_rows_ctas(int rows) { return rows <= 4 ? 2 : 1; }
constexpr int paged_few_ctas(int d, int rows, int warps) {
    return (d == 64 ? rows <= 16 ? 16 : 12 : 8) / warps;
}
// Scratch of one call: partial results of split tiles (0: nothing is split).
size_t paged_workspace_bytes(const PagedProblem &p);
cudaError_t launch_paged_rows(const PagedProblem &p, sa_dtype dtype, cudaStream_t stream);
cudaError_t launch_paged_few(const PagedProblem &p, cudaStream_t stream);
cudaError_t launch_paged_tile(const PagedProblem &p, sa_dtype dtype, cudaStream_t stream);
cudaError_t launch_paged_tc(const PagedProblem &p, cudaStream_t stream);
cudaError_t launch_paged_merge(const PagedProblem &p, sa_dtype dtype, int num_sms, cudaStream_t stream);

// Writing and moving pages (paged_cache.cu).
struct AppendProblem {
    const void *Kn, *Vn;  // [B][Hkv][m][d]
    void *K, *V;          // [num_pages][Hkv][page][d]
    int B, Hkv, m;
    int row_bytes;        // d * element size
    int page, log_page, num_pages, max_pages;
    const int32_t *table, *lens, *qlens;
    unsigned *status;
};
cudaError_t launch_cache_append(const AppendProblem &p, int num_sms, cudaStream_t stream);

struct PoolProblem {
    uint8_t *K, *V;       // [layers][num_pages][page_bytes]
    int layers, num_pages;
    size_t page_bytes;
    int page, log_page, B, max_pages;
    const int32_t *table_in, *lens_in, *refs_in;
    int32_t *table_out, *lens_out, *refs_out;
    const int32_t *src, *dst;  // rows or pages, `n` of each
    int n;
    const int32_t *qlens;
    int reach;
    const int32_t *gidx;
    int ng;
    unsigned *status;
    int32_t *ws;
};
// Scratch words (int32) of the calls below, an upper bound over all of them.
size_t cache_workspace_words(int num_pages, int B);
cudaError_t launch_cache_copy(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches);
cudaError_t launch_cache_fork(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches);
cudaError_t launch_cache_free(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches);
cudaError_t launch_cache_trim(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches);
cudaError_t launch_cache_reserve(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches);
cudaError_t launch_cache_compact(const PoolProblem &p, int num_sms, cudaStream_t stream, int *launches);

// Shared with the other entry points (api.cu): the current device's status
// word and SM count; SA_ERR_UNSUPPORTED off sm_103. The launch count of the
// calling thread's last call; options.
sa_status api_device(unsigned **status, int *num_sms);
void api_set_launches(int n);
bool api_force_simt();
unsigned long long api_wait_ns();

}  // namespace sa
