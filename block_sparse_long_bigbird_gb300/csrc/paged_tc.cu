// Attention of many new tokens over a paged cache on the tensor cores (bf16):
// chunks of a prompt, drafts, and single tokens whose query heads share a key
// head.
//
// A unit's query rows (tokens x the query heads of one key head, up to 2 x 128)
// are two MMA tiles of 128 rows that share every key and value they load: a
// 128-key stage serves 2 x 128 x 128 products, which halves the L2 traffic per
// flop, and one tile's softmax overlaps the other's MMAs.
//   * Two loader warps walk the unit's 64-key blocks two at a time, look the
//     pages up (a step ahead), and load K and V with one tensor copy per page
//     piece; a third warp writes down what each step holds for the
//     two tiles. The pool is {d, page, num_pages * Hkv}, a box is 64 columns of
//     one page (at most 64 tokens). A missing page is loaded from coordinate
//     -1, which fills with zeros, so stages always fill.
//   * The MMA warp runs S_x = Q_x K^T for each tile into 128 TMEM columns and
//     O_x += P_x V with P_x read from TMEM, where the softmax wrote it (bf16)
//     over the first half of S_x. One thread issues all MMAs, so they complete
//     in order: S_x of a step complete means P_x V of the step before is too.
//   * A warpgroup per tile runs the softmax, one thread per row: masks, running
//     maximum (kept until it grows by more than 2^8, then O is rescaled in
//     place), weights and their sum in fp32, P rounded to bf16 (relative 2^-8,
//     the rounding the dense path of this library makes too).
// Memory where no token was written may hold NaN: those V rows are zeroed in
// shared memory before the product. Any other masked infinity or NaN makes its
// row's O not finite, and exact_row then computes that row again.
// Roles' waits are bounded; on expiry the CTA latches SA_ERR_TIMEOUT, drains
// its copies and MMAs, frees TMEM and exits.
#include <cuda.h>

#include <type_traits>

#include "paged_common.cuh"
#include "tc_sync.cuh"

namespace sa {
namespace {

using namespace ptx;
using namespace tcsync;

constexpr int kTcThreads = 384;  // 8 softmax warps, K loader, MMA issuer, step records, V loader
constexpr int kRegion = 128 * 128;  // 128 rows x 128 B: one 64-column piece of a tile
constexpr float kGrow = 8.0f;       // growth of the maximum (log2) that rescales O
constexpr int kSI = 4;              // step records in flight

struct StepRec {
    int blk[2];          // 64-key blocks (-1: none)
    int use;             // bit x: tile x has a row that sees something here; bit 2 + x: every row sees every key
    int vz0, vz1;        // V rows to zero (keys where no token was written)
    int pad;
    uint64_t gbits[2];   // global keys
    uint64_t present[2]; // keys whose page is there
};

template <int D>
struct TcCfg {
    static constexpr int DC = D / 64;               // 64-column pieces
    static constexpr int TILE = DC * kRegion;       // Q tile, K or V stage
    static constexpr int NST = D == 64 ? 8 : 4;     // stages, K and V alternating
    static constexpr int Q_OFF = 0;
    static constexpr int ST_OFF = 2 * TILE;
    static constexpr int BAR_OFF = ST_OFF + NST * TILE;
    static constexpr int B_KF = 0, B_KE = B_KF + NST, B_IF = B_KE + NST, B_IE = B_IF + kSI, B_QF = B_IE + kSI,
                         B_QE = B_QF + 1, B_SF = B_QE + 1, B_PF = B_SF + 2, B_OF = B_PF + 4, B_OE = B_OF + 2,
                         B_MF = B_OE + 2, B_ME = B_MF + 1, B_DRAIN = B_ME + 1, B_COUNT = B_DRAIN + 1;
    static constexpr int REC_OFF = (BAR_OFF + B_COUNT * 8 + 15) & ~15;
    static constexpr int MISC_OFF = REC_OFF + kSI * (int)sizeof(StepRec);
    static constexpr int ML_OFF = MISC_OFF + 16;       // one-tile units: the second chain's (maximum, sum) per row
    static constexpr int PLAN_OFF = ML_OFF + 128 * 8;
    static constexpr uint32_t O_COL = 256;
};
static_assert(sizeof(StepRec) == 56 && (kSI * sizeof(StepRec)) % 16 == 0, "step record layout");

// What tile x of a unit sees, and whether it has rows at all.
struct TileSpan {
    int p0, p1;   // positions of its first and last token
    int first;    // first position that any of its rows may see in a window
    int last;     // first position that the windows of all its rows hold (stride 1)
    bool live;
};

__device__ __forceinline__ TileSpan tile_span(const PagedProblem &p, const Plan &P, const Unit &U, int x, int stride) {
    TileSpan s;
    const int t0 = U.t0 + x * p.tpt_half;
    s.live = U.live && t0 < U.q && (x == 0 || p.tpt > p.tpt_half);
    const int p0 = s.p0 = U.s - U.q + t0;
    s.p1 = U.s - U.q + min(t0 + p.tpt_half, U.q) - 1;
    s.first = max(0, p0 - head_reach(p, stride));
    s.last = s.p1 - head_reach(p, 1);
    if (p.ng && s.live) {
        const int i = lower_bound(P.gpos, p.ng, p0);
        if (i < p.ng && P.gpos[i] <= s.p1) s.first = 0;
    }
    return s;
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const PagedProblem p) {
    using C = TcCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    StepRec *recs = reinterpret_cast<StepRec *>(smem + C::REC_OFF);
    auto bar = [&](int i) { return sbase + C::BAR_OFF + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Ctl ctl{abort_flag, p.status, p.wait_ns};

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(bar(C::B_KF + i), 1);
            mbar_init(bar(C::B_KE + i), 1);
        }
        for (int i = 0; i < kSI; ++i) {
            mbar_init(bar(C::B_IF + i), 1);
            mbar_init(bar(C::B_IE + i), 9);  // 8 softmax warps and the MMA warp
        }
        mbar_init(bar(C::B_QF), 1);
        mbar_init(bar(C::B_QE), 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(C::B_SF + x), 1);
            mbar_init(bar(C::B_PF + 2 * x), 4);
            mbar_init(bar(C::B_PF + 2 * x + 1), 4);
            mbar_init(bar(C::B_OF + x), 1);
            mbar_init(bar(C::B_OE + x), 4);
        }
        mbar_init(bar(C::B_MF), 4);
        mbar_init(bar(C::B_ME), 4);
        mbar_init(bar(C::B_DRAIN), 1);
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_holder), 512);
        tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    Plan P = plan_at(smem + C::PLAN_OFF, p.B, p.ng, p.Hkv);
    tc_fence_before();
    make_plan(p, P);
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    asm volatile("griddepcontrol.launch_dependents;");  // the join may start planning
    uint32_t g = 0;   // steps so far; every role counts the same ones
    bool ok = true;
    const bool one = p.tpt == p.tpt_half;  // units of one tile: its steps alternate between two chains
    Units units(p, P, blockIdx.x);
    Unit U;
    // Position in the stage ring of step i's K and V, in a unit of n steps that
    // begins at step g0. Two tiles: K and V in turn, as they are used. Two
    // chains of one tile: V of a step is used after K of the next.
    auto k_at = [&](uint32_t g0, int i) { return 2 * g0 + (uint32_t)(one && i > 0 ? 2 * i - 1 : 2 * i); };
    auto v_at = [&](uint32_t g0, int i, int n) {
        return 2 * g0 + (uint32_t)(one ? (i == n - 1 ? 2 * n - 1 : 2 * i + 2) : 2 * i + 1);
    };

    // The launch gave every thread 168 registers (384 x 168 = 64512); the
    // softmax holds a row of scores, so its 8 warps take 192 and the others 120
    // (256 x 192 + 128 x 120 = 64512).
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        // ================================================================ softmax and epilogue of tile x
        const int x = warp >> 2;
        const int tid = threadIdx.x & 127;  // row of the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + x * 128, o_addr = tmem + lane_base + C::O_COL + x * D;
        const int half_rows = p.tpt_half * p.group;
        const float sl2 = p.scale_log2;
        uint32_t sc = 0, oc = 0, oc2 = 0, mc = 0;
        while (ok && units.next(p, P, U)) {
            const int n = U.live ? (U.e1 - U.e0 + 1) >> 1 : 0;
            const uint32_t g0 = g;
            int t = 0, head = 0;
            Row row = {};
            const bool in = tid < half_rows;
            if (in) {
                row_token(p, U, tid, p.tpt_half, t, head);
                if (!one) t += x * p.tpt_half;
                row = make_row(p, P, U, head, t);
            }
            const bool busy = __any_sync(kAllLanes, row.valid);
            float mref = -CUDART_INF_F, l = 0.f;
            bool had = false;
            for (int i = 0; i < n; ++i, ++g) {
                const uint32_t slot = g % kSI;
                if (!(ok = wait_warp(bar(C::B_IF + slot), (g / kSI) & 1, ctl))) break;
                const int use = recs[slot].use, vz0 = recs[slot].vz0, vz1 = recs[slot].vz1;
                uint64_t w[2] = {~0ull, ~0ull};
                const bool all = (use >> (2 + x)) & 1;
                if (((use >> x) & 1) && !all) {
                    w[0] = w[1] = 0ull;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (recs[slot].blk[k] >= 0)
                            w[k] = row_mask(row, recs[slot].blk[k], recs[slot].gbits[k], recs[slot].present[k]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_IE + slot));
                if (!((use >> x) & 1)) continue;
                if (!(ok = wait_warp(bar(C::B_SF + x), sc & 1, ctl))) break;
                ++sc;
                // Unwritten memory: no NaN may meet a zero weight. (Not before S is
                // there: only then are the products that read what the stage held
                // before complete, and the wait below is for this step's V.)
                if (vz0 < vz1) {
                    const uint32_t sidx = v_at(g0, i, n), st = sidx % C::NST;
                    if (!(ok = wait_warp(bar(C::B_KF + st), (sidx / C::NST) & 1, ctl))) break;
                    uint8_t *v = smem + C::ST_OFF + st * C::TILE;
                    for (int c = tid; c < (vz1 - vz0) * 8 * C::DC; c += 128) {
                        const int r = vz0 + c / (8 * C::DC), q = c % (8 * C::DC);
                        *reinterpret_cast<uint4 *>(v + (q >> 3) * kRegion + r * 128 + (q & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                if (busy) {
                    tc_fence_after();
                    const bool full = all || __all_sync(kAllLanes, (w[0] & w[1]) == ~0ull || !row.valid);
                    float s[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, s[c]);
                    tmem_wait_ld();
                    if (!full) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t b = (uint32_t)(w[c >> 1] >> ((c & 1) * 32));
#pragma unroll
                            for (int k = 0; k < 32; ++k) s[c][k] = (b >> k) & 1u ? s[c][k] : -CUDART_INF_F;
                        }
                    }
                    float mx4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int k = 0; k < 32; k += 2)
#pragma unroll
                        for (int c = 0; c < 4; ++c) mx4[c] = fmax3(mx4[c], s[c][k], s[c][k + 1]);
                    float mx = fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]);
                    mx = row.valid ? mx * sl2 : -CUDART_INF_F;
                    const bool grow = mx > mref + kGrow || (mref == -CUDART_INF_F && mx > mref);
                    if (__any_sync(kAllLanes, grow)) {
                        const float ref = grow ? mx : mref;
                        const float f = grow ? ex2(mref - ref) : 1.f;  // 0 the first time
                        l *= f;
                        mref = ref;
                        if (had) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float o[32];
                                tmem_ld32(o_addr + c * 32, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] *= f;
                                tmem_st32(o_addr + c * 32, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float nref = mref == -CUDART_INF_F ? 0.f : -mref;
                    const uint64_t sl2x2 = f2_pack(sl2, sl2), nrefx2 = f2_pack(nref, nref);
                    uint64_t sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[32];
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int k = 0; k < 32; k += 2) {
                                float a, e;
                                f2_unpack(f2_fma(f2_pack(s[2 * h + c][k], s[2 * h + c][k + 1]), sl2x2, nrefx2), a, e);
                                a = ex2(a);
                                e = ex2(e);
                                if (k & 2) sum1 = f2_add(sum1, f2_pack(a, e));
                                else sum0 = f2_add(sum0, f2_pack(a, e));
                                const __nv_bfloat162 two = __floats2bfloat162_rn(a, e);
                                pk[c * 16 + k / 2] = *reinterpret_cast<const uint32_t *>(&two);
                            }
                        tmem_st32u(s_addr + h * 32, pk);
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::B_PF + 2 * x + h));
                    }
                    float a, e;
                    f2_unpack(f2_add(sum0, sum1), a, e);
                    l += a + e;
                } else if (lane == 0) {  // no row of this warp is used: let the others go on
                    mbar_arrive(bar(C::B_PF + 2 * x));
                    mbar_arrive(bar(C::B_PF + 2 * x + 1));
                }
                had = true;
            }
            if (!ok) break;
            // ---- epilogue
            // One-tile units: the second chain hands over its maximum and sum, and
            // the first chain's warps join both O's (they hold the same lanes).
            bool had2 = false;
            float f1 = 1.f, f2 = 0.f;
            if (one && n > 0) {
                float2 *ml = reinterpret_cast<float2 *>(smem + C::ML_OFF);
                if (x == 1) {
                    if (mc > 0 && !(ok = wait_warp(bar(C::B_ME), (mc - 1) & 1, ctl))) break;
                    ml[tid] = make_float2(had ? mref : -CUDART_INF_F, had ? l : -1.f);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_MF));
                    ++mc;
                    continue;
                }
                if (!(ok = wait_warp(bar(C::B_MF), mc & 1, ctl))) break;
                ++mc;
                const float2 other = ml[tid];
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_ME));
                had2 = other.y >= 0.f || other.y != other.y;  // -1: no step was its own
                if (had2) {
                    const float m = fmaxf(mref, other.x), ref = m == -CUDART_INF_F ? 0.f : m;
                    f1 = ex2(mref - ref);
                    f2 = ex2(other.x - ref);
                    l = l * f1 + other.y * f2;
                    mref = m;
                }
                had2 = __any_sync(kAllLanes, had2);
            } else if (one && x == 1) {
                continue;  // the first chain's warps write the zeros
            }
            if (had) {
                if (!(ok = wait_warp(bar(C::B_OF + x), oc & 1, ctl))) break;
                ++oc;
                tc_fence_after();
            }
            if (had2) {
                if (!(ok = wait_warp(bar(C::B_OF + 1), oc2 & 1, ctl))) break;
                ++oc2;
                tc_fence_after();
            }
            const int prow = x * half_rows + tid;  // row within the unit
            bool bad = false;
            const float inv = row.valid && l != 0.f ? 1.f / l : 0.f;
            if (busy || !had) {
                __nv_bfloat16 *orow = static_cast<__nv_bfloat16 *>(p.O) +
                                      (((size_t)U.b * p.Hq + head) * p.m + (t < p.m ? t : 0)) * D;
                const size_t at = (size_t)U.slot * p.rows + prow;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    if (had) {
                        tmem_ld32(o_addr + c * 32, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0.f;
                    }
                    if (had2) {
                        float o2[32];
                        tmem_ld32(o_addr + D + c * 32, o2);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = o[k] * f1 + o2[k] * f2;
                    }
                    float z = 0.f;
#pragma unroll
                    for (int k = 0; k < 32; ++k) z = fmaf(o[k], 0.f, z);  // NaN if any is infinite or NaN
                    bad |= z != 0.f;
                    if (!in || (!row.valid && t >= p.m)) continue;
                    if (U.split) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4 *>(p.part_o + at * D + c * 32 + k) =
                                make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t b4[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float a = row.valid ? o[q * 8 + 2 * k] * inv : 0.f;
                                const float e = row.valid ? o[q * 8 + 2 * k + 1] * inv : 0.f;
                                const __nv_bfloat162 two = __floats2bfloat162_rn(a, e);
                                b4[k] = *reinterpret_cast<const uint32_t *>(&two);
                            }
                            *reinterpret_cast<uint4 *>(orow + c * 32 + q * 8) = make_uint4(b4[0], b4[1], b4[2], b4[3]);
                        }
                    }
                }
                if (U.split && in) p.part_ml[at] = make_float2(row.valid ? mref : -CUDART_INF_F, row.valid ? l : 0.f);
            } else if (U.split && in) {  // no valid row in this warp: the merge writes their zeros
                p.part_ml[(size_t)U.slot * p.rows + prow] = make_float2(-CUDART_INF_F, 0.f);
            } else if (in && t < p.m) {
                uint4 *orow = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.O) +
                                                        (((size_t)U.b * p.Hq + head) * p.m + t) * D);
                for (int c = 0; c < D / 8; ++c) orow[c] = make_uint4(0u, 0u, 0u, 0u);
            }
            if (had || had2) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (had) mbar_arrive(bar(C::B_OE + x));
                    if (had2) mbar_arrive(bar(C::B_OE + 1));
                }
            }
            unsigned again = __ballot_sync(kAllLanes, row.valid && (had || had2) && (bad || not_finite(l)));
            while (again) {
                const int r = __ffs(again) - 1;
                again &= again - 1;
                const int rt = __shfl_sync(kAllLanes, t, r), rh = __shfl_sync(kAllLanes, head, r);
                float a[D / 32];
                __syncwarp();
                const float2 ml = exact_row<__nv_bfloat16, D>(p, P, U, rt, rh, a);
                store_exact_row<__nv_bfloat16, D>(p, U, rt, rh, x * half_rows + (warp & 3) * 32 + r, ml, a);
            }
        }
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp == 8 || warp == 11) {
        // ================================================================ K (8) and V (11) loaders
        const bool is_k = warp == 8;
        const CUtensorMap *tm = is_k ? &tmK : &tmV;
        const int log_bp = min(p.log_page, 6);  // tokens of a box: a page, at most 64
        const int log_ppb = 6 - log_bp;         // boxes per block and 64-column piece
        const int nbox = (2 << log_ppb) * C::DC;
        const bool big = p.page > 64;
        // this lane's box of a stage, before the lanes are moved on: a thread's
        // copies complete one after another, different threads' overlap
        uint32_t qc = 0, turn = 0;
        uint32_t armed = 0, phase = 0;  // per stage: filled by this warp, and the parity of the last time
        while (ok && units.next(p, P, U)) {
            const int n = (U.e1 - U.e0 + 1) >> 1;
            if (!U.live || n == 0) continue;
            if (is_k) {
                if (qc > 0 && !(ok = wait_warp(bar(C::B_QE), (qc - 1) & 1, ctl))) break;
                const int halves = !one && U.t0 + p.tpt_half < U.q ? 2 : 1;
                const int bytes = p.tpt_half * p.group * 128;
                if (lane == 0) mbar_arrive_expect_tx(bar(C::B_QF), (uint32_t)(halves * C::DC * bytes));
                __syncwarp();
                if (lane < halves * C::DC) {
                    const int x = lane / C::DC, dc = lane % C::DC;
                    tma_load_3d(sbase + C::Q_OFF + x * C::TILE + dc * kRegion, &tmQ, bar(C::B_QF), dc * 64,
                                U.t0 + x * p.tpt_half, U.b * p.Hq + U.hk * p.group);
                }
                ++qc;
            }
            // coordinates (y, z) of this lane's box in step i; z = -1 reads zeros
            auto look = [&](int i, int box, int &y) -> int {
                const int piece = box / C::DC, e = U.e0 + 2 * i + (piece >> log_ppb);
                y = 0;
                if (box >= nbox || i >= n || e >= U.e1) return -1;
                const int blk = entry_block(P, U, e);
                const int pos = (blk << 6) + ((piece & ((1 << log_ppb) - 1)) << log_bp);
                const int pg = pos < U.s ? page_of(p, U.b, pos) : -1;
                if (pg < 0) return -1;
                if (big) y = (blk & 1) * 64;
                return pg * p.Hkv + U.hk;
            };
            int y, z, box = (lane - (int)turn) & 31;
            z = look(0, box, y);
            for (int i = 0; i < n; ++i) {
                const uint32_t sidx = is_k ? k_at(g, i) : v_at(g, i, n), st = sidx % C::NST;
                turn = (turn + nbox) & 31;
                const int box1 = (lane - (int)turn) & 31;
                int y1;
                const int z1 = look(i + 1, box1, y1);  // on its way during this step's wait
                if (sidx >= C::NST && !(ok = wait_warp(bar(C::B_KE + st), ((sidx / C::NST) - 1) & 1, ctl))) break;
                if (lane == 0) mbar_arrive_expect_tx(bar(C::B_KF + st), C::TILE);
                __syncwarp();
                if (box < nbox)
                    tma_load_3d(sbase + C::ST_OFF + st * C::TILE + (box % C::DC) * kRegion +
                                    ((box / C::DC) << log_bp) * 128,
                                tm, bar(C::B_KF + st), (box % C::DC) * 64, y, z);
                armed |= 1u << st;
                phase = (phase & ~(1u << st)) | (((sidx / C::NST) & 1u) << st);
                box = box1;
                y = y1;
                z = z1;
            }
            g += n;
        }
        if (!ok) {  // abort: wait for this warp's copies still in flight
            for (int i = 0; i < C::NST; ++i)
                if ((armed >> i) & 1u) wait_drain(bar(C::B_KF + i), (phase >> i) & 1u);
            if (is_k && qc) wait_drain(bar(C::B_QF), (qc - 1) & 1);
        }
    } else if (warp == 10) {
        // ================================================================ step records
        // What each step holds for the tiles, ahead of their use. Lane l looks
        // up piece l % ppb of entry l / ppb.
        const int log_bp = min(p.log_page, 6), log_ppb = 6 - log_bp, ppb = 1 << log_ppb;
        while (ok && units.next(p, P, U)) {
            const int n = (U.e1 - U.e0 + 1) >> 1;
            if (!U.live || n == 0) continue;
            const int stride = p.dilation ? P.hstride[U.hk] : 1;
            const TileSpan sp0 = tile_span(p, P, U, 0, stride), sp1 = tile_span(p, P, U, 1, stride);
            auto look = [&](int i, int &blk) -> int {
                const int e = U.e0 + 2 * i + (lane >> log_ppb);
                blk = -1;
                if (lane >= 2 * ppb || e >= U.e1) return -1;
                blk = entry_block(P, U, e);
                const int pos = (blk << 6) + ((lane & (ppb - 1)) << log_bp);
                return pos < U.s ? page_of(p, U.b, pos) : -1;
            };
            int blk, pg = look(0, blk);
            for (int i = 0; i < n; ++i, ++g) {
                const uint32_t slot = g % kSI;
                int nblk = -1, npg = -1;
                if (i + 1 < n) npg = look(i + 1, nblk);
                // lanes 0 and 1 each do one of the step's two blocks
                const unsigned there = __ballot_sync(kAllLanes, pg >= 0) >> ((lane & 1) << log_ppb);
                const int b = __shfl_sync(kAllLanes, blk, (lane & 1) << log_ppb);
                uint64_t w = 0ull;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (s < ppb && ((there >> s) & 1u)) w |= low_bits(1 << log_bp) << (s << log_bp);
                const uint64_t gb = b < 0 ? 0ull : global_bits(P, p, b);
                const int j0 = b << 6;
                int use = 0, written = 64;
                if (b >= 0) {
                    if (sp0.live && j0 <= sp0.p1 && (j0 + 63 >= sp0.first || gb)) use |= 1;
                    if (sp1.live && j0 <= sp1.p1 && (j0 + 63 >= sp1.first || gb)) use |= 2;
                    written = max(min(U.s - j0, 64), 0);  // keys of the block that hold tokens
                }
                const bool whole = stride == 1 && w == ~0ull;
                int all = 0;
                if (whole && j0 + 63 <= sp0.p0 && j0 >= sp0.last) all |= 4;
                if (whole && j0 + 63 <= sp1.p0 && j0 >= sp1.last) all |= 8;
                const int use2 = use | __shfl_xor_sync(kAllLanes, use, 1);
                const int all2 = all & __shfl_xor_sync(kAllLanes, all, 1);
                const int written2 = __shfl_xor_sync(kAllLanes, written, 1);
                if (g >= kSI && !(ok = wait_warp(bar(C::B_IE + slot), ((g / kSI) - 1) & 1, ctl))) break;
                if (lane < 2) {
                    StepRec &r = recs[slot];
                    r.blk[lane] = b;
                    r.gbits[lane] = gb;
                    r.present[lane] = w;
                    if (lane == 0) {
                        r.use = one ? ((use2 & 1) << (i & 1)) | ((all2 & 4) ? 12 : 0) : use2 | all2;
                        // only the last block of a sequence holds unwritten keys
                        r.vz0 = written < 64 ? written : 64 + written2;
                        r.vz1 = written < 64 ? 64 : 128;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_IF + slot));
                blk = nblk;
                pg = npg;
            }
        }
    } else if (warp == 9) {
        // ================================================================ MMA issuer
        constexpr uint32_t idesc_qk = idesc_bf16(128, 128, false);
        constexpr uint32_t idesc_pv = idesc_bf16(128, D, true);
        // The whole warp runs the loop and the waits, so descriptors and TMEM
        // addresses stay warp-uniform; one elected lane issues the MMAs and the
        // commits that track them.
        const bool leader = elect_one();
        const uint64_t dQ0 = desc_sw128(sbase + C::Q_OFF, 16);
        const uint64_t dK0 = desc_sw128(sbase + C::ST_OFF, 16);
        const uint64_t dV0 = desc_sw128(sbase + C::ST_OFF, kRegion);
        uint32_t qc = 0, pc[2] = {0, 0}, oc[2] = {0, 0};
        auto filled = [&](uint32_t sidx) {
            return wait_warp(bar(C::B_KF + sidx % C::NST), (sidx / C::NST) & 1, ctl);
        };
        // tiles that use step gs; waits for its record
        auto step_use = [&](uint32_t gs, int &use) -> bool {
            const uint32_t slot = gs % kSI;
            if (!wait_warp(bar(C::B_IF + slot), (gs / kSI) & 1, ctl)) return false;
            use = recs[slot].use & 3;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_IE + slot));
            return true;
        };
        while (ok && units.next(p, P, U)) {
            const int n = (U.e1 - U.e0 + 1) >> 1;
            if (!U.live || n == 0) continue;
            int use = 0, next_use = 0;
            if (!(ok = step_use(g, next_use))) break;
            if (!(ok = wait_warp(bar(C::B_QF), qc & 1, ctl))) break;
            ++qc;
            const uint32_t g0 = g;
            int prev = 0;        // tiles whose P of the step before is to be used
            int started = 0;     // tiles with a product in O already
            // S_X = Q_X K^T with the K of ring position kx
            auto scores = [&](auto X, uint32_t kx) {
                constexpr int x = decltype(X)::value;
                tc_fence_after();
                if (leader) {
                    const uint64_t dQ = one ? dQ0 : dQ0 + (uint64_t)((x * C::TILE) >> 4);
                    const uint64_t dK = dK0 + (uint64_t)(((kx % C::NST) * C::TILE) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t off = (uint64_t)(((kk >> 2) * kRegion + (kk & 3) * 32) >> 4);
                        mma_bf16_ss(tmem + x * 128, dQ + off, dK + off, idesc_qk, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(bar(C::B_SF + x));
                }
                __syncwarp();
            };
            // O_X (+)= P_X V with the V of ring position vx: 64 keys as soon as their weights are there
            auto weigh = [&](auto X, uint32_t vx) -> bool {
                constexpr int x = decltype(X)::value;
                const bool first = !((started >> x) & 1);
                if (first && oc[x] > 0 && !wait_warp(bar(C::B_OE + x), (oc[x] - 1) & 1, ctl)) return false;
                const uint64_t dV = dV0 + (uint64_t)(((vx % C::NST) * C::TILE) >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!wait_warp(bar(C::B_PF + 2 * x + h), pc[x] & 1, ctl)) return false;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                            mma_bf16_ts(tmem + C::O_COL + x * D, tmem + x * 128 + kk * 8,
                                        dV + (uint64_t)((kk * 2048) >> 4), idesc_pv, (first && kk == 0) ? 0u : 1u);
                    }
                    __syncwarp();
                }
                ++pc[x];
                started |= 1 << x;
                return true;
            };
            auto release = [&](uint32_t sidx) {
                if (leader) mma_commit(bar(C::B_KE + sidx % C::NST));
                __syncwarp();
            };
            const std::integral_constant<int, 0> T0{};
            const std::integral_constant<int, 1> T1{};
            for (int i = 0; i <= n; ++i) {
                use = i < n ? next_use : 0;
                const uint32_t kx = k_at(g0, i), vx = i > 0 ? v_at(g0, i - 1, n) : 0;
                if (one) {  // the chains take turns: this step's scores need not wait for the other's weights
                    if (i < n) {
                        if (!(ok = filled(kx))) break;
                        if (use & 1) scores(T0, kx);
                        if (use & 2) scores(T1, kx);
                        release(kx);
                    }
                    if (i + 1 < n && !(ok = step_use(g + 1, next_use))) break;
                    if (i > 0) {
                        if (!(ok = filled(vx))) break;
                        if ((prev & 1) && !(ok = weigh(T0, vx))) break;
                        if ((prev & 2) && !(ok = weigh(T1, vx))) break;
                        release(vx);
                    }
                } else {
                    if (i < n && !(ok = filled(kx))) break;
                    if (i > 0 && !(ok = filled(vx))) break;
                    if ((prev & 1) && !(ok = weigh(T0, vx))) break;
                    if (use & 1) scores(T0, kx);
                    // while the other tile's softmax works: the next step's record
                    if (i + 1 < n && !(ok = step_use(g + 1, next_use))) break;
                    if ((prev & 2) && !(ok = weigh(T1, vx))) break;
                    if (use & 2) scores(T1, kx);
                    if (i > 0) release(vx);
                    if (i < n) release(kx);
                }
                if (leader) {
                    if (i == n - 1) mma_commit(bar(C::B_QE));
                    if (i == n) {
                        if (started & 1) mma_commit(bar(C::B_OF + 0));
                        if (started & 2) mma_commit(bar(C::B_OF + 1));
                    }
                }
                __syncwarp();
                prev = use;
                if (i < n) ++g;
            }
            oc[0] += started & 1;
            oc[1] += (started >> 1) & 1;
        }
        // every MMA issued has completed once this arrives
        if (leader) mma_commit(bar(C::B_DRAIN));
        __syncwarp();
        wait_drain(bar(C::B_DRAIN), 0);
    }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(ptr);
        return nullptr;
    }();
    return fn;
}

// {d, rows, slices} bf16, boxes of 64 columns x box_rows x box_slices, 128-byte swizzle.
bool make_map(CUtensorMap *m, const void *base, int d, int rows, long long slices, int box_rows, int box_slices) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)slices};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)rows * d * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_slices};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_tc_d(const PagedProblem &p, cudaStream_t stream) {
    using C = TcCfg<D>;
    const size_t smem = C::PLAN_OFF + plan_bytes(p.B, p.ng, p.Hkv) + 1024;
    if (smem > 232448) return cudaErrorNotSupported;
    CUtensorMap mq, mk, mv;
    const int bp = p.page < 64 ? p.page : 64;
    if (!make_map(&mq, p.Q, D, p.m, (long long)p.B * p.Hq, p.tpt_half, p.group) ||
        !make_map(&mk, p.K, D, p.page, (long long)p.num_pages * p.Hkv, bp, 1) ||
        !make_map(&mv, p.V, D, p.page, (long long)p.num_pages * p.Hkv, bp, 1))
        return cudaErrorInvalidValue;
    auto kern = paged_tc<D>;
    static std::atomic<bool> done[64];
    cudaError_t e = allow_smem(kern, done, smem);
    if (e != cudaSuccess) return e;
    kern<<<p.slots, kTcThreads, smem, stream>>>(mq, mk, mv, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tc(const PagedProblem &p, cudaStream_t stream) {
    return p.d == 64 ? launch_tc_d<64>(p, stream) : launch_tc_d<128>(p, stream);
}

static_assert(TcCfg<128>::PLAN_OFF + 1024 + (2 * kPagedMaxBatch + 2 * kPagedMaxGlobal + kPagedMaxHeads + 2) * 4 + 16 +
                      (kPagedMaxBatch + 1 + kPagedMaxGlobal) * 8 <= 232448,
              "the largest plan fits beside the tiles");

}  // namespace sa
