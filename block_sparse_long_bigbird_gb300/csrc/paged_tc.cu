// Attention of many new tokens over a paged cache on the tensor cores (bf16):
// chunks of a prompt, drafts, and single tokens whose query heads share a key
// head.
//
// A unit's query rows (tokens x the query heads of one key head, up to 2 x 128)
// are two MMA tiles of 128 rows that share every key and value they load: a
// 128-key stage serves 2 x 128 x 128 products, which halves the L2 traffic per
// flop, and one tile's softmax overlaps the other's MMAs.
//   * The producer warp walks the unit's 64-key blocks two at a time, looks the
//     pages up (a step ahead), and loads K and V with one tensor copy per page
//     piece: the pool is {d, page, num_pages * Hkv}, a box is 64 columns of one
//     page (at most 64 tokens). A missing page is loaded from coordinate -1,
//     which fills with zeros, so stages always fill.
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

#include "paged_common.cuh"
#include "tc_sync.cuh"

namespace sa {
namespace {

using namespace ptx;
using namespace tcsync;

constexpr int kTcThreads = 384;  // 8 softmax warps, producer, MMA, two spare (register budget of warpgroups)
constexpr int kRegion = 128 * 128;  // 128 rows x 128 B: one 64-column piece of a tile
constexpr float kGrow = 8.0f;       // growth of the maximum (log2) that rescales O
constexpr int kSI = 4;              // step records in flight

struct StepRec {
    int blk[2];          // 64-key blocks (-1: none)
    int use;             // bit x: tile x has a row that sees something here
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
                         B_QE = B_QF + 1, B_SF = B_QE + 1, B_PF = B_SF + 2, B_OF = B_PF + 2, B_OE = B_OF + 2,
                         B_MF = B_OE + 2, B_ME = B_MF + 1, B_DRAIN = B_ME + 1, B_COUNT = B_DRAIN + 1;
    static constexpr int REC_OFF = (BAR_OFF + B_COUNT * 8 + 15) & ~15;
    static constexpr int MISC_OFF = REC_OFF + kSI * (int)sizeof(StepRec);
    static constexpr int ML_OFF = MISC_OFF + 16;       // one-tile units: the second chain's (maximum, sum) per row
    static constexpr int PLAN_OFF = ML_OFF + 128 * 8;
    static constexpr uint32_t O_COL = 256;
};
static_assert(sizeof(StepRec) == 56 && (kSI * sizeof(StepRec)) % 16 == 0, "step record layout");

// Last token of tile x of a unit, its first visible position, and whether it has rows at all.
struct TileSpan {
    int p1, first;
    bool live;
};

__device__ __forceinline__ TileSpan tile_span(const PagedProblem &p, const Plan &P, const Unit &U, int x, int stride) {
    TileSpan s;
    const int t0 = U.t0 + x * p.tpt_half;
    s.live = U.live && t0 < U.q && (x == 0 || p.tpt > p.tpt_half);
    const int p0 = U.s - U.q + t0;
    s.p1 = U.s - U.q + min(t0 + p.tpt_half, U.q) - 1;
    s.first = max(0, p0 - head_reach(p, stride));
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
            mbar_init(bar(C::B_PF + x), 4);
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
    Plan P = plan_at(smem + C::PLAN_OFF, p.B, p.ng);
    tc_fence_before();
    make_plan(p, P);
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int total = P.ubase[p.B];
    uint32_t g = 0;   // steps so far; every role counts the same ones
    bool ok = true;
    const bool one = p.tpt == p.tpt_half;  // units of one tile: its steps alternate between two chains

    // The launch gave every thread 168 registers (384 x 168 = 64512); the
    // softmax holds a row of scores, so its 8 warps take 200 and the others 104
    // (256 x 200 + 128 x 104 = 64512).
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ================================================================ softmax and epilogue of tile x
        const int x = warp >> 2;
        const int tid = threadIdx.x & 127;  // row of the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + x * 128, o_addr = tmem + lane_base + C::O_COL + x * D;
        const int half_rows = p.tpt_half * p.group;
        const float sl2 = p.scale_log2;
        uint32_t sc = 0, oc = 0, oc2 = 0, mc = 0;
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
            const Unit U = decode_unit(p, P, u);
            const int n = U.live ? (U.e1 - U.e0 + 1) >> 1 : 0;
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
                uint64_t w[2] = {0ull, 0ull};
                if (((use >> x) & 1) && row.valid) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (recs[slot].blk[k] >= 0)
                            w[k] = row_mask(row, recs[slot].blk[k], recs[slot].gbits[k], recs[slot].present[k]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_IE + slot));
                if (!((use >> x) & 1)) continue;
                if (vz0 < vz1) {  // unwritten memory: no NaN may meet a zero weight
                    const uint32_t sidx = 2 * g + 1, st = sidx % C::NST;
                    if (!(ok = wait_warp(bar(C::B_KF + st), (sidx / C::NST) & 1, ctl))) break;
                    uint8_t *v = smem + C::ST_OFF + st * C::TILE;
                    for (int c = tid; c < (vz1 - vz0) * 8 * C::DC; c += 128) {
                        const int r = vz0 + c / (8 * C::DC), q = c % (8 * C::DC);
                        *reinterpret_cast<uint4 *>(v + (q >> 3) * kRegion + r * 128 + (q & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                if (!(ok = wait_warp(bar(C::B_SF + x), sc & 1, ctl))) break;
                ++sc;
                if (busy) {
                    tc_fence_after();
                    const bool full = __all_sync(kAllLanes, (w[0] & w[1]) == ~0ull || !row.valid);
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
                    }
                    float a, e;
                    f2_unpack(f2_add(sum0, sum1), a, e);
                    l += a + e;
                    tmem_wait_st();
                    tc_fence_before();
                }
                had = true;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_PF + x));
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
                    if (U.ns > 1) {
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
                if (U.ns > 1 && in) p.part_ml[at] = make_float2(row.valid ? mref : -CUDART_INF_F, row.valid ? l : 0.f);
            } else if (U.ns > 1 && in) {  // no valid row in this warp: the merge writes their zeros
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8) {
        // ================================================================ producer
        const int bp = min(p.page, 64);      // tokens of a box
        const int log_bp = min(p.log_page, 6);
        const int ppb = 64 >> log_bp;        // boxes per block and piece
        const int log_ppb = 6 - log_bp;
        const int nbox = 2 * ppb * C::DC;    // per K or V stage
        const uint64_t sub_bits = low_bits(bp);
        uint32_t qc = 0, armed = 0;
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
            const Unit U = decode_unit(p, P, u);
            const int n = (U.e1 - U.e0 + 1) >> 1;
            if (!U.live || n == 0) continue;
            int stride = 1;
            if (p.dilation)
                for (int h = 0; h < p.group; ++h) stride = max(stride, head_stride(p, U.hk * p.group + h));
            const TileSpan sp0 = tile_span(p, P, U, 0, stride), sp1 = tile_span(p, P, U, 1, stride);
            // this lane's page of step i: entry lane / ppb of the step, piece lane % ppb
            auto look = [&](int i, int &blk) -> int {
                const int e = U.e0 + 2 * i + (lane >> log_ppb);
                blk = -1;
                if (lane >= 2 * ppb || e >= U.e1) return -1;
                blk = entry_block(P, U, e);
                const int pos = (blk << 6) + ((lane & (ppb - 1)) << log_bp);
                return pos < U.s ? page_of(p, U.b, pos) : -1;
            };
            int blk, pg = look(0, blk);
            if (qc > 0 && !(ok = wait_warp(bar(C::B_QE), (qc - 1) & 1, ctl))) break;
            {
                const int halves = sp1.live ? 2 : 1;
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
            for (int i = 0; i < n; ++i, ++g) {
                const uint32_t slot = g % kSI;
                int nblk = -1, npg = -1;
                if (i + 1 < n) npg = look(i + 1, nblk);  // on its way during this step's waits
                // the step's record: every lane computes it, lane 0 stores it
                StepRec r;
                const unsigned there = __ballot_sync(kAllLanes, pg >= 0);
                r.use = 0;
                r.vz0 = r.vz1 = 0;
                r.pad = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int b = __shfl_sync(kAllLanes, blk, k << log_ppb);
                    r.blk[k] = b;
                    r.gbits[k] = b < 0 ? 0ull : global_bits(P, p, b);
                    uint64_t w = 0ull;
                    for (int s = 0; s < ppb; ++s)
                        if ((there >> ((k << log_ppb) + s)) & 1u) w |= sub_bits << (s << log_bp);
                    r.present[k] = w;
                    if (b < 0) continue;
                    const int j0 = b << 6;
                    if (sp0.live && j0 <= sp0.p1 && (j0 + 63 >= sp0.first || r.gbits[k])) r.use |= 1;
                    if (sp1.live && j0 <= sp1.p1 && (j0 + 63 >= sp1.first || r.gbits[k])) r.use |= 2;
                    const int written = U.s - j0;  // keys of the block that hold tokens
                    if (written < 64) {
                        r.vz0 = k * 64 + max(written, 0);
                        r.vz1 = k * 64 + 64;
                    }
                }
                if (one) r.use = (r.use & 1) << (i & 1);
                if (g >= kSI && !(ok = wait_warp(bar(C::B_IE + slot), ((g / kSI) - 1) & 1, ctl))) break;
                if (lane == 0) {
                    recs[slot] = r;
                    mbar_arrive(bar(C::B_IF + slot));
                }
                __syncwarp();
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t sidx = 2 * g + kv, st = sidx % C::NST;
                    if (sidx >= C::NST && !(ok = wait_warp(bar(C::B_KE + st), ((sidx / C::NST) - 1) & 1, ctl))) break;
                    if (lane == 0) mbar_arrive_expect_tx(bar(C::B_KF + st), C::TILE);
                    __syncwarp();
                    ++armed;
                    // box index of this lane, moved on every stage: a thread's
                    // copies complete one after another, different threads' overlap
                    const int box = (lane - (int)((sidx * (uint32_t)nbox) & 31u)) & 31;
                    const int piece = box / C::DC, dc = box % C::DC;
                    const int from = box < nbox ? piece : 0;
                    const int bpg = __shfl_sync(kAllLanes, pg, from), bblk = __shfl_sync(kAllLanes, blk, from);
                    if (box < nbox) {
                        const int y = p.page > 64 ? (bblk & 1) * 64 : 0;
                        const int z = bpg < 0 ? -1 : bpg * p.Hkv + U.hk;
                        tma_load_3d(sbase + C::ST_OFF + st * C::TILE + dc * kRegion + (piece << log_bp) * 128,
                                    kv ? &tmV : &tmK, bar(C::B_KF + st), dc * 64, z < 0 ? 0 : y, z);
                    }
                }
                if (!ok) break;
                blk = nblk;
                pg = npg;
            }
        }
        if (!ok) {  // abort: wait for the copies still in flight
            for (uint32_t i = 0; i < (uint32_t)C::NST && i < armed; ++i)
                wait_drain(bar(C::B_KF + i), ((armed - 1 - i) / C::NST) & 1);
            if (qc) wait_drain(bar(C::B_QF), (qc - 1) & 1);
        }
    } else if (warp == 9) {
        // ================================================================ MMA issuer
        constexpr uint32_t idesc_qk = idesc_bf16(128, 128, false);
        constexpr uint32_t idesc_pv = idesc_bf16(128, D, true);
        const bool leader = elect_one();
        const uint64_t dQ0 = desc_sw128(sbase + C::Q_OFF, 16);
        const uint64_t dK0 = desc_sw128(sbase + C::ST_OFF, 16);
        const uint64_t dV0 = desc_sw128(sbase + C::ST_OFF, kRegion);
        uint32_t qc = 0, pc[2] = {0, 0}, oc[2] = {0, 0};
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
            const Unit U = decode_unit(p, P, u);
            const int n = (U.e1 - U.e0 + 1) >> 1;
            if (!U.live || n == 0) continue;
            if (!(ok = wait_warp(bar(C::B_QF), qc & 1, ctl))) break;
            ++qc;
            int prev = 0;        // tiles whose P of the step before is to be used
            int started = 0;     // tiles with a product in O already
            for (int i = 0; i <= n; ++i) {
                int use = 0;
                const uint32_t sk = (2 * g) % C::NST, sv = (2 * g - 1) % C::NST;  // K of step g, V of step g - 1
                if (i < n) {
                    const uint32_t slot = g % kSI;
                    if (!(ok = wait_warp(bar(C::B_IF + slot), (g / kSI) & 1, ctl))) break;
                    use = recs[slot].use;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_IE + slot));
                    if (!(ok = wait_warp(bar(C::B_KF + sk), ((2 * g) / C::NST) & 1, ctl))) break;
                }
                if (i > 0 && !(ok = wait_warp(bar(C::B_KF + sv), ((2 * g - 1) / C::NST) & 1, ctl))) break;
                auto scores = [&](int x) {
                    tc_fence_after();
                    if (leader) {
                        const uint64_t dQ = dQ0 + (uint64_t)(((one ? 0 : x) * C::TILE) >> 4);
                        const uint64_t dK = dK0 + (uint64_t)((sk * C::TILE) >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t off = (uint64_t)(((kk >> 2) * kRegion + (kk & 3) * 32) >> 4);
                            mma_bf16_ss(tmem + x * 128, dQ + off, dK + off, idesc_qk, kk > 0 ? 1u : 0u);
                        }
                        mma_commit(bar(C::B_SF + x));
                    }
                    __syncwarp();
                };
                // chains that do not follow on themselves need not wait for the other's weights
                const bool early = (prev & use) == 0;
                if (early) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        if ((use >> x) & 1) scores(x);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if ((prev >> x) & 1) {
                        if (!(ok = wait_warp(bar(C::B_PF + x), pc[x] & 1, ctl))) break;
                        ++pc[x];
                        const bool first = !((started >> x) & 1);
                        if (first && oc[x] > 0 && !(ok = wait_warp(bar(C::B_OE + x), (oc[x] - 1) & 1, ctl))) break;
                        tc_fence_after();
                        if (leader) {
                            const uint64_t dV = dV0 + (uint64_t)((sv * C::TILE) >> 4);
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                mma_bf16_ts(tmem + C::O_COL + x * D, tmem + x * 128 + kk * 8,
                                            dV + (uint64_t)((kk * 2048) >> 4), idesc_pv, (first && kk == 0) ? 0u : 1u);
                        }
                        __syncwarp();
                        started |= 1 << x;
                    }
                    if (!early && ((use >> x) & 1)) scores(x);
                }
                if (!ok) break;
                if (leader) {
                    if (i > 0) mma_commit(bar(C::B_KE + sv));
                    if (i < n) mma_commit(bar(C::B_KE + sk));
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
    const size_t smem = C::PLAN_OFF + plan_bytes(p.B, p.ng) + 1024;
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
    const long long units = (long long)p.B * p.Hkv * ((p.m + p.tpt - 1) / p.tpt) + (p.cut ? p.max_parts : 0);
    kern<<<(int)(units < p.slots ? units : p.slots), kTcThreads, smem, stream>>>(mq, mk, mv, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tc(const PagedProblem &p, cudaStream_t stream) {
    return p.d == 64 ? launch_tc_d<64>(p, stream) : launch_tc_d<128>(p, stream);
}

static_assert(TcCfg<128>::PLAN_OFF + 1024 + ((5 * kPagedMaxBatch + 2 * kPagedMaxGlobal + 6 + kCuts) * 4 + 16) +
                      kPagedMaxGlobal * 8 <= 232448,
              "the largest plan fits beside the tiles");

}  // namespace sa
