// Attention of many new tokens over a paged cache on the tensor cores (bf16):
// chunks of a prompt, and whatever gives a key head more than 24 query rows.
//
//     O_r = sum_j w_rj V_j / sum_j w_rj,   w_rj = 2^(s_rj - m_r),   s = q . k log2(e) / sqrt(d)
//
// A unit's query rows (tokens x the query heads of one key head, up to 2 x 128)
// are two MMA tiles of 128 rows that share every key and value they load: a
// 128-key stage serves 2 x 128 x 128 products, which halves the L2 traffic per
// flop, and one tile's softmax overlaps the other's MMAs.
//   * The loader warp walks the unit's 64-key blocks two at a time, looks the
//     pages up (a step ahead), and loads K and V with one tensor copy per page
//     piece; another warp writes down what each step holds for the
//     two tiles. The pool is {d, page, num_pages * Hkv}, a box is 64 columns of
//     one page (at most 64 tokens). A missing page is loaded from coordinate
//     -1, which fills with zeros, so stages always fill.
//   * An MMA warp per tile runs S_x = Q_x K^T into two slots of 64 TMEM columns,
//     a half step each, and O_x += P_x V with P_x read from TMEM, where the
//     softmax wrote it (bf16) over its S slot. One thread issues a tile's MMAs,
//     so they complete in order. While the softmax works on one half, the MMAs
//     use the other's weights and fill its slot again: with one slot of 128
//     columns both waited for each other (a step of two tiles took 3700 clocks
//     at d = 64, of which the MMAs need 1024).
//   * A warpgroup per tile runs the softmax, one thread per row: masks, running
//     maximum (kept until it grows by more than 2^8, then O is rescaled in
//     place), weights and their sum in fp32, P rounded to bf16 (relative 2^-8,
//     the rounding the dense path of this library makes too).
// Memory where no token was written may hold NaN: those V rows are zeroed in
// shared memory before the product. Any other masked infinity or NaN makes its
// row's O not finite; the softmax warps take such rows again (rows_again) when
// the CTA is through with its units.
// Roles' waits are bounded; on expiry the CTA latches SA_ERR_TIMEOUT, drains
// its copies and MMAs, frees TMEM and exits.
//
// Measured: 4096 tokens at the end of 32768 keys, 16 query and 4 key heads, d =
// 128: 826 us, 1250 TFLOP/s (0.63 of the measured bf16 rate); with as many key as
// query heads, 2 x 2048 tokens over 16384 keys: d = 128 444 us, 1160 TFLOP/s, d = 64
// 423 us, 610 TFLOP/s. A 64-key block of two tiles takes 1.0 us whatever d is: the
// softmax bounds it (16384 exponentials per block, one thread per row), not the
// tensor pipe (47% busy at d = 128) or the memory (3%). A window of 512, 4 x 4096
// tokens, 12 heads, d = 64: 66 us; a unit of ten blocks takes 18400 clocks there: 2800 to
// start (record, rows, first scores), 10500 in its steps, 2000 for the last product
// and 3100 to write O. Units of one tile that see little pay more: the first chain's
// warps join both O's and write them (2300 to 6000 clocks). Loading their next
// queries ahead, into the place of the second tile, changed nothing.
#include <cuda.h>

#include <type_traits>

#include "paged_common.cuh"
#include "tc_sync.cuh"

namespace sa {
namespace {

using namespace ptx;
using namespace tcsync;

constexpr int kTcThreads = 384;  // 8 softmax warps, loader, two MMA issuers, step records
constexpr int kRegion = 128 * 128;  // 128 rows x 128 B: one 64-column piece of a tile
constexpr float kGrow = 8.0f;       // growth of the maximum (log2) that rescales O
constexpr int kSI = 4;              // step records in flight
constexpr int kNU = 4;              // units in flight

constexpr int kNowhere = 0x40000200;  // past every position

struct UnitRec {
    Unit U;
    int n;      // steps
    int end;    // nonzero: there is no further unit
};

struct StepRec {
    int j0[2];           // first keys of the two 64-key blocks (kNowhere: none)
    int use;             // bit x: tile x has a row that sees something here; 2 + x: all its rows see every key;
                         // 4: every row sees an interval of the keys and no others
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
                         B_QE = B_QF + 1, B_SF = B_QE + 1, B_PF = B_SF + 4, B_PD = B_PF + 4, B_OF = B_PD + 2, B_OE = B_OF + 2,
                         B_MF = B_OE + 2, B_ME = B_MF + 1, B_UF = B_ME + 1, B_UE = B_UF + kNU, B_DRAIN = B_UE + kNU, B_COUNT = B_DRAIN + 2;
    static constexpr int REC_OFF = (BAR_OFF + B_COUNT * 8 + 15) & ~15;
    static constexpr int UNIT_OFF = REC_OFF + kSI * (int)sizeof(StepRec);
    static constexpr int MISC_OFF = UNIT_OFF + kNU * (int)sizeof(UnitRec);
    static constexpr int ML_OFF = MISC_OFF + 16;       // one-tile units: the second chain's (maximum, sum) per row
    static constexpr int PLAN_OFF = ML_OFF + 128 * 8;
    static constexpr uint32_t O_COL = 256;
};
static_assert((kSI * sizeof(StepRec)) % 16 == 0 && (kNU * sizeof(UnitRec)) % 16 == 0, "record layout");

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

// `n` bits from bit `at` on (both clamped to 32).
__device__ __forceinline__ uint32_t bit_run(int at, int n) {
    uint32_t m;
    asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(at), "r"(n));
    return m;
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
    volatile int *again = abort_flag + 1;  // whether a row is to be taken again
    StepRec *recs = reinterpret_cast<StepRec *>(smem + C::REC_OFF);
    UnitRec *unit_recs = reinterpret_cast<UnitRec *>(smem + C::UNIT_OFF);
    auto bar = [&](int i) { return sbase + C::BAR_OFF + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Ctl ctl{abort_flag, p.status, p.wait_ns};
    const bool one = p.tpt == p.tpt_half;  // units of one tile: its steps alternate between two chains

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *again = 0;
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(bar(C::B_KF + i), 1);
            mbar_init(bar(C::B_KE + i), one ? 1 : 2);  // the MMA warps that read the stage
        }
        for (int i = 0; i < kSI; ++i) {
            mbar_init(bar(C::B_IF + i), 1);
            mbar_init(bar(C::B_IE + i), one ? 8 : 10);  // 8 softmax warps, with two tiles the MMA warps too
        }
        for (int i = 0; i < kNU; ++i) {
            mbar_init(bar(C::B_UF + i), 1);
            mbar_init(bar(C::B_UE + i), 11);  // all warps but the one that writes them
        }
        mbar_init(bar(C::B_QF), 1);
        mbar_init(bar(C::B_QE), 2);
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(C::B_SF + 2 * x), 1);
            mbar_init(bar(C::B_SF + 2 * x + 1), 1);
            mbar_init(bar(C::B_PD + x), 1);
            mbar_init(bar(C::B_PF + 2 * x), 4);
            mbar_init(bar(C::B_PF + 2 * x + 1), 4);
            mbar_init(bar(C::B_OF + x), 1);
            mbar_init(bar(C::B_OE + x), 4);
        }
        mbar_init(bar(C::B_MF), 4);
        mbar_init(bar(C::B_ME), 4);
        mbar_init(bar(C::B_DRAIN), 1);
        mbar_init(bar(C::B_DRAIN + 1), 1);
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
    make_plan(p, P);
    // The mbarriers and the TMEM address above are every warp's from here on,
    // also on calls that need no plan (make_plan has no barrier there).
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    asm volatile("griddepcontrol.launch_dependents;");  // the join may start planning
    uint32_t g = 0;   // steps so far; every role counts the same ones
    bool ok = true;
    uint32_t uc = 0;  // units so far
    // The following unit's record; `done` once there is none.
    bool done = false;
    auto next_unit = [&]() -> const UnitRec & {
        const uint32_t slot = uc % kNU;
        ok = wait_warp(bar(C::B_UF + slot), (uc / kNU) & 1, ctl);
        ++uc;
        done = !ok || unit_recs[slot].end;
        return unit_recs[slot];
    };
    auto unit_done = [&]() {  // this warp has no more use for the unit's record
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_UE + (uc - 1) % kNU));
    };
    // Stage of step i's K (kv = 0) or V (1) in the unit that begins at step g,
    // and the number of times that it has been filled before. Two tiles use one
    // ring of all stages; two chains of one tile have a ring each, since a
    // chain that ran ahead on a shared ring could take the parity of a stage
    // that the other's data has yet to fill for that of its own.
    // (h0, h1: steps of the two chains so far.)
    uint32_t h0 = 0, h1 = 0;
    struct Pos {
        uint32_t st, times;
    };
    auto stage = [&](int i, int kv) -> Pos {
        if (!one) {
            const uint32_t n = 2 * (g + (uint32_t)i) + (uint32_t)kv;
            return {n % C::NST, n / C::NST};
        }
        const uint32_t n = 2 * ((i & 1 ? h1 : h0) + (uint32_t)(i >> 1)) + (uint32_t)kv;
        return {(i & 1 ? C::NST / 2 : 0) + n % (C::NST / 2), n / (C::NST / 2)};
    };
    auto unit_steps = [&](int n) {  // past a unit of n steps
        g += (uint32_t)n;
        h0 += (uint32_t)(n + 1) >> 1;
        h1 += (uint32_t)n >> 1;
    };

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
        const int my_g = tid / p.tpt_half, my_t = tid - my_g * p.tpt_half + (one ? 0 : x * p.tpt_half);
        const bool in = tid < half_rows;
        uint32_t sc = 0, oc = 0, oc2 = 0, mc = 0;
        uint32_t handed = 0;  // halves whose weights were handed over
        while (ok) {
            const UnitRec &R = next_unit();
            if (done) break;
            const Unit &U = R.U;
            const int n = R.n;
            const int t = in ? U.t0 + my_t : 0, head = in ? U.hk * p.group + my_g : 0;
            Row row = {};
            if (in) row = make_row(p, P, U, head, t);
            // positions the row's window holds (stride 1): [first, after)
            const int after = row.valid ? row.pos + 1 : -1;
            const int first = row.glob ? -1 : max(row.pos - row.reach, -1);
            const bool busy = __any_sync(kAllLanes, row.valid);
            float mref = -CUDART_INF_F, l = 0.f;
            bool had = false;
            for (int i = 0; i < n; ++i) {
                const uint32_t gs = g + (uint32_t)i, slot = gs % kSI;
                if (!(ok = wait_warp(bar(C::B_IF + slot), (gs / kSI) & 1, ctl))) break;
                const int use = recs[slot].use, vz0 = recs[slot].vz0, vz1 = recs[slot].vz1;
                uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};  // visible keys, 32 at a time
                const bool all = (use >> (2 + x)) & 1;
                if (((use >> x) & 1) && !all) {
                    const int j0[2] = {recs[slot].j0[0], recs[slot].j0[1]};
                    if (use & 16) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int j = j0[c >> 1] + (c & 1) * 32;
                            const int lo = max(first - j, 0), hi = min(after - j, 32);
                            w[c] = bit_run(lo, max(hi - lo, 0));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint64_t m =
                                j0[k] == kNowhere ? 0ull : row_mask(row, j0[k] >> 6, recs[slot].gbits[k], recs[slot].present[k]);
                            w[2 * k] = (uint32_t)m;
                            w[2 * k + 1] = (uint32_t)(m >> 32);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_IE + slot));
                if (!((use >> x) & 1)) continue;
                // The step's two 64-key halves: while one half's weights are worked
                // out, the other's product and the next scores run. (Not unrolled:
                // a loop body that the instruction caches of the schedulers hold
                // is worth more than anything else here. Unrolled, the warps
                // waited for instructions 3.9 clocks per issue.)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w0 = h ? w[2] : w[0], w1 = h ? w[3] : w[1];
                    if (!(ok = wait_warp(bar(C::B_SF + 2 * x + h), sc & 1, ctl))) break;
                    // Unwritten memory: no NaN may meet a zero weight. (Not before S
                    // is there: only then are the fills of what the stage held before
                    // complete, and the wait below is for this step's V.)
                    if (h == 0 && vz0 < vz1) {
                        const Pos v_at = stage(i, 1);
                        if (!(ok = wait_warp(bar(C::B_KF + v_at.st), v_at.times & 1, ctl))) break;
                        uint8_t *v = smem + C::ST_OFF + v_at.st * C::TILE;
                        for (int c = tid; c < (vz1 - vz0) * 8 * C::DC; c += 128) {
                            const int r = vz0 + c / (8 * C::DC), q = c % (8 * C::DC);
                            *reinterpret_cast<uint4 *>(v + (q >> 3) * kRegion + r * 128 + (q & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                    if (busy) {
                        tc_fence_after();
                        // 32 keys that no row of the warp sees need no exponentials,
                        // those that all see need no masks
                        int some = 3, full = 3;
                        if (!all) {
                            some = full = 0;
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t wc = c ? w1 : w0;
                                if (__any_sync(kAllLanes, wc != 0u)) some |= 1 << c;
                                if (__all_sync(kAllLanes, wc == ~0u || !row.valid)) full |= 1 << c;
                            }
                        }
                        float s[2][32];
#pragma unroll
                        for (int c = 0; c < 2; ++c) tmem_ld32(s_addr + h * 64 + c * 32, s[c]);
                        tmem_wait_ld();
                        if (full != 3) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t wc = c ? w1 : w0;
                                if (!((full >> c) & 1)) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k) s[c][k] = (wc >> k) & 1u ? s[c][k] : -CUDART_INF_F;
                                }
                            }
                        }
                        float m4[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) m4[k] = fmaxf(s[k >> 1][2 * (k & 1)], s[k >> 1][2 * (k & 1) + 1]);
#pragma unroll
                        for (int k = 4; k < 32; k += 4) {
                            m4[0] = fmax3(m4[0], s[0][k], s[0][k + 1]);
                            m4[1] = fmax3(m4[1], s[0][k + 2], s[0][k + 3]);
                            m4[2] = fmax3(m4[2], s[1][k], s[1][k + 1]);
                            m4[3] = fmax3(m4[3], s[1][k + 2], s[1][k + 3]);
                        }
                        float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
                        mx = row.valid ? mx * sl2 : -CUDART_INF_F;
                        const bool grow = mx > mref + kGrow || (mref == -CUDART_INF_F && mx > mref);
                        if (__any_sync(kAllLanes, grow)) {
                            const float ref = grow ? mx : mref;
                            const float f = grow ? ex2(mref - ref) : 1.f;  // 0 the first time
                            l *= f;
                            mref = ref;
                            if (had) {
                                // the last product handed over may still be running (S of
                                // this half shows only the one before it complete)
                                if (!(ok = wait_warp(bar(C::B_PD + x), (handed - 1) & 1, ctl))) break;
                                tc_fence_after();
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
                        uint32_t pk[32];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            if (!((some >> c) & 1)) {
#pragma unroll
                                for (int k = 0; k < 16; ++k) pk[c * 16 + k] = 0u;
                                continue;
                            }
#pragma unroll
                            for (int k = 0; k < 32; k += 2) {
                                float a, e;
                                f2_unpack(f2_fma(f2_pack(s[c][k], s[c][k + 1]), sl2x2, nrefx2), a, e);
                                a = ex2(a);
                                e = ex2(e);
                                if (k & 2) sum1 = f2_add(sum1, f2_pack(a, e));
                                else sum0 = f2_add(sum0, f2_pack(a, e));
                                pk[c * 16 + k / 2] = pack_bf16(a, e);
                            }
                        }
                        tmem_st32u(s_addr + h * 64, pk);
                        float a, e;
                        f2_unpack(f2_add(sum0, sum1), a, e);
                        l += a + e;
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_PF + 2 * x + h));
                    ++handed;
                    had = true;
                }
                if (!ok) break;
                ++sc;
            }
            if (!ok) break;
            unit_steps(n);
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
                    unit_done();
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
                unit_done();
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
                // where this lane's row goes (-1: nowhere)
                const long long out_at = in && t < p.m ? (((long long)U.b * p.Hq + head) * p.m + t) * D : -1;
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
                    float z[4] = {0.f, 0.f, 0.f, 0.f};  // NaN if any is infinite or NaN
#pragma unroll
                    for (int k = 0; k < 32; ++k) z[k & 3] = fmaf(o[k], 0.f, z[k & 3]);
                    bad |= z[0] + z[1] + z[2] + z[3] != 0.f;
                    if (U.split) {
                        if (in) {
#pragma unroll
                            for (int k = 0; k < 32; k += 4)
                                *reinterpret_cast<float4 *>(p.part_o + part_at<D>(p, U.slot, c * 8 + k / 4, prow)) =
                                    make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                        }
                    } else {
                        // Four lanes hold the 64 bytes of four rows each; a 4 x 4
                        // exchange lets them write one row's 64 bytes together
                        // instead of 16 bytes of four rows (a quarter of the lines
                        // per store: the epilogue took 3200 clocks before, of a
                        // unit's 20000 at window 512).
                        uint32_t b4[4][4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float a = row.valid ? o[q * 8 + 2 * k] * inv : 0.f;
                                const float e = row.valid ? o[q * 8 + 2 * k + 1] * inv : 0.f;
                                b4[q][k] = pack_bf16(a, e);
                            }
#pragma unroll
                        for (int o2 = 1; o2 < 4; o2 <<= 1)  // swap [q][lane] with [lane][q], a bit at a time
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if (q & o2) continue;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const bool up = lane & o2;
                                    const uint32_t give = up ? b4[q][k] : b4[q | o2][k];
                                    const uint32_t got = __shfl_xor_sync(kAllLanes, give, o2);
                                    if (up) b4[q][k] = got; else b4[q | o2][k] = got;
                                }
                            }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {  // row (lane & ~3) + q, its 16 bytes number lane & 3
                            const long long r_at = __shfl_sync(kAllLanes, out_at, (lane & ~3) + q);
                            if (r_at >= 0)
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.O) + r_at + c * 32 + (lane & 3) * 8) =
                                    make_uint4(b4[q][0], b4[q][1], b4[q][2], b4[q][3]);
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
            if (row.valid && (had || had2) && (bad || not_finite(l))) *again = 1;
            unit_done();
        }
        // All softmax warps get here (their waits are bounded), their results written.
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (*again && !*abort_flag) rows_again<__nv_bfloat16, D, 4>(p, smem + C::PLAN_OFF, warp, 8);
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8) {
        // ================================================================ loader of Q, K and V
        const int log_bp = min(p.log_page, 6);  // tokens of a box: a page, at most 64
        const int log_ppb = 6 - log_bp;         // boxes per block and 64-column piece
        const int nbox = (2 << log_ppb) * C::DC;  // at most 16 per stage
        const bool big = p.page > 64;
        uint32_t qc = 0, turn = 0;
        uint32_t armed = 0, phase = 0;  // per stage: filled, and the parity of the last time
        while (ok) {
            const UnitRec &R = next_unit();
            if (done) break;
            const Unit U = R.U;
            const int n = R.n;
            unit_done();
            if (n == 0) continue;
            // A step's boxes: K on lanes [turn, turn + nbox), V on the nbox after
            // them, modulo 32; the lanes move on every step, as a thread's copies
            // complete one after another and different threads' overlap. Each lane
            // has the coordinates of its box; z = -1 reads zeros.
            auto look = [&](int i, int &box, int &y) -> int {
                box = (lane - (int)turn) & 31;
                const int kb = box < nbox ? box : box - nbox;
                const int piece = kb / C::DC, e = U.e0 + 2 * i + (piece >> log_ppb);
                y = 0;
                if (kb >= nbox || i >= n || e >= U.e1) return -1;
                const int blk = entry_block(P, U, e);
                const int pos = (blk << 6) + ((piece & ((1 << log_ppb) - 1)) << log_bp);
                const int pg = pos < U.s ? page_of(p, U.b, pos) : -1;
                if (pg < 0) return -1;
                if (big) y = (blk & 1) * 64;
                return pg * p.Hkv + U.hk;
            };
            auto fill = [&](const CUtensorMap *tm, Pos at, int kb, int y, int z) -> bool {
                const uint32_t st = at.st;
                if (at.times > 0 && !wait_warp(bar(C::B_KE + st), (at.times - 1) & 1, ctl)) return false;
                if (lane == 0) mbar_arrive_expect_tx(bar(C::B_KF + st), C::TILE);
                __syncwarp();
                if (kb >= 0 && kb < nbox)
                    tma_load_3d(sbase + C::ST_OFF + st * C::TILE + (kb % C::DC) * kRegion + ((kb / C::DC) << log_bp) * 128,
                                tm, bar(C::B_KF + st), (kb % C::DC) * 64, y, z);
                armed |= 1u << st;
                phase = (phase & ~(1u << st)) | ((at.times & 1u) << st);
                return true;
            };
            int box, y, z = look(0, box, y);
            if (qc > 0 && !(ok = wait_warp(bar(C::B_QE), (qc - 1) & 1, ctl))) break;
            {
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
            int pbox = 0, py = 0, pz = 0;  // the step before, whose V is still to be loaded (one tile)
            for (int i = 0; i < n; ++i) {
                turn = (turn + 2 * nbox) & 31;
                int box1, y1;
                const int z1 = look(i + 1, box1, y1);  // on its way during this step's waits
                if (!(ok = fill(&tmK, stage(i, 0), box, y, z))) break;
                if (one) {
                    if (i > 0 && !(ok = fill(&tmV, stage(i - 1, 1), pbox - nbox, py, pz))) break;
                    if (i == n - 1 && !(ok = fill(&tmV, stage(i, 1), box - nbox, y, z))) break;
                    pbox = box;
                    py = y;
                    pz = z;
                } else if (!(ok = fill(&tmV, stage(i, 1), box - nbox, y, z))) {
                    break;
                }
                box = box1;
                y = y1;
                z = z1;
            }
            unit_steps(n);
        }
        if (!ok) {  // abort: wait for the copies still in flight
            for (int i = 0; i < C::NST; ++i)
                if ((armed >> i) & 1u) wait_drain(bar(C::B_KF + i), (phase >> i) & 1u);
            if (qc) wait_drain(bar(C::B_QF), (qc - 1) & 1);
        }
    } else if (warp == 10) {
        // ================================================================ step records
        // What each step holds for the tiles, ahead of their use. Lane l looks
        // up piece l % ppb of entry l / ppb.
        const int log_bp = min(p.log_page, 6), log_ppb = 6 - log_bp, ppb = 1 << log_ppb;
        Units units;
        units.begin(p, P, blockIdx.x);
        Unit U;
        for (bool more = true; ok && more; ++uc) {
            more = units.next(p, P, U);
            const int n = more && U.live ? (U.e1 - U.e0 + 1) >> 1 : 0;
            const uint32_t us = uc % kNU;
            if (uc >= kNU && !(ok = wait_warp(bar(C::B_UE + us), ((uc / kNU) - 1) & 1, ctl))) break;
            if (lane == 0) {
                if (more) unit_recs[us].U = U;
                unit_recs[us].n = n;
                unit_recs[us].end = !more;
                mbar_arrive(bar(C::B_UF + us));
            }
            __syncwarp();
            if (n == 0) continue;
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
                // "plain": rows see an interval of the block's keys and no others
                int all = stride == 1 && gb == 0ull && (b < 0 || (w | ~low_bits(written)) == ~0ull) ? 16 : 0;
                const bool whole = stride == 1 && w == ~0ull;
                if (whole && j0 + 63 <= sp0.p0 && j0 >= sp0.last) all |= 4;
                if (whole && j0 + 63 <= sp1.p0 && j0 >= sp1.last) all |= 8;
                const int use2 = use | __shfl_xor_sync(kAllLanes, use, 1);
                const int all2 = all & __shfl_xor_sync(kAllLanes, all, 1);
                const int written2 = __shfl_xor_sync(kAllLanes, written, 1);
                if (g >= kSI && !(ok = wait_warp(bar(C::B_IE + slot), ((g / kSI) - 1) & 1, ctl))) break;
                if (lane < 2) {
                    StepRec &r = recs[slot];
                    r.j0[lane] = b < 0 ? kNowhere : j0;
                    r.gbits[lane] = gb;
                    r.present[lane] = w;
                    if (lane == 0) {
                        r.use = one ? ((use2 & 1) << (i & 1)) | ((all2 & 4) ? 12 : 0) | (all2 & 16) : use2 | all2;
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
    } else {
        // ================================================================ MMA issuers: warp 9 for tile (or chain) 0, 11 for 1
        // The whole warp runs the loop and the waits, so descriptors and TMEM
        // addresses stay warp-uniform; one elected lane issues the MMAs and the
        // commits that track them.
        constexpr uint32_t idesc_qk = idesc_bf16(128, 64, false);
        constexpr uint32_t idesc_pv = idesc_bf16(128, D, true);
        const int x = (warp - 9) >> 1;
        const bool leader = elect_one();
        const uint64_t dQ = desc_sw128(sbase + C::Q_OFF + (one ? 0 : x) * C::TILE, 16);
        const uint64_t dK0 = desc_sw128(sbase + C::ST_OFF, 16);
        const uint64_t dV0 = desc_sw128(sbase + C::ST_OFF, kRegion);
        const uint32_t s_col = tmem + x * 128, o_col = tmem + C::O_COL + x * D;
        const uint32_t b_sf = bar(C::B_SF + 2 * x), b_pf = bar(C::B_PF + 2 * x);
        uint32_t qc = 0, pc = 0, oc = 0;
        auto filled = [&](Pos at) { return wait_warp(bar(C::B_KF + at.st), at.times & 1, ctl); };
        while (ok) {
            const int n = next_unit().n;
            if (done) break;
            unit_done();
            if (n == 0) continue;
            if (!(ok = wait_warp(bar(C::B_QF), qc & 1, ctl))) break;
            ++qc;
            bool started = false;
            int pend = -1;  // step whose weights are to be used
            // By halves of 64 keys: O (+)= P V of the pending step (`pend`) as soon
            // as the half's weights are there, then the scores of step i, whose S
            // takes their place. So a tile's softmax finds the next scores ready.
            auto halves = [&](int i, bool scores) -> bool {
                Pos vx = {0, 0}, kx = {0, 0};
                if (scores) {
                    kx = stage(i, 0);
                    if (!filled(kx)) return false;
                }
                if (pend >= 0) {
                    vx = stage(pend, 1);
                    if (!started && oc > 0 && !wait_warp(bar(C::B_OE + x), (oc - 1) & 1, ctl)) return false;
                    if (!filled(vx)) return false;
                }
                const uint64_t dV = dV0 + (uint64_t)((vx.st * C::TILE) >> 4);
                const uint64_t dK = dK0 + (uint64_t)((kx.st * C::TILE) >> 4);
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (pend >= 0 && !wait_warp(b_pf + 8 * h, pc & 1, ctl)) return false;
                    tc_fence_after();
                    if (leader) {
                        if (pend >= 0) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_bf16_ts(o_col, s_col + h * 64 + kk * 8, dV + (uint64_t)(((4 * h + kk) * 2048) >> 4),
                                            idesc_pv, (!started && h == 0 && kk == 0) ? 0u : 1u);
                            mma_commit(bar(C::B_PD + x));
                            if (h == 1) mma_commit(bar(C::B_KE + vx.st));
                        }
                        if (scores) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t off = (uint64_t)(((kk >> 2) * kRegion + (kk & 3) * 32) >> 4);
                                mma_bf16_ss(s_col + h * 64, dQ + off, dK + off + (uint64_t)((h * 8192) >> 4), idesc_qk,
                                            kk > 0 ? 1u : 0u);
                            }
                            mma_commit(b_sf + 8 * h);
                            if (h == 1) mma_commit(bar(C::B_KE + kx.st));
                        }
                    }
                    __syncwarp();
                }
                if (pend >= 0) {
                    ++pc;
                    started = true;
                }
                pend = scores ? i : -1;
                return true;
            };
            // With one tile every step is used: its blocks lie in the window, or hold
            // a global key before it (the plan's lists are ascending).
            const int step = one ? 2 : 1;
            for (int i = one ? x : 0; i < n; i += step) {
                bool use = true;
                if (!one) {
                    const uint32_t gs = g + i, slot = gs % kSI;
                    if (!(ok = wait_warp(bar(C::B_IF + slot), (gs / kSI) & 1, ctl))) break;
                    use = (recs[slot].use >> x) & 1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_IE + slot));
                }
                if ((use || pend >= 0) && !(ok = halves(i, use))) break;
                if (!use) {  // the other tile's alone. (Its stages are filled: an arrival
                             // cannot be taken for one of the time before.)
                    const Pos kx = stage(i, 0), vx = stage(i, 1);
                    if (!(ok = filled(kx)) || !(ok = filled(vx))) break;
                    if (lane == 0) {
                        mbar_arrive(bar(C::B_KE + kx.st));
                        mbar_arrive(bar(C::B_KE + vx.st));
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            if (leader) mma_commit(bar(C::B_QE));
            __syncwarp();
            if (pend >= 0 && !(ok = halves(n, false))) break;
            if (started) {
                if (leader) mma_commit(bar(C::B_OF + x));
                __syncwarp();
                ++oc;
            }
            unit_steps(n);
        }
        // every MMA issued has completed once this arrives
        if (leader) mma_commit(bar(C::B_DRAIN + x));
        __syncwarp();
        wait_drain(bar(C::B_DRAIN + x), 0);
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

static_assert(TcCfg<128>::PLAN_OFF + 1024 + plan_bytes(kPagedMaxBatch, kPagedMaxGlobal, kPagedMaxHeads) <= 232448,
              "the largest plan fits beside the tiles");

}  // namespace sa
