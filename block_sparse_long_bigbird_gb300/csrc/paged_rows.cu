// Attention of a few new tokens per sequence over a paged cache (single-token
// steps, short drafts), bf16 and fp32, on the ordinary units.
//
//     O_r = sum_j w_rj V_j / sum_j w_rj,   w_rj = 2^(s_rj - max_j s_rj),   s = q . k log2(e) / sqrt(d)
//
// A call reads each visible key and value row once per key head and does a few
// flops per byte: the memory bounds it as long as a key head has few rows: one in
// bf16, up to R = 8 in fp32 (tokens x query heads of the key head). One warp takes 16 keys
// at a time (one page, one table entry): each key's row is spread over
// D / 8 (bf16) or D / 4 (fp32) lanes, 16 bytes each, so all loads are full
// lines; K and V of the 16 keys are requested together before either is used.
// Every group of lanes keeps a running maximum, sum and D-sum of its own keys
// in registers and in fp32; groups, then warps, are joined once at the end of
// the unit. Masked keys are not loaded: dilated heads read only their own
// keys, and unwritten memory is never touched. Long sweeps are cut into units
// by the plan; their partial results are joined by paged_merge in a fixed
// order, so results do not depend on timing.
//
// Measured (16 sequences of 32768 keys, one row per key head): bf16, 8 key heads, d =
// 64 173 us, 6.2 TB/s; d = 128 320 us, 6.7 TB/s (a plain copy: 6.7); fp32, 4 key heads,
// 16384 keys, d = 128, 170 us, 6.3 TB/s, two rows 173, four 199, eight 377. Eight rows
// leave an SM one CTA of 8 warps at 249 registers, which issues half of the time, much
// of it the shuffles that sum each score over its lanes; the multiply-adds take 28% of
// their rate and the memory 31%. The smallest call takes 5.5 us, half of it launch and plan.
#include "paged_common.cuh"

namespace sa {
namespace {

constexpr int kRowsWarps = 8;
constexpr int kItem = 16;  // keys a warp takes at a time

template <typename T, int D, int R>
__global__ void __launch_bounds__(kRowsWarps * 32, R == 8 ? 1 : 2)
    paged_rows(const __grid_constant__ PagedProblem p) {
    constexpr int VE = 16 / sizeof(T);  // elements of a 16-byte load
    constexpr int LPK = D / VE;         // lanes per key
    constexpr int KPL = 32 / LPK;       // keys per warp-wide load
    constexpr int NIT = kItem / KPL;    // loads per item
    constexpr int CH = 4;               // of which this many are in flight together
    static_assert(NIT % CH == 0, "whole chunks");
    extern __shared__ __align__(16) uint8_t smem[];
    // joining the warps' results: [warp][R] maxima and sums, [warp][R][D] sums
    float *jm = reinterpret_cast<float *>(smem);
    float *jl = jm + kRowsWarps * R;
    float *ja = jl + kRowsWarps * R;
    UnitRoom *room = reinterpret_cast<UnitRoom *>(ja + kRowsWarps * R * D);
    Plan P = plan_at(room + 1, p.B, p.ng, p.Hkv);
    make_plan(p, P);
    asm volatile("griddepcontrol.launch_dependents;");  // the join may start planning
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = lane / LPK, sub = lane % LPK;
    const T *Kp = static_cast<const T *>(p.K), *Vp = static_cast<const T *>(p.V);

    if (tid == 0) {
        room->units.begin(p, P, blockIdx.x);
        fill_room(p, P, room, 0);
    }
    __syncthreads();
    for (int k = 0; room->more[k]; k ^= 1) {
        const Unit &U = room->U[k];
        float q[R][VE], acc[R][VE], m[R], l[R];
        // lane r masks for row r; the warp reads the masks from there
        Row mine;
        {
            int t, head;
            row_token(p, U, lane < p.rows ? lane : 0, p.tpt, t, head);
            mine = make_row(p, P, U, head, t);
            mine.valid = mine.valid && lane < p.rows;
        }
        const uint32_t rows_in = __ballot_sync(kAllLanes, mine.valid);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int t, head;
            row_token(p, U, r < p.rows ? r : 0, p.tpt, t, head);
            m[r] = -CUDART_INF_F;
            l[r] = 0.f;
#pragma unroll
            for (int i = 0; i < VE; ++i) acc[r][i] = q[r][i] = 0.f;
            if ((rows_in >> r) & 1u) {
                const uint4 w = *reinterpret_cast<const uint4 *>(
                    static_cast<const T *>(p.Q) + (((size_t)U.b * p.Hq + head) * p.m + t) * D + sub * VE);
#pragma unroll
                for (int i = 0; i < VE; ++i) q[r][i] = element<T>(w, i) * p.scale_log2;
            }
        }
        // Items of this unit: four per 64-key block, dealt to the warps in turn, in
        // chunks of CH loads. The next chunk's keys and values (R <= 2: registers
        // allow it) and the page of the item after next are on their way while a
        // chunk is worked on.
        constexpr int NCH = NIT / CH;
        constexpr bool AHEAD = R <= 2;
        const int i_end = 4 * U.e1;
        struct Item {
            int i, blk, pg;
        };
        auto item_at = [&](int i) -> Item {
            Item x = {i, 0, -1};
            if (i < i_end) {
                x.blk = entry_block(P, U, i >> 2);
                x.pg = page_of(p, U.b, (x.blk << 6) + (i & 3) * kItem);
            }
            return x;
        };
        struct Masks {
            uint32_t m[R], any;
            bool same;
        };
        auto masks_of = [&](const Item &x) -> Masks {
            Masks k;
            k.any = 0u;
            uint32_t all = 0xffffu, w = 0u;
            if (x.pg >= 0)
                w = (uint32_t)(row_mask(mine, x.blk, global_bits(P, p, x.blk), ~0ull) >> ((x.i & 3) * kItem)) & 0xffffu;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                k.m[r] = __shfl_sync(kAllLanes, w, r);
                k.any |= k.m[r];
                if ((rows_in >> r) & 1u) all &= k.m[r];
            }
            k.same = all == k.any;  // every row sees the same keys
            return k;
        };
        // keys [c CH KPL, ...) of the item; what no row sees is not loaded
        auto load = [&](const Item &x, uint32_t any, int c, uint4 (&kw)[CH], uint4 (&vw)[CH]) {
            const int j0 = (x.blk << 6) + (x.i & 3) * kItem;
            const size_t at = any ? ((((size_t)x.pg * p.Hkv + U.hk) << p.log_page) + (j0 & (p.page - 1))) * D + sub * VE : 0;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int kk = (c * CH + i) * KPL + grp;
                kw[i] = make_uint4(0u, 0u, 0u, 0u);
                if ((any >> kk) & 1u) kw[i] = __ldg(reinterpret_cast<const uint4 *>(Kp + at + (size_t)kk * D));
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int kk = (c * CH + i) * KPL + grp;
                vw[i] = make_uint4(0u, 0u, 0u, 0u);
                if ((any >> kk) & 1u) vw[i] = __ldg(reinterpret_cast<const uint4 *>(Vp + at + (size_t)kk * D));
            }
        };
        auto work = [&](const Masks &k, int c, const uint4 (&kw)[CH], const uint4 (&vw)[CH]) {
            float s[R][CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
#pragma unroll
                for (int r = 0; r < R; ++r) s[r][i] = 0.f;
#pragma unroll
                for (int x = 0; x < VE; ++x) {
                    const float kf = element<T>(kw[i], x);
#pragma unroll
                    for (int r = 0; r < R; ++r) s[r][i] = fmaf(q[r][x], kf, s[r][i]);
                }
            }
#pragma unroll
            for (int o = LPK / 2; o; o >>= 1)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < CH; ++i) s[r][i] += __shfl_xor_sync(kAllLanes, s[r][i], o);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float mn = m[r];
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    if (!((k.m[r] >> ((c * CH + i) * KPL + grp)) & 1u)) s[r][i] = -CUDART_INF_F;
                    mn = fmaxf(mn, s[r][i]);
                }
                const float ref = mn == -CUDART_INF_F ? 0.f : mn;
                const float f = ptx::ex2(m[r] - ref);  // 0 from the initial -inf
                m[r] = mn;
                l[r] *= f;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    s[r][i] = ptx::ex2(s[r][i] - ref);
                    l[r] += s[r][i];
                }
#pragma unroll
                for (int x = 0; x < VE; ++x) acc[r][x] *= f;
            }
            if (k.same) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
#pragma unroll
                    for (int x = 0; x < VE; ++x) {
                        const float vx = element<T>(vw[i], x);
#pragma unroll
                        for (int r = 0; r < R; ++r) acc[r][x] = fmaf(s[r][i], vx, acc[r][x]);
                    }
                }
            } else {  // a value that some row does not see may be anything: keep 0 x NaN out of that row
#pragma unroll
                for (int i = 0; i < CH; ++i) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const bool sees = (k.m[r] >> ((c * CH + i) * KPL + grp)) & 1u;
#pragma unroll
                        for (int x = 0; x < VE; ++x)
                            acc[r][x] = sees ? fmaf(s[r][i], element<T>(vw[i], x), acc[r][x]) : acc[r][x];
                    }
                }
            }
        };
        Item now = item_at(4 * U.e0 + warp), after = item_at(4 * U.e0 + warp + kRowsWarps);
        Masks km = masks_of(now);
        uint4 kw[CH], vw[CH];
        if (AHEAD && now.i < i_end) load(now, km.any, 0, kw, vw);
        if (tid == 0) fill_room(p, P, room, k ^ 1);  // while the first items are on their way
        __syncwarp();
        while (now.i < i_end) {
            const Item third = item_at(after.i + kRowsWarps);
            Masks kn = km;
#pragma unroll 1
            for (int c = 0; c < NCH; ++c) {
                if constexpr (AHEAD) {
                    uint4 kw2[CH], vw2[CH];
                    const bool last = c == NCH - 1;
                    if (last) kn = masks_of(after);
                    load(last ? after : now, last ? kn.any : km.any, last ? 0 : c + 1, kw2, vw2);
                    if (km.any) work(km, c, kw, vw);
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        kw[i] = kw2[i];
                        vw[i] = vw2[i];
                    }
                } else if (km.any) {
                    load(now, km.any, c, kw, vw);
                    work(km, c, kw, vw);
                }
            }
            if constexpr (!AHEAD) kn = masks_of(after);
            now = after;
            after = third;
            km = kn;
        }
        // join the groups of lanes of a warp
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int o = LPK; o < 32; o <<= 1) {
                const float m2 = __shfl_xor_sync(kAllLanes, m[r], o), l2 = __shfl_xor_sync(kAllLanes, l[r], o);
                const float mn = fmaxf(m[r], m2), ref = mn == -CUDART_INF_F ? 0.f : mn;
                const float f = ptx::ex2(m[r] - ref), f2 = ptx::ex2(m2 - ref);
                l[r] = l[r] * f + l2 * f2;
#pragma unroll
                for (int x = 0; x < VE; ++x) {
                    const float a2 = __shfl_xor_sync(kAllLanes, acc[r][x], o);
                    acc[r][x] = acc[r][x] * f + a2 * f2;
                }
                m[r] = mn;
            }
            if (grp == 0) {
#pragma unroll
                for (int x = 0; x < VE; ++x) ja[(warp * R + r) * D + sub * VE + x] = acc[r][x];
            }
            if (lane == 0) {
                jm[warp * R + r] = m[r];
                jl[warp * R + r] = l[r];
            }
        }
        __syncthreads();
        // and the warps, in order
        for (int idx = tid; idx < p.rows * D; idx += kRowsWarps * 32) {
            const int r = idx / D, x = idx % D;
            float mx = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w) mx = fmaxf(mx, jm[w * R + r]);
            const float ref = mx == -CUDART_INF_F ? 0.f : mx;
            float ls = 0.f, a = 0.f;
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w) {
                const float f = ptx::ex2(jm[w * R + r] - ref);
                ls = fmaf(jl[w * R + r], f, ls);
                a = fmaf(ja[(w * R + r) * D + x], f, a);
            }
            int t, head;
            row_token(p, U, r, p.tpt, t, head);
            if (U.split) {
                p.part_o[part_at<D>(p, U.slot, x >> 2, r) + (x & 3)] = a;
                if (x == 0) p.part_ml[(size_t)U.slot * p.rows + r] = make_float2(mx, ls);
            } else if (t < p.m) {
                static_cast<T *>(p.O)[(((size_t)U.b * p.Hq + head) * p.m + t) * D + x] =
                    from_float<T>(ls == 0.f ? 0.f : a / ls);
            }
        }
        __syncthreads();
    }
}

// Joins the partial results of split tiles, piece by piece in order. A work item
// is a boundary between two CTAs (a tile belongs to the first boundary inside
// it) and a share of its tile's groups of sixteen elements; a thread takes a
// group. Where a tile is cut into many pieces (few rows against a long cache)
// kMergeShare threads take a group, each a stretch of the pieces. Launched so
// that its plan is computed while the sweeps still run.
constexpr int kMergeThreads = 128, kMergeShare = 8, kMergeMany = 12;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge(const PagedProblem p, int per_tile) {
    extern __shared__ __align__(16) uint8_t smem[];
    Plan P = plan_at(smem, p.B, p.ng, p.Hkv);
    make_plan(p, P);
    const int groups = p.rows * (D / 16);
    const int half_rows = p.tpt_half * p.group;
    const long long n_items = (long long)(P.ctas - 1) * per_tile;
    for (long long w = blockIdx.x; w < n_items && P.cut; w += gridDim.x) {
        const int c = 1 + (int)(w / per_tile), chunk = (int)(w % per_tile);
        const long long at = cta_begin(P, c);
        const Tile tile = find_tile(p, P, at);
        if (!tile.live || tile.begin == at || tile.begin < cta_begin(P, c - 1)) continue;
        const int ns = cta_of(P, tile.end - 1, c) - c + 2;  // pieces: slot 2 c - 1, then 2 c, 2 c + 2, ...
        const int share = ns > kMergeMany ? kMergeShare : 1;
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the sweeps' results are visible from here on
        auto slot = [&](int k) { return k == 0 ? 2 * c - 1 : 2 * (c + k - 1); };
        for (int idx = chunk * kMergeThreads + (int)threadIdx.x; idx - (int)threadIdx.x < groups * share;
             idx += per_tile * kMergeThreads) {
            const int gi = idx / share, part = idx % share;  // the threads that share a group are neighbours
            const bool in = gi < groups;
            const int row = in ? gi % p.rows : 0, k16 = in ? gi / p.rows : 0;
            float mx = -CUDART_INF_F;
            for (int k = part; k < ns; k += share) mx = fmaxf(mx, p.part_ml[(size_t)slot(k) * p.rows + row].x);
            for (int o = 1; o < share; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAllLanes, mx, o));
            const float ref = mx == -CUDART_INF_F ? 0.f : mx;
            float l = 0.f, acc[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = 0.f;
            const int k0 = ns * part / share, k1 = ns * (part + 1) / share;
#pragma unroll 2
            for (int k = k0; k < k1; ++k) {
                const float2 y = p.part_ml[(size_t)slot(k) * p.rows + row];
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = *reinterpret_cast<const float4 *>(p.part_o + part_at<D>(p, slot(k), 4 * k16 + i, row));
                const float f = ptx::ex2(y.x - ref);
                l = fmaf(y.y, f, l);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[4 * i] = fmaf(v[i].x, f, acc[4 * i]);
                    acc[4 * i + 1] = fmaf(v[i].y, f, acc[4 * i + 1]);
                    acc[4 * i + 2] = fmaf(v[i].z, f, acc[4 * i + 2]);
                    acc[4 * i + 3] = fmaf(v[i].w, f, acc[4 * i + 3]);
                }
            }
            for (int o = 1; o < share; o <<= 1) {
                l += __shfl_xor_sync(kAllLanes, l, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] += __shfl_xor_sync(kAllLanes, acc[i], o);
            }
            if (!in || part != 0) continue;
            // the two halves of a unit hold different tokens
            Unit U;
            const int x = row / half_rows;
            U.hk = tile.hk;
            U.t0 = tile.t0 + x * p.tpt_half;
            int t, head;
            row_token(p, U, row - x * half_rows, p.tpt_half, t, head);
            if (t >= p.m) continue;
            const bool zero = t >= tile.q || l == 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = zero ? 0.f : acc[i] / l;
            store16<T>(static_cast<T *>(p.O) + (((size_t)tile.b * p.Hq + head) * p.m + t) * D + 16 * k16, acc);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // whatever follows this launch follows the sweeps too
}

template <typename T, int D, int R>
cudaError_t launch_rows(const PagedProblem &p, cudaStream_t stream) {
    const size_t smem = (size_t)kRowsWarps * R * (D + 2) * 4 + sizeof(UnitRoom) + plan_bytes(p.B, p.ng, p.Hkv);
    static std::atomic<bool> done[64];
    auto kern = paged_rows<T, D, R>;
    cudaError_t e = allow_smem(kern, done, smem);
    if (e != cudaSuccess) return e;
    kern<<<p.slots, kRowsWarps * 32, smem, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_rows_r(const PagedProblem &p, cudaStream_t stream) {
    if constexpr (sizeof(T) == 4) {
        if (p.rows > 4) return launch_rows<T, D, 8>(p, stream);
        if (p.rows > 2) return launch_rows<T, D, 4>(p, stream);
        if (p.rows > 1) return launch_rows<T, D, 2>(p, stream);
    }
    return launch_rows<T, D, 1>(p, stream);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedProblem &p, sa_dtype dtype, cudaStream_t stream) {
    if (dtype == SA_FP32)
        return p.d == 64 ? launch_rows_r<float, 64>(p, stream) : launch_rows_r<float, 128>(p, stream);
    return p.d == 64 ? launch_rows_r<__nv_bfloat16, 64>(p, stream)
                     : launch_rows_r<__nv_bfloat16, 128>(p, stream);
}

cudaError_t launch_paged_merge(const PagedProblem &p, sa_dtype dtype, int num_sms, cudaStream_t stream) {
    const size_t smem = plan_bytes(p.B, p.ng, p.Hkv);
    void (*kern)(const PagedProblem, int) =
        dtype == SA_FP32 ? (p.d == 64 ? paged_merge<float, 64> : paged_merge<float, 128>)
                         : (p.d == 64 ? paged_merge<__nv_bfloat16, 64> : paged_merge<__nv_bfloat16, 128>);
    static_assert(plan_bytes(kPagedMaxBatch, kPagedMaxGlobal, kPagedMaxHeads) <= 48 * 1024,
                  "no more shared memory than a kernel has without asking");  // 29 KB
    // CTAs per tile: as many as its groups keep busy, within what fits the GPU at a time
    const long long tiles = (long long)p.B * p.Hkv * ((p.m + p.tpt - 1) / p.tpt);
    const int share = p.slots / tiles >= kMergeMany ? kMergeShare : 1;
    const long long busy = ((long long)p.rows * (p.d / 16) * share + kMergeThreads - 1) / kMergeThreads;
    long long per_tile = 16ll * num_sms / p.slots;
    per_tile = per_tile > busy ? busy : per_tile < 1 ? 1 : per_tile;
    const long long items = per_tile * p.slots, grid = 8ll * num_sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items < grid ? items : grid));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, (int)per_tile);
}

}  // namespace sa
