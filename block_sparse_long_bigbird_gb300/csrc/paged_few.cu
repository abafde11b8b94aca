// Attention of a few new tokens per sequence over a paged cache in bf16, 2 to
// 24 rows per key head (rows = tokens x query heads of the key head).
//
//     O_r = sum_j w_rj V_j / sum_j w_rj,   w_rj = 2^(s_rj - max_j s_rj),   s = q . k log2(e) / sqrt(d)
//
// Each visible key and value row is read once per key head, so the memory
// bounds it as long as the arithmetic keeps up: 4 R flops per element of the
// cache for R rows, which the ordinary units manage for one row, and which the
// 128-row tiles of the tensor cores bury under a softmax of 128 rows. So a warp
// takes 16 keys at a time and multiplies them with tiles of 8 rows by warp-level
// matrix instructions (m16n8k16), keys or elements of V down, rows across:
//   S^T (16 x 8) = K Q^T, weights from S in registers, O^T (d x 8) += V^T P^T.
// No operand goes through a shared layout:
//   * the sum over d may run in any order, so a lane's 16-byte piece of a key
//     row serves as its share of two k-steps of S; Q is held in the same order;
//   * the rows of O^T may stand in any order, so a lane reads 16-byte pieces of
//     four value rows and pairs up their elements for four tiles; its sums end
//     up as 8 neighbouring elements of two rows of O.
// Copies (cp.async) go to a ring of the warp's own, two items deep: 128 KB in
// flight per SM, and no barrier. (Three items leave L1, which the copies go
// through, too little room: 64 sequences of 4096 keys, 8 key heads, d = 128, take
// 207 us instead of 176.) A copy instruction takes whole lines: the 64 bytes of
// eight keys that the lanes themselves would use were fetched from L2 twice.
// Masked keys are copied as zeros without being read.
// With rows down instead of across a tile would be 16 rows and take twice the
// matrix instructions for 8.
// Up to 8 rows P V is computed with P as the sum of two bf16 numbers (relative
// 2^-16), which the rate allows; with more, P is rounded to bf16 (2^-8 of each
// weight), as in the kernel for many rows.
// Measured (16 sequences of 32768 keys, 8 key heads): d = 128, 4 rows 320 us, 6.7 TB/s
// (a plain copy: 6.7), 16 rows 324, 24 rows 336 us; d = 64 170, 175 and 190 us, 6.3 to
// 5.7 TB/s. One sequence of 900 keys takes 10.9 us (d = 64), a few hundred
// clocks per item and warp: latency.
// A row that does not see a key multiplies its value by 0; where that value is
// infinite or NaN the row's sums come out so, and rows_again takes it again.
#include "paged_common.cuh"

namespace sa {
namespace {

constexpr int kItem = 16;    // keys a warp takes at a time
constexpr float kGrow = 8.f;  // growth of a maximum (log2) that rescales the sums
constexpr int kStages = 2;   // items in flight per warp

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes from global to shared memory, or zeros (nothing is read). Through L1
// and with the widest prefetch into L2: past L1 (.cg) the same kernel reads 5.0
// to 5.3 TB/s instead of 6.2 to 6.7.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.ca.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Transposes an 8 x 8 matrix of 16-bit numbers, two of a row per lane.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int D, int NT, int W>
struct Few {
    static constexpr int ctas = paged_few_ctas(D, 8 * NT, W);  // per SM
    static constexpr int pieces = kItem * D * 2 * 2 / 512;  // a lane's 16-byte pieces of an item: K, then V
    static constexpr int f4 = NT * D / 16;                  // float4 of a lane's sums
    static constexpr int stages = kStages * pieces * 512, results = f4 * 512 + NT * 64;
    static constexpr int ring = stages > results ? stages : results;  // bytes per warp
    static size_t smem(const PagedProblem &p) {
        return (size_t)W * ring + sizeof(UnitRoom) + 16 + plan_bytes(p.B, p.ng, p.Hkv);
    }
};

template <int D, int NT, int W>
__global__ void __launch_bounds__(W * 32, Few<D, NT, W>::ctas) paged_few(const __grid_constant__ PagedProblem p) {
    using C = Few<D, NT, W>;
    using bf16 = __nv_bfloat16;
    constexpr int SETS = D / 64, CH = D / 32;
    constexpr int PK = D / 8;  // 16-byte pieces of a key
    extern __shared__ __align__(16) uint8_t smem[];
    UnitRoom *room = reinterpret_cast<UnitRoom *>(smem + W * C::ring);
    int *again = reinterpret_cast<int *>(room + 1);  // whether a row is to be taken again
    Plan P = plan_at(again + 4, p.B, p.ng, p.Hkv);
    make_plan(p, P);
    asm volatile("griddepcontrol.launch_dependents;");  // the join may start planning
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = lane >> 2, quad = lane & 3;
    const bf16 *Kp = static_cast<const bf16 *>(p.K), *Vp = static_cast<const bf16 *>(p.V);
    uint8_t *mine_at = smem + warp * C::ring;
    const uint4 *ring = reinterpret_cast<const uint4 *>(mine_at) + lane;
    const uint32_t stage_at = ptx::smem_u32(mine_at), ring_at = stage_at + lane * 16;
    // piece 4 c + quad of key n, from the lane's own place: pieces of odd keys are
    // swapped in fours, so that eight lanes read from eight places
    const int odd = 4 * (n & 1), own = n * PK + quad - lane;

    if (tid == 0) {
        *again = 0;
        room->units.begin(p, P, blockIdx.x);
        fill_room(p, P, room, 0);
    }
    __syncthreads();
    for (int k = 0; room->more[k]; k ^= 1) {
        const Unit &U = room->U[k];
        Row mine;  // lane r masks for row r
        {
            int t, head;
            row_token(p, U, lane < p.rows ? lane : 0, p.tpt, t, head);
            mine = make_row(p, P, U, head, t);
            mine.valid = mine.valid && lane < p.rows;
        }
        const uint32_t rows_in = __ballot_sync(kAllLanes, mine.valid);
        int full0 = 0, full1 = 0x7fffffff;  // blocks that every row sees whole
        if (mine.valid) {
            full0 = mine.glob ? 0 : mine.stride > 1 ? 0x7fffffff : (max(0, mine.pos - mine.reach) + 63) >> 6;
            full1 = (mine.pos + 1) >> 6;
        }
        full0 = __reduce_max_sync(kAllLanes, full0);
        full1 = __reduce_min_sync(kAllLanes, full1);
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
            uint32_t w;     // the keys that the lane's row sees
            uint32_t both;  // keys that any row sees, and those that all see (upper half)
        };
        // Starts the copies of an item.
        auto fetch = [&](const Item &x, int st) -> Masks {
            uint32_t w = 0u, any = 0u, all = 0u;
            if (x.pg >= 0 && x.blk >= full0 && x.blk < full1) {
                w = any = all = 0xffffu;
            } else if (x.pg >= 0) {
                w = (uint32_t)(row_mask(mine, x.blk, global_bits(P, p, x.blk), ~0ull) >> ((x.i & 3) * kItem)) & 0xffffu;
                any = __reduce_or_sync(kAllLanes, w);
                all = __reduce_and_sync(kAllLanes, mine.valid ? w : 0xffffu);
            }
            __syncwarp();  // all lanes have read what the copies overwrite
            if (any) {
                const int j0 = (x.blk << 6) + (x.i & 3) * kItem;
                const size_t at = ((((size_t)x.pg * p.Hkv + U.hk) << p.log_page) + (j0 & (p.page - 1))) * D;
                uint32_t to = ring_at + st * (C::pieces * 512);
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i) {
                    const int key = (i * 32 + lane) / PK, x = lane % PK;
                    copy16(stage_at + st * (C::pieces * 512) + (key * PK + (x ^ (4 * (key & 1)))) * 16,
                           Kp + at + key * D + x * 8, (any >> key) & 1u);
                }
                to += 2 * CH * 512;
#pragma unroll
                for (int s = 0; s < SETS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i, to += 512) {
                        const int kk = 2 * quad + (i & 1) + 4 * (i & 2);
                        copy16(to, Vp + at + kk * D + s * 64 + n * 8, (any >> kk) & 1u);
                    }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            return {w, any | all << 16};
        };
        Item next = item_at(4 * U.e0 + warp);
        Masks w[kStages];  // of the items in flight, oldest first
        {
            Item x[kStages + 1];
            x[0] = next;
#pragma unroll
            for (int s = 1; s <= kStages; ++s) x[s] = item_at(4 * U.e0 + warp + s * W);
#pragma unroll
            for (int s = 0; s < kStages; ++s) w[s] = fetch(x[s], s);
            next = x[kStages];
        }
        uint4 q[NT][CH];  // row 8 nt + n, zeros past the last
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = 8 * nt + n;
            int t, head;
            row_token(p, U, row < p.rows ? row : 0, p.tpt, t, head);
            const bf16 *at = static_cast<const bf16 *>(p.Q) + (((size_t)U.b * p.Hq + head) * p.m + t) * D + quad * 8;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                q[nt][c] = make_uint4(0u, 0u, 0u, 0u);
                if ((rows_in >> row) & 1u) q[nt][c] = __ldg(reinterpret_cast<const uint4 *>(at + c * 32));
            }
        }
        // sums of O^T: [x] is (element 2 t, row 2 quad), (2 t, 2 quad + 1), then those of 2 t + 1
        float acc[NT][SETS][4][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                m[nt][x] = -CUDART_INF_F;
                l[nt][x] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < SETS * 16; ++i) acc[nt][i / 16][(i / 4) % 4][i % 4] = 0.f;
        }
        if (tid == 0) fill_room(p, P, room, k ^ 1);  // while the first items are on their way
        __syncwarp();
        int st = 0;
#pragma unroll 1
        for (int i = 4 * U.e0 + warp; i < i_end; i += W) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            const uint4 *at = ring + st * (C::pieces * 32);
            const uint32_t all = w[0].both >> 16;
            if (w[0].both & 0xffffu) {
                float s[NT][4];  // keys n, n, n + 8, n + 8 for rows 2 quad, 2 quad + 1 in turn
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[nt][x] = 0.f;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint4 k0 = at[own + ((4 * c) ^ odd)], k1 = at[own + 8 * PK + ((4 * c) ^ odd)];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], k0.x, k1.x, k0.y, k1.y, q[nt][c].x, q[nt][c].y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], k0.z, k1.z, k0.w, k1.w, q[nt][c].z, q[nt][c].w);
                }
                uint32_t hi[NT][2], lo[2];  // weights as the right operand
                bool up = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t sees =
                            all == 0xffffu ? 0xffffu : __shfl_sync(kAllLanes, w[0].w, 8 * nt + 2 * quad + x);
                        s[nt][x] = (sees >> n) & 1u ? s[nt][x] * p.scale_log2 : -CUDART_INF_F;
                        s[nt][2 + x] = (sees >> (n + 8)) & 1u ? s[nt][2 + x] * p.scale_log2 : -CUDART_INF_F;
                        up |= fmaxf(s[nt][x], s[nt][2 + x]) > m[nt][x] + kGrow;
                    }
                }
                if (__any_sync(kAllLanes, up)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float f[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float mn = fmaxf(s[nt][x], s[nt][2 + x]);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(kAllLanes, mn, o));
                            mn = fmaxf(mn, m[nt][x]);
                            f[x] = mn == -CUDART_INF_F ? 0.f : ptx::ex2(m[nt][x] - mn);  // 0 from the initial -inf
                            m[nt][x] = mn;
                            l[nt][x] *= f[x];
                        }
#pragma unroll
                        for (int i = 0; i < SETS * 16; ++i) acc[nt][i / 16][(i / 4) % 4][i % 4] *= f[i & 1];
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float ref = m[nt][x] == -CUDART_INF_F ? 0.f : m[nt][x];
                        s[nt][x] = ptx::ex2(s[nt][x] - ref);
                        s[nt][2 + x] = ptx::ex2(s[nt][2 + x] - ref);
                        l[nt][x] += s[nt][x] + s[nt][2 + x];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // keys n, then n + 8
                        const float a = s[nt][2 * h], b = s[nt][2 * h + 1];
                        const uint32_t u = pack_bf16(a, b);
                        hi[nt][h] = transposed(u);
                        if constexpr (NT == 1)
                            lo[h] = transposed(pack_bf16(a - __uint_as_float(u << 16), b - __uint_as_float(u & 0xffff0000u)));
                    }
                }
#pragma unroll
                for (int set = 0; set < SETS; ++set) {
                    uint4 v[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) v[x] = at[(2 * CH + set * 4 + x) * 32];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t a0 = __byte_perm(word(v[0], t), word(v[1], t), 0x5410u);
                        const uint32_t a1 = __byte_perm(word(v[0], t), word(v[1], t), 0x7632u);
                        const uint32_t a2 = __byte_perm(word(v[2], t), word(v[3], t), 0x5410u);
                        const uint32_t a3 = __byte_perm(word(v[2], t), word(v[3], t), 0x7632u);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816(acc[nt][set][t], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
                        if constexpr (NT == 1) mma16816(acc[0][set][t], a0, a1, a2, a3, lo[0], lo[1]);
                    }
                }
            }
#pragma unroll
            for (int s = 0; s + 1 < kStages; ++s) w[s] = w[s + 1];
            const Item x = next;
            next = item_at(i + (kStages + 1) * W);
            w[kStages - 1] = fetch(x, st);
            st = st + 1 == kStages ? 0 : st + 1;
        }
        // Results into the warp's ring, which has nothing in flight any more: [f4][lane]
        // sums, then [rows] maxima and [rows] sums of the weights.
        float *jm = reinterpret_cast<float *>(mine_at + C::f4 * 512);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int set = 0; set < SETS; ++set)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {  // elements 8 n + 4 f + (0 ... 3) of the set
                        const auto &a = acc[nt][set];
                        reinterpret_cast<float4 *>(mine_at)[(((nt * 2 + x) * SETS + set) * 2 + f) * 32 + lane] =
                            make_float4(a[2 * f][x], a[2 * f][2 + x], a[2 * f + 1][x], a[2 * f + 1][2 + x]);
                    }
                float sum = l[nt][x];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(kAllLanes, sum, o);
                if (n == 0) {
                    jm[8 * nt + 2 * quad + x] = m[nt][x];
                    jm[8 * NT + 8 * nt + 2 * quad + x] = sum;
                }
            }
        __syncthreads();
        for (int idx = tid; idx < C::f4 * 32; idx += W * 32) {
            const int ln = idx & 31, i = idx >> 5, f = i & 1, set = (i >> 1) % SETS, part = (i >> 1) / SETS;
            const int row = 8 * (part >> 1) + 2 * (ln & 3) + (part & 1), col = set * 64 + (ln >> 2) * 8 + 4 * f;
            if (row >= p.rows) continue;
            float mx = -CUDART_INF_F;
#pragma unroll
            for (int v = 0; v < W; ++v)
                mx = fmaxf(mx, reinterpret_cast<const float *>(smem + v * C::ring + C::f4 * 512)[row]);
            const float ref = mx == -CUDART_INF_F ? 0.f : mx;
            float ls = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int v = 0; v < W; ++v) {
                const float *jw = reinterpret_cast<const float *>(smem + v * C::ring + C::f4 * 512);
                const float4 y = reinterpret_cast<const float4 *>(smem + v * C::ring)[idx];
                const float g = ptx::ex2(jw[row] - ref);
                ls = fmaf(jw[8 * NT + row], g, ls);
                a.x = fmaf(y.x, g, a.x);
                a.y = fmaf(y.y, g, a.y);
                a.z = fmaf(y.z, g, a.z);
                a.w = fmaf(y.w, g, a.w);
            }
            int t, head;
            row_token(p, U, row, p.tpt, t, head);
            const bool valid = (rows_in >> row) & 1u;
            if (valid && (not_finite(ls) || not_finite(a.x + a.y + a.z + a.w))) *again = 1;
            if (U.split) {
                *reinterpret_cast<float4 *>(p.part_o + part_at<D>(p, U.slot, col >> 2, row)) = a;
                if (col == 0) p.part_ml[(size_t)U.slot * p.rows + row] = make_float2(mx, ls);
            } else if (t < p.m) {
                const float inv = valid && ls != 0.f ? 1.f / ls : 0.f;
                const bool on = inv != 0.f;
                uint2 o;
                o.x = on ? pack_bf16(a.x * inv, a.y * inv) : 0u;
                o.y = on ? pack_bf16(a.z * inv, a.w * inv) : 0u;
                *reinterpret_cast<uint2 *>(static_cast<bf16 *>(p.O) + (((size_t)U.b * p.Hq + head) * p.m + t) * D + col) = o;
            }
        }
        __syncthreads();
    }
    if (*again) rows_again<bf16, D, 1>(p, again + 4, warp, W);
}

template <int D, int NT, int W>
cudaError_t launch_few(const PagedProblem &p, cudaStream_t stream) {
    const size_t smem = Few<D, NT, W>::smem(p);
    static std::atomic<bool> done[64];
    auto kern = paged_few<D, NT, W>;
    cudaError_t e = allow_smem(kern, done, smem);
    if (e != cudaSuccess) return e;
    kern<<<p.slots, W * 32, smem, stream>>>(p);
    return cudaGetLastError();
}

template <int D, int NT, int W>
cudaError_t launch_few_w(const PagedProblem &p, cudaStream_t stream) {
    return p.warps == 4 ? launch_few<D, NT, 4>(p, stream) : launch_few<D, NT, W>(p, stream);
}

}  // namespace

cudaError_t launch_paged_few(const PagedProblem &p, cudaStream_t stream) {
    if (p.d == 64)
        return p.rows <= 8    ? launch_few_w<64, 1, 8>(p, stream)
               : p.rows <= 16 ? launch_few_w<64, 2, 8>(p, stream)
                              : launch_few_w<64, 3, 12>(p, stream);
    return p.rows <= 8    ? launch_few_w<128, 1, 8>(p, stream)
           : p.rows <= 16 ? launch_few_w<128, 2, 8>(p, stream)
                          : launch_few_w<128, 3, 8>(p, stream);
}

}  // namespace sa
