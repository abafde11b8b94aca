// Attention of a few new tokens per sequence over pages held in 4 bits, in tiles of 1 to 24
// rows per key head (rows = tokens x query heads of the key head), queries in bf16 or fp32:
// bf16 up to 3 or 4 such tiles, fp32 any number.
//
//     O_r = sum_j w_rj V_j / sum_j w_rj,   w_rj = 2^(s_rj - m_r),   s = q . k log2(e) / sqrt(d)
//
// Codes come to 9/16 byte per element, so at the memory's rate an SM has some 3
// thread instructions for each: the issue slots bound it as much as the memory
// does, and one multiply-add per element and row on the ordinary units would be too
// many already. So warp-level matrix instructions (m16n8k16, halves) do the
// products for any number of rows, keys or elements down, rows across:
//   S^T (16 x 8) = K Q^T, weights from S in registers, O^T (d x 8) += V^T P^T.
// Codes become halves by conversion instructions, two at a time (85 elements per
// clock and SM measured, with a product each), times their scale: both exact.
//   * The sum over d may run in any order: a lane's piece of a key row, as it lies in
//     memory, serves as its share of all steps of S; Q is held in the same order.
//   * The rows of O^T may stand in any order too: a lane takes d / 8 neighbouring
//     elements of four value rows. The keys of a matrix instruction are paired in its
//     registers: nibbles of two rows are sorted into bytes that hold one element of
//     both (4 instructions per 16 codes) and converted together. (Pages that hold two
//     tokens' codes in a byte would save these, and cost every append of a single token a read.)
//   * Queries in halves: each row times a power of two that brings its largest element to
//     2^13 ... 2^14, so bf16 numbers keep all their bits down to 2^-28 of that; fp32
//     ones are the sum of two halves (2^-22 of each, or 2^-38 of the largest). The
//     power of two leaves with the softmax's factor.
//   * Weights in halves: relative 2^-11, and 2^-32 of the largest; with fp32 queries the sum
//     of two (2^-22, and 2^-39). They are kept up to 2^15, so that small ones are far from a half's
//     smallest number: 2^7 at the reference, or 2^14 in fp32, where sums are rescaled as soon as a maximum
//     doubles the weights (1% of the time). Sums of weights and products are fp32, with fp32
//     queries rounded to the nearest every 16 keys.
// A warp takes 64 keys (d = 64) or 32 at a time (page numbers by 16) into a ring of its
// own by cp.async, whole pieces of 16 bytes, two items ahead. The pieces are
// stored so that neither the reads of K (a row per four lanes) nor those of V (four rows
// at once) meet in a bank.
// A key that no row sees has its value's scale zeroed, whatever memory holds there. A row
// that does not see a key multiplies its value by 0: where that value is NaN the row's sums
// come out so, and rows_again takes it again.
//
// Measured (16 sequences of 32768 keys, 8 key heads; the same over bf16 pages in brackets): d =
// 128, 1 to 4 rows 121 us, 5.0 TB/s (320), 16 rows 175 (324), 24 rows 218 (336); d = 64 74, 105 and
// 121 us (170, 175, 190), the first at 4.1 TB/s; fp32, 8 rows, d = 128 171 us. A plain copy: 6.8
// TB/s. 32 keys of one 8-row tile take 640 instructions at d = 128, 256 of them conversions and
// scales; two thirds of the issue slots are used, the rest is lost to results that are waited
// for (1.3 of 7 clocks a warp and issue), the conversions' pipe (1.0) and instructions on their way
// (1.2): there are 4 warps to a scheduler, as a lane's sums and queries take 128 registers. With
// 96 they spill, and with more of them L1 is too small: 20 warps 311 us. Smaller loop bodies (one
// tile of 16 keys at a time) need more instructions for the softmax and gain nothing; rows token by
// token, so that ragged drafts leave tiles of 8 out, gained nothing either: the full ones decide.
#pragma once

#include <type_traits>

#include "paged_common.cuh"

namespace sa {
namespace {


__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first of a chain: onto zeros.
__device__ __forceinline__ void mma16816_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                           uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 16 bytes from global to shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Transposes an 8 x 8 matrix of 16-bit numbers, two of a row per lane.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The lower four bits of each byte of a, the upper ones of b. (As one instruction.)
__device__ __forceinline__ uint32_t low_of(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, 0x0f0f0f0f, 0xe4;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <typename T, int D, int NT, int W>
struct Few4 {
    static constexpr int parts = sizeof(T) == 4 ? 2 : 1;     // halves to a query element, and to a weight
    static constexpr float grow = parts == 2 ? 1.f : 8.f;    // growth of a maximum (log2) that rescales the sums
    static constexpr float above = 15.f - grow;              // weights are 2^above at the reference, and up to 2^15
    static constexpr int ctas = paged_few4_ctas(D, 8 * NT, sizeof(T) == 4, W);  // per SM
    static constexpr int keys = D == 64 ? 64 : 32;           // a warp takes at a time
    static constexpr int codes = keys * D / 2, scales = keys * D / 16;
    static constexpr int item = 2 * (codes + scales);        // bytes: K codes, V codes, K scales, V scales
    static constexpr int stages = 2;                         // items in flight per warp
    static constexpr int f4 = NT * D / 16;                   // float4 of a lane's sums
    static constexpr int results = f4 * 512 + NT * 64;
    static constexpr int ring = stages * item > results ? stages * item : results;  // bytes per warp
    static size_t smem(const PagedProblem &p) {
        return (size_t)W * ring + sizeof(UnitRoom) + 16 + plan_bytes(p.B, p.ng, p.Hkv);
    }
};

// Where 16-byte piece c of key k's codes is stored. Rows of 64 bytes (d = 128) lie two to 128
// bytes, rows of 32 four; pieces of keys that are read together are moved apart.
template <int D>
__device__ __forceinline__ int piece_at(int k, int c) {
    if (D == 128) return (k >> 1) * 128 + ((((k & 1) << 2 | c) ^ (k & 2) ^ (k & 4)) << 4);
    return (k >> 2) * 128 + ((((k & 3) << 1 | c) ^ (k & 4)) << 4);
}

// A set of an item's keys.
template <int D>
using Keys = std::conditional_t<D == 64, uint64_t, uint32_t>;
__device__ __forceinline__ uint32_t or_lanes(uint32_t v) { return __reduce_or_sync(kAllLanes, v); }
__device__ __forceinline__ uint32_t and_lanes(uint32_t v) { return __reduce_and_sync(kAllLanes, v); }
__device__ __forceinline__ uint64_t or_lanes(uint64_t v) {
    return or_lanes((uint32_t)v) | (uint64_t)or_lanes((uint32_t)(v >> 32)) << 32;
}
__device__ __forceinline__ uint64_t and_lanes(uint64_t v) {
    return and_lanes((uint32_t)v) | (uint64_t)and_lanes((uint32_t)(v >> 32)) << 32;
}

template <typename T, int D, int NT, int W>
__global__ void __launch_bounds__(W * 32, Few4<T, D, NT, W>::ctas) paged_few4(const __grid_constant__ PagedProblem p) {
    using C = Few4<T, D, NT, W>;
    using M = Keys<D>;
    constexpr M kEvery = (M)~(M)0;
    constexpr int PARTS = C::parts;
    constexpr int KS = D / 16;           // k-steps of S, and tiles of O^T
    constexpr int PPK = D / 32;          // 16-byte pieces of a key's codes
    constexpr int WPL = D / 32;          // words of a lane's share of a key row
    constexpr int SUB = C::keys / 16;    // 16-key tiles of an item
    constexpr int PER = 64 / C::keys;    // items of a block
    extern __shared__ __align__(16) uint8_t smem[];
    UnitRoom *room = reinterpret_cast<UnitRoom *>(smem + W * C::ring);
    int *again = reinterpret_cast<int *>(room + 1);  // whether a row is to be taken again
    Plan P = plan_at(again + 4, p.B, p.ng, p.Hkv);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing is read before the launch in front has ended
    make_plan(p, P);
    asm volatile("griddepcontrol.launch_dependents;");  // the join may start planning
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = lane >> 2, quad = lane & 3;
    uint8_t *mine_at = smem + warp * C::ring;
    const uint32_t stage_at = ptx::smem_u32(mine_at);
    const size_t page_bytes = q4_page_bytes(p.page, D);
    // Row r of a 16-key tile is key 4 (r & 1) + (r >> 1 & 3) + (r & 8): the two keys of a
    // register are then 4 apart, and the four lanes of a row of the right operand
    // read four neighbours.
    const int my_key = 4 * (n & 1) + (n >> 1);
    // where the lane's pieces of codes go, 512 bytes (512 / (D / 2) keys) apart, and its piece of scales
    const uint32_t to_codes = piece_at<D>(lane / PPK, lane % PPK), to_scales = 2 * C::codes + lane * 16;
    const uint8_t *const scale_pool = static_cast<const uint8_t *>(lane < 16 ? p.K : p.V);

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
        // the queries first: on their way while pages are looked up
        constexpr int VE = 16 / sizeof(T), PC = D / 4 / VE;
        uint4 qw[NT][PC];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = 8 * nt + n;
            int t, head;
            row_token(p, U, row < p.rows ? row : 0, p.tpt, t, head);
            const uint4 *from = reinterpret_cast<const uint4 *>(
                static_cast<const T *>(p.Q) + (((size_t)U.b * p.Hq + head) * p.m + t) * D + quad * (D / 4));
#pragma unroll
            for (int c = 0; c < PC; ++c) {
                qw[nt][c] = make_uint4(0u, 0u, 0u, 0u);
                if ((rows_in >> row) & 1u) qw[nt][c] = __ldg(from + c);
            }
        }
        int full0 = 0, full1 = 0x7fffffff;  // blocks that every row sees whole
        if (mine.valid) {
            full0 = mine.glob ? 0 : mine.stride > 1 ? 0x7fffffff : (max(0, mine.pos - mine.reach) + 63) >> 6;
            full1 = (mine.pos + 1) >> 6;
        }
        full0 = __reduce_max_sync(kAllLanes, full0);
        full1 = __reduce_min_sync(kAllLanes, full1);
        const int i_end = PER * U.e1, hk = U.hk, n_glob = U.n_glob, far = U.lo_blk - U.n_glob;
        const int32_t *const pages = p.table + (size_t)U.b * p.max_pages;
        struct Item {
            int i, blk, pg;  // pg: page of the lane's 16 keys, from 16 (SUB lane / 32) on, as the table has it
        };
        auto item_at = [&](int i) -> Item {
            Item x = {i, 0, -1};
            if (i < i_end) {
                const int e = i / PER;
                x.blk = e < n_glob ? P.gblk[e] : far + e;
                const int c = ((x.blk << 6) + (i % PER) * C::keys + lane / (32 / SUB) * 16) >> p.log_page;
                if (c < p.max_pages) x.pg = __ldg(pages + c);
            }
            return x;
        };
        struct Masks {
            M w;         // the keys that the lane's row sees
            M any, all;  // keys that any row sees, and those that all see
        };
        // Starts the copies of an item.
        auto fetch = [&](Item x, int st) -> Masks {
            Masks k = {0, 0, 0};
            const bool whole = __all_sync(kAllLanes, (uint32_t)x.pg < (uint32_t)p.num_pages) && x.blk >= full0 && x.blk < full1;
            if (whole) {
                k.w = k.any = k.all = kEvery;
            } else {
                if (x.pg >= p.num_pages || x.pg < -1) {
                    atomicOr(p.status, kDevBadIndex);
                    x.pg = -1;
                }
                const unsigned have = __ballot_sync(kAllLanes, x.pg >= 0);
                M there = 0;
#pragma unroll
                for (int u = 0; u < SUB; ++u)
                    if ((have >> (u * (32 / SUB))) & 1u) there |= (M)0xffffu << (16 * u);
                if (have) {
                    k.w = (M)(row_mask(mine, x.blk, global_bits(P, p, x.blk), ~0ull) >> ((x.i % PER) * C::keys)) & there;
                    k.any = or_lanes(k.w);
                    k.all = and_lanes(mine.valid ? k.w : kEvery);
                }
            }
            __syncwarp();  // all lanes have read what the copies overwrite
            if (k.any) {
                const int j0 = (x.blk << 6) + (x.i % PER) * C::keys;
                const uint32_t to = stage_at + st * C::item;
                constexpr int PIECE_KEYS = 512 / (D / 2);  // keys of 32 lanes' pieces
                if (whole && p.page >= C::keys) {  // one run of codes, one of scales
                    const size_t base = ((size_t)__shfl_sync(kAllLanes, x.pg, 0) * p.Hkv + hk) * page_bytes;
                    const int in = j0 & (p.page - 1);
                    const size_t from = base + (in * (D / 2) + lane * 16);
                    const uint8_t *kp = static_cast<const uint8_t *>(p.K) + from, *vp = static_cast<const uint8_t *>(p.V) + from;
#pragma unroll
                    for (int i = 0; i < C::codes / 512; ++i) {
                        copy16(to + to_codes + i * 512, kp + i * 512);
                        copy16(to + to_codes + C::codes + i * 512, vp + i * 512);
                    }
                    copy16(to + to_scales, scale_pool + base + (p.page * (D / 2) + in * (D / 16) + (lane & 15) * 16));
                } else {
                    // 16 keys at a time; what no row sees is not read, and what the stage holds there is
                    // masked: a number for codes whatever it is, by its scale for values
#pragma unroll 1
                    for (int i = 0; i < C::codes / 512; ++i) {
                        const int key = i * PIECE_KEYS + lane / PPK, u = i * PIECE_KEYS / 16;
                        const int pg = __shfl_sync(kAllLanes, x.pg, u * (32 / SUB));
                        if (!((k.any >> key) & 1u)) continue;
                        const size_t from = ((size_t)pg * p.Hkv + hk) * page_bytes +
                                            (((j0 + key) & (p.page - 1)) * (D / 2) + lane % PPK * 16);
                        copy16(to + to_codes + i * 512, static_cast<const uint8_t *>(p.K) + from);
                        copy16(to + to_codes + C::codes + i * 512, static_cast<const uint8_t *>(p.V) + from);
                    }
                    constexpr int SPAN = 16 / (D / 16);  // keys of a piece of scales
                    const int key = (lane & 15) * SPAN;
                    const int pg = __shfl_sync(kAllLanes, x.pg, key / 16 * (32 / SUB));
                    if ((k.any >> key) & (M)((1u << SPAN) - 1u))
                        copy16(to + to_scales, scale_pool + (((size_t)pg * p.Hkv + hk) * page_bytes +
                                                             (p.page * (D / 2) + ((j0 + key) & (p.page - 1)) * (D / 16))));
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            return k;
        };
        Item next;
        Masks w[C::stages];  // of the items in flight, oldest first
        {
            Item x[C::stages + 1];
#pragma unroll
            for (int s = 0; s <= C::stages; ++s) x[s] = item_at(PER * U.e0 + warp + s * W);
#pragma unroll
            for (int s = 0; s < C::stages; ++s) w[s] = fetch(x[s], s);
            next = x[C::stages];
        }
        // Row 8 nt + n, elements D / 4 quad ..., as halves (zeros past the last row), and
        // the softmax's factor of rows 8 nt + 2 quad (+ 1).
        uint32_t q[NT][PARTS][D / 8];
        float sl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const auto &v = qw[nt];
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < PC; ++c)
#pragma unroll
                for (int x = 0; x < VE; ++x) top = fmaxf(top, fabsf(element<T>(v[c], x)));
            top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, 2));
            // 2^(13 - exponent of the largest), at most 2^120; as it is where there is none
            const int e = (int)(__float_as_uint(top) >> 23) - 127;
            const int up = top > 0.f && top <= 3.402823466e38f ? min(13 - e, 120) : 0;
            const float f = __uint_as_float((uint32_t)(127 + up) << 23), inv = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float a = element<T>(v[2 * i / VE], (2 * i) % VE) * f, b = element<T>(v[2 * i / VE], (2 * i + 1) % VE) * f;
                q[nt][0][i] = pack_half(a, b);
                if constexpr (PARTS == 2) {
                    const float2 h = half2_floats(q[nt][0][i]);
                    q[nt][1][i] = pack_half(a - h.x, b - h.y);
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) sl[nt][x] = p.scale_log2 * __shfl_sync(kAllLanes, inv, 4 * (2 * quad + x));
        }
        // sums of O^T: [x] is (element 2 t, row 2 quad), (2 t, 2 quad + 1), then those of 2 t + 1
        float acc[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                m[nt][x] = -CUDART_INF_F;
                l[nt][x] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < KS * 4; ++i) acc[nt][i / 4][i % 4] = 0.f;
        }
        if (tid == 0) fill_room(p, P, room, k ^ 1);  // while the first items are on their way
        __syncwarp();
        int st = 0;
#pragma unroll 1
        for (int i = PER * U.e0 + warp; i < i_end; i += W) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::stages - 1) : "memory");
            __syncwarp();
            const uint8_t *at = mine_at + st * C::item;
            const M any = w[0].any, all = w[0].all;
            if (any) {
                float s[SUB][NT][4];  // per 16 keys: rows n, n, n + 8, n + 8 of the tile for rows 2 quad, 2 quad + 1 in turn
#pragma unroll
                for (int u = 0; u < SUB; u += 2) {  // two tiles side by side: their sums are chains of products
                    uint32_t c[2][2][WPL], sc[2][2][2];  // the lane's words of two keys of each, their scales
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int v = i >> 1, h = i & 1, off = 16 * (u + v) + 8 * h, key = off + my_key;
                        const uint8_t *scale = at + 2 * C::codes + key * (D / 16);
                        if constexpr (D == 128) {
                            const uint4 t = *reinterpret_cast<const uint4 *>(at + piece_at<D>(my_key, quad) + off * (D / 2));
                            c[v][h][0] = t.x, c[v][h][1] = t.y, c[v][h][WPL - 2] = t.z, c[v][h][WPL - 1] = t.w;
                            const uint32_t b = *reinterpret_cast<const uint16_t *>(scale + quad * 2);
                            sc[v][h][0] = q4_scale2(b & 255u);
                            sc[v][h][1] = q4_scale2(b >> 8);
                        } else {
                            const uint2 t = *reinterpret_cast<const uint2 *>(at + piece_at<D>(my_key, quad >> 1) + off * (D / 2) +
                                                                             (quad & 1) * 8);
                            c[v][h][0] = t.x, c[v][h][1] = t.y;
                            sc[v][h][0] = sc[v][h][1] = q4_scale2(scale[quad]);
                        }
                    }
#pragma unroll
                    for (int x = 0; x < WPL; ++x)
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            uint32_t a[2][4];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                q4_halves(c[v][h][x], a[h]);
#pragma unroll
                                for (int j = 0; j < 4; ++j) a[h][j] = mul_half2(a[h][j], sc[v][h][x >> 1]);
                            }
#pragma unroll
                            for (int y = 0; y < 2; ++y)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int z = 0; z < PARTS; ++z) {
                                        float(&to)[4] = s[u + v][nt];
                                        const uint32_t b0 = q[nt][z][4 * x + 2 * y], b1 = q[nt][z][4 * x + 2 * y + 1];
                                        if (x + y + z == 0) mma16816_0(to, a[0][0], a[1][0], a[0][1], a[1][1], b0, b1);
                                        else mma16816(to, a[0][2 * y], a[1][2 * y], a[0][2 * y + 1], a[1][2 * y + 1], b0, b1);
                                    }
                        }
                }
                if (all != kEvery) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const M sees = __shfl_sync(kAllLanes, w[0].w, 8 * nt + 2 * quad + x) >> my_key;
#pragma unroll
                            for (int y = 0; y < 2 * SUB; ++y)  // keys my_key + 8 y
                                if (!((sees >> (8 * y)) & 1u)) s[y >> 1][nt][2 * (y & 1) + x] = -CUDART_INF_F;
                        }
                }
                float top[NT][2];  // sl > 0: the largest score is the largest sum's
                bool up = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float t = fmaxf(s[0][nt][x], s[0][nt][2 + x]);
#pragma unroll
                        for (int u = 1; u < SUB; ++u) t = ptx::fmax3(t, s[u][nt][x], s[u][nt][2 + x]);
                        top[nt][x] = t * sl[nt][x];
                        up |= top[nt][x] > m[nt][x] + C::grow;
                    }
                if (__any_sync(kAllLanes, up)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float f[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float mn = top[nt][x];
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(kAllLanes, mn, o));
                            mn = fmaxf(mn, m[nt][x]);
                            f[x] = mn == -CUDART_INF_F ? 0.f : ptx::ex2(m[nt][x] - mn);  // 0 from the initial -inf
                            m[nt][x] = mn;
                            l[nt][x] *= f[x];
                        }
#pragma unroll
                        for (int i = 0; i < KS * 4; ++i) acc[nt][i / 4][i % 4] *= f[i & 1];
                    }
                }
                uint32_t scale_v[SUB][2];  // the values' scales, those of two keys: quad + 8 h and 4 further on
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = 16 * u + 8 * h + quad;
                        const uint8_t *scale = at + 2 * C::codes + C::scales + key * (D / 16) + (D == 128 ? n : n >> 1);
                        scale_v[u][h] = (uint32_t)scale[0] * 0x80u + (uint32_t)scale[4 * (D / 16)] * 0x800000u;
                    }
                if (any != kEvery) {  // none for keys that no row sees
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t k = (uint32_t)(any >> (16 * u + 8 * h)) >> quad;
                            scale_v[u][h] &= (k & 1u ? 0xffffu : 0u) | (k & 16u ? 0xffff0000u : 0u);
                        }
                }
                uint32_t wt[SUB][NT][PARTS][2];  // weights as the right operand
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float ref[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) ref[x] = m[nt][x] == -CUDART_INF_F ? 0.f : C::above - m[nt][x];
                    const uint64_t sl2 = ptx::f2_pack(sl[nt][0], sl[nt][1]), ref2 = ptx::f2_pack(ref[0], ref[1]);
                    uint64_t sum = ptx::f2_pack(l[nt][0], l[nt][1]);
#pragma unroll
                    for (int y = 0; y < 2 * SUB; ++y) {
                        float &a = s[y >> 1][nt][2 * (y & 1)], &b = s[y >> 1][nt][2 * (y & 1) + 1];
                        ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(a, b), sl2, ref2), a, b);
                        a = ptx::ex2(a);
                        b = ptx::ex2(b);
                        sum = ptx::f2_add(sum, ptx::f2_pack(a, b));
                    }
                    ptx::f2_unpack(sum, l[nt][0], l[nt][1]);
#pragma unroll
                    for (int y = 0; y < 2 * SUB; ++y) {
                        const float a = s[y >> 1][nt][2 * (y & 1)], b = s[y >> 1][nt][2 * (y & 1) + 1];
                        const uint32_t v = pack_half(a, b);
                        wt[y >> 1][nt][0][y & 1] = transposed(v);
                        if constexpr (PARTS == 2) {
                            const float2 h = half2_floats(v);
                            wt[y >> 1][nt][1][y & 1] = transposed(pack_half(a - h.x, b - h.y));
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    // keys quad + 4 y of the 16: words of the lane's D / 8 elements
                    uint32_t c[4][WPL / 2];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        // piece_at of key 16 u + 4 y + quad, by parts that are constants
                        const uint8_t *v = at + C::codes + 16 * u * (D / 2) + (y >> 1) * 8 * (D / 2);
                        if constexpr (D == 128) {
                            const uint2 t = *reinterpret_cast<const uint2 *>(v + piece_at<D>(4 * (y & 1) + quad, n >> 1) + (n & 1) * 8);
                            c[y][0] = t.x, c[y][WPL / 2 - 1] = t.y;
                        } else {
                            c[y][0] = *reinterpret_cast<const uint32_t *>(v + piece_at<D>(4 * (y & 1) + quad, n >> 2) + (n & 3) * 4);
                        }
                    }
#pragma unroll
                    for (int x = 0; x < WPL / 2; ++x) {
                        uint32_t a[2][2][4];  // [pair of keys][even or odd element][byte]
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t ca = c[2 * h][x], cb = c[2 * h + 1][x];
                            q4_halves(low_of(ca, cb << 4), a[h][0]);
                            q4_halves(low_of(ca >> 4, cb), a[h][1]);
#pragma unroll
                            for (int j = 0; j < 8; ++j) a[h][j >> 2][j & 3] = mul_half2(a[h][j >> 2][j & 3], scale_v[u][h]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float(&to)[4] = acc[nt][4 * x + j];
                                if constexpr (PARTS == 2) {
                                    // Matrix instructions cut off what they do not hold, and long sums in them lean: 32768
                                    // keys were 75 u off (u = 2^-24; 12 u so, at 4% of the time, 14% for 16 rows at d =
                                    // 128, which spill). So they sum 16 keys, and those sums are added as floats are.
                                    float t[4];
                                    mma16816_0(t, a[0][0][j], a[0][1][j], a[1][0][j], a[1][1][j],
                                               wt[u][nt][0][0], wt[u][nt][0][1]);
                                    mma16816(t, a[0][0][j], a[0][1][j], a[1][0][j], a[1][1][j],
                                             wt[u][nt][1][0], wt[u][nt][1][1]);
#pragma unroll
                                    for (int i = 0; i < 4; i += 2)
                                        ptx::f2_unpack(ptx::f2_add(ptx::f2_pack(to[i], to[i + 1]), ptx::f2_pack(t[i], t[i + 1])),
                                                       to[i], to[i + 1]);
                                } else {
                                    mma16816(to, a[0][0][j], a[0][1][j], a[1][0][j], a[1][1][j],
                                             wt[u][nt][0][0], wt[u][nt][0][1]);
                                }
                            }
                    }
                }
            }
#pragma unroll
            for (int s = 0; s + 1 < C::stages; ++s) w[s] = w[s + 1];
            const Item x = next;
            next = item_at(i + (C::stages + 1) * W);
            w[C::stages - 1] = fetch(x, st);
            st = st + 1 == C::stages ? 0 : st + 1;
        }
        // Results into the warp's ring, which has nothing in flight any more: [f4][lane]
        // sums, then [rows] maxima and [rows] sums of the weights.
        float *jm = reinterpret_cast<float *>(mine_at + C::f4 * 512);
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int f = 0; f < KS / 2; ++f) {  // elements D / 8 n + 4 f + (0 ... 3)
                    const auto &a = acc[nt];
                    reinterpret_cast<float4 *>(mine_at)[((nt * 2 + x) * (KS / 2) + f) * 32 + lane] =
                        make_float4(a[2 * f][x], a[2 * f][2 + x], a[2 * f + 1][x], a[2 * f + 1][2 + x]);
                }
                float sum = l[nt][x];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(kAllLanes, sum, o);
                if (n == 0) {
                    jm[8 * nt + 2 * quad + x] = m[nt][x] - C::above;  // what the weights are relative to
                    jm[8 * NT + 8 * nt + 2 * quad + x] = sum;
                }
            }
        __syncthreads();
        for (int idx = tid; idx < C::f4 * 32; idx += W * 32) {
            const int ln = idx & 31, i = idx >> 5, f = i % (KS / 2), part = i / (KS / 2);
            const int row = 8 * (part >> 1) + 2 * (ln & 3) + (part & 1), col = (ln >> 2) * (D / 8) + 4 * f;
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
                T *out = static_cast<T *>(p.O) + (((size_t)U.b * p.Hq + head) * p.m + t) * D + col;
                if constexpr (sizeof(T) == 2) {
                    uint2 o;
                    o.x = on ? pack_bf16(a.x * inv, a.y * inv) : 0u;
                    o.y = on ? pack_bf16(a.z * inv, a.w * inv) : 0u;
                    *reinterpret_cast<uint2 *>(out) = o;
                } else {
                    *reinterpret_cast<float4 *>(out) = on ? make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv)
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
        }
        __syncthreads();
    }
    if (*again) rows_again<T, D, 1, true>(p, again + 4, warp, W);
}

template <typename T, int D, int NT, int W>
cudaError_t launch_few4(const PagedProblem &p, cudaStream_t stream) {
    const size_t smem = Few4<T, D, NT, W>::smem(p);
    static std::atomic<bool> done[64];
    auto kern = paged_few4<T, D, NT, W>;
    cudaError_t e = allow_smem(kern, done, smem);
    if (e != cudaSuccess) return e;
    return launch_behind(kern, dim3((unsigned)p.slots), W * 32, smem, stream, p);
}

template <typename T, int D, int NT>
cudaError_t launch_few4_w(const PagedProblem &p, cudaStream_t stream) {
    constexpr int W = paged_few4_ctas(D, 8 * NT, sizeof(T) == 4, 1) >= 16 ? 16 : 8;
    return p.warps == 4 ? launch_few4<T, D, NT, 4>(p, stream) : launch_few4<T, D, NT, W>(p, stream);
}

template <typename T, int D>
cudaError_t launch_few4_d(const PagedProblem &p, cudaStream_t stream) {
    if (p.rows <= 8) return launch_few4_w<T, D, 1>(p, stream);
    if (p.rows <= 16) return launch_few4_w<T, D, 2>(p, stream);
    if constexpr (sizeof(T) == 2 || D == 64) return launch_few4_w<T, D, 3>(p, stream);
    return cudaErrorNotSupported;
}

}  // namespace
}  // namespace sa
