// Attention of many new tokens over a paged cache on the ordinary units: the
// fp32 path, and bf16 where SA_OPT_FORCE_SIMT asks for a cross-check.
//
// A unit's 64 query rows (tokens x the query heads of one key head) walk the
// 64-key blocks that any of them sees. Scores and output are 8 x 4 register
// tiles of fp32 multiply-adds per thread: 32 multiply-adds for three 16-byte
// shared loads, so the multiply-add rate bounds it. Q and K are held
// transposed (the inner loop runs over d and reads four keys and eight rows at
// a time); V takes K's buffer once the scores are done, which leaves room for
// four CTAs per SM (d = 64; two at d = 128) to hide one another's loads and barriers:
// with three, 512 tokens over 8192 keys (2 sequences, 16 heads, d = 64, fp32) took 1458
// us, with four 1000 to 1020 us, 33 TFLOP/s of 75 that the multiply-adds allow (d = 128:
// 2690 us, 25 TFLOP/s). Rows in use matter: a unit is 64 rows whatever it holds.
// Global keys before a tile's window are gathered 64 to a step, wherever they lie;
// a step per block that holds one was half of all steps with 16 of them spread out.
#include "paged_common.cuh"

namespace sa {
namespace {

constexpr int kTR = 64;        // rows and keys of a tile
constexpr int kTT = 128;       // threads
constexpr int kPad = kTR + 4;  // row stride of the transposed arrays (16-byte aligned, off the banks' period)

template <typename T, int D>
struct TileSmem {
    static constexpr int Q = 0;
    static constexpr int KV = Q + D * kTR * 4;
    static constexpr int S = KV + (D * kPad > kTR * D ? D * kPad : kTR * D) * 4;
    static constexpr int MASK = S + kTR * kPad * 4;
    static constexpr int FLAG = MASK + kTR * 8;
    static constexpr int ROOM = FLAG + 16;
    static constexpr int PLAN = ROOM + (int)sizeof(UnitRoom);
};

template <typename T, int D>
__global__ void __launch_bounds__(kTT, D == 64 ? 4 : 2) paged_tile(const __grid_constant__ PagedProblem p) {
    using L = TileSmem<T, D>;
    constexpr int VE = 16 / sizeof(T);
    constexpr int ND = D / 64;  // 4-wide output columns per thread
    extern __shared__ __align__(16) uint8_t smem[];
    float *Qs = reinterpret_cast<float *>(smem + L::Q);    // [D][64]
    float *KV = reinterpret_cast<float *>(smem + L::KV);   // K: [D][kPad], then V: [64][D]
    float *Ps = reinterpret_cast<float *>(smem + L::S);    // [key][kPad rows]
    uint64_t *masks = reinterpret_cast<uint64_t *>(smem + L::MASK);
    int *flags = reinterpret_cast<int *>(smem + L::FLAG);  // which keys are there (2), whether a row is to be taken again
    Plan P = plan_at(smem + L::PLAN, p.B, p.ng, p.Hkv);
    make_plan(p, P);
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ty = tid >> 4, tx = tid & 15;  // rows ty * 8 ..., keys and columns tx * 4 ...
    const T *Kp = static_cast<const T *>(p.K), *Vp = static_cast<const T *>(p.V);

    UnitRoom *room = reinterpret_cast<UnitRoom *>(smem + L::ROOM);
    if (tid == 0) {
        flags[2] = 0;
        room->units.begin(p, P, blockIdx.x);
        fill_room(p, P, room, 0);
    }
    __syncthreads();
    for (int room_k = 0; room->more[room_k]; room_k ^= 1) {
        const Unit &U = room->U[room_k];
        // threads 0..63: one row each, for the masks
        Row row = {};
        if (tid < kTR) {
            int t = 0, head = 0;
            if (tid < p.rows) {
                row_token(p, U, tid, p.tpt_half, t, head);
                row = make_row(p, P, U, head, t);
            }
        }
        // queries, transposed and scaled; a lane per row
        for (int i = tid; i < kTR * (D / VE); i += kTT) {
            const int r = i % kTR, c = i / kTR;
            int t, head;
            row_token(p, U, r < p.rows ? r : 0, p.tpt_half, t, head);
            const bool ok = U.live && r < p.rows && t < U.q;
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (ok)
                w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.Q) +
                                                          (((size_t)U.b * p.Hq + head) * p.m + t) * D + c * VE));
#pragma unroll
            for (int k = 0; k < VE; ++k) Qs[(c * VE + k) * kTR + r] = element<T>(w, k) * p.scale_log2;
        }
        float acc[8][4 * ND], m[8], l[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            m[r] = -CUDART_INF_F;
            l[r] = 0.f;
#pragma unroll
            for (int x = 0; x < 4 * ND; ++x) acc[r][x] = 0.f;
        }
        if (tid == kTT - 1) fill_room(p, P, room, room_k ^ 1);  // a warp without masks to work out
        const int far = far_globals(p, P, U);
        for (int e = U.e0; e < U.e1; ++e) {
            const bool listed = e < U.n_glob;  // 64 of the far global keys, which every row sees
            const int blk = listed ? 0 : entry_block(P, U, e), j0 = blk << 6;
            __syncthreads();  // the previous step is done with KV, Ps and masks
            if (tid < kTR)
                masks[tid] = !listed ? row_mask(row, blk, global_bits(P, p, blk), ~0ull)
                             : row.valid ? low_bits(far - 64 * e) : 0ull;
            // one key per lane: keys past the sequence or without a page count as
            // zeros and are masked below
            const int key = tid & 63;
            const int pos = !listed ? j0 + key : 64 * e + key < far ? P.gpos[64 * e + key] : U.s;
            const int pg = pos < U.s ? page_of(p, U.b, pos) : -1;
            const size_t at = ((((size_t)(pg < 0 ? 0 : pg) * p.Hkv + U.hk) << p.log_page) + (pos & (p.page - 1))) * D;
#pragma unroll 4
            for (int c = tid >> 6; c < D / VE; c += kTT / 64) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (pg >= 0) w = __ldg(reinterpret_cast<const uint4 *>(Kp + at + c * VE));
    #pragma unroll
                for (int k = 0; k < VE; ++k) KV[(c * VE + k) * kPad + key] = element<T>(w, k);
            }
            const unsigned there = __ballot_sync(kAllLanes, pg >= 0);  // of keys 32 (warp & 1) ...
            if (warp < 2 && lane == 0) flags[warp] = (int)there;
            __syncthreads();
            const uint64_t present = (uint32_t)flags[0] | ((uint64_t)(uint32_t)flags[1] << 32);
            float s[8][4];
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[r][x] = 0.f;
#pragma unroll 4
            for (int k = 0; k < D; ++k) {
                const float4 a0 = *reinterpret_cast<const float4 *>(Qs + k * kTR + ty * 8);
                const float4 a1 = *reinterpret_cast<const float4 *>(Qs + k * kTR + ty * 8 + 4);
                const float4 b = *reinterpret_cast<const float4 *>(KV + k * kPad + tx * 4);
                const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    s[r][0] = fmaf(a[r], b.x, s[r][0]);
                    s[r][1] = fmaf(a[r], b.y, s[r][1]);
                    s[r][2] = fmaf(a[r], b.z, s[r][2]);
                    s[r][3] = fmaf(a[r], b.w, s[r][3]);
                }
            }
            __syncthreads();  // K is done with
            {
                // V rows as they are: a warp per key row piece
                for (int i = tid; i < kTR * (D / VE); i += kTT) {
                    const int vk = i / (D / VE), c = i % (D / VE);
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if ((present >> vk) & 1ull) {
                        const int vpos = listed ? P.gpos[64 * e + vk] : j0 + vk;
                        const int vpg = page_of(p, U.b, vpos);
                        w = __ldg(reinterpret_cast<const uint4 *>(
                            Vp + ((((size_t)vpg * p.Hkv + U.hk) << p.log_page) + (vpos & (p.page - 1))) * D + c * VE));
                    }
        #pragma unroll
                    for (int k = 0; k < VE; ++k) KV[vk * D + c * VE + k] = element<T>(w, k);
                }
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const uint32_t w = (uint32_t)((masks[ty * 8 + r] & present) >> (tx * 4)) & 15u;
                float mn = m[r];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (!((w >> x) & 1u)) s[r][x] = -CUDART_INF_F;
                    mn = fmaxf(mn, s[r][x]);
                }
#pragma unroll
                for (int o = 8; o; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(kAllLanes, mn, o));
                const float ref = mn == -CUDART_INF_F ? 0.f : mn;
                const float f = ptx::ex2(m[r] - ref);
                m[r] = mn;
                float sum = 0.f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    s[r][x] = ptx::ex2(s[r][x] - ref);
                    sum += s[r][x];
                }
                l[r] = l[r] * f + sum;  // this thread's keys; joined at the end
#pragma unroll
                for (int x = 0; x < 4 * ND; ++x) acc[r][x] *= f;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float *dst = Ps + (tx * 4 + x) * kPad + ty * 8;
                *reinterpret_cast<float4 *>(dst) = make_float4(s[0][x], s[1][x], s[2][x], s[3][x]);
                *reinterpret_cast<float4 *>(dst + 4) = make_float4(s[4][x], s[5][x], s[6][x], s[7][x]);
            }
            __syncthreads();
#pragma unroll 4
            for (int k = 0; k < kTR; ++k) {
                const float4 a0 = *reinterpret_cast<const float4 *>(Ps + k * kPad + ty * 8);
                const float4 a1 = *reinterpret_cast<const float4 *>(Ps + k * kPad + ty * 8 + 4);
                const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                for (int h = 0; h < ND; ++h) {
                    const float4 b = *reinterpret_cast<const float4 *>(KV + k * D + h * 64 + tx * 4);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        acc[r][h * 4 + 0] = fmaf(a[r], b.x, acc[r][h * 4 + 0]);
                        acc[r][h * 4 + 1] = fmaf(a[r], b.y, acc[r][h * 4 + 1]);
                        acc[r][h * 4 + 2] = fmaf(a[r], b.z, acc[r][h * 4 + 2]);
                        acc[r][h * 4 + 3] = fmaf(a[r], b.w, acc[r][h * 4 + 3]);
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
#pragma unroll
            for (int o = 8; o; o >>= 1) l[r] += __shfl_xor_sync(kAllLanes, l[r], o);
            const int rr = ty * 8 + r;
            if (rr >= p.rows) continue;
            int t, head;
            row_token(p, U, rr, p.tpt_half, t, head);
            const bool valid = U.live && t < U.q;
            bool bad = not_finite(l[r]);
#pragma unroll
            for (int x = 0; x < 4 * ND; ++x) bad |= not_finite(acc[r][x]);
            if (bad && valid) flags[2] = 1;
            if (U.split) {
#pragma unroll
                for (int h = 0; h < ND; ++h)
                    *reinterpret_cast<float4 *>(p.part_o + part_at<D>(p, U.slot, h * 16 + tx, rr)) =
                        make_float4(acc[r][h * 4], acc[r][h * 4 + 1], acc[r][h * 4 + 2], acc[r][h * 4 + 3]);
                if (tx == 0) p.part_ml[(size_t)U.slot * p.rows + rr] = make_float2(m[r], l[r]);
            } else if (t < p.m) {
                T *o = static_cast<T *>(p.O) + (((size_t)U.b * p.Hq + head) * p.m + t) * D;
                const float inv = valid && l[r] != 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
                for (int h = 0; h < ND; ++h)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        o[h * 64 + tx * 4 + x] = from_float<T>(valid ? acc[r][h * 4 + x] * inv : 0.f);
            }
        }
        __syncthreads();  // every warp is done with the unit
    }
    if (flags[2]) rows_again<T, D, 4>(p, smem + L::PLAN, warp, kTT / 32);
}

template <typename T, int D>
cudaError_t launch_tile(const PagedProblem &p, cudaStream_t stream) {
    const size_t smem = TileSmem<T, D>::PLAN + plan_bytes(p.B, p.ng, p.Hkv);
    static std::atomic<bool> done[64];
    auto kern = paged_tile<T, D>;
    cudaError_t e = allow_smem(kern, done, smem);
    if (e != cudaSuccess) return e;
    kern<<<p.slots, kTT, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tile(const PagedProblem &p, sa_dtype dtype, cudaStream_t stream) {
    if (dtype == SA_FP32)
        return p.d == 64 ? launch_tile<float, 64>(p, stream) : launch_tile<float, 128>(p, stream);
    return p.d == 64 ? launch_tile<__nv_bfloat16, 64>(p, stream)
                     : launch_tile<__nv_bfloat16, 128>(p, stream);
}

}  // namespace sa
