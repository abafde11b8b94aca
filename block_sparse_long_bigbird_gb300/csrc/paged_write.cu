// Appending to a paged cache with the rotation of positions on the way, into pages of
// the new rows' type or of 4 bits, and reading 4-bit pages back.
//
// Rotation: a pair (a, b) of a row at position p becomes (a c - b s, b c + a s), with c, s
// from row p of the caller's tables. Scales and codes of 4-bit pages (paged_q4.cuh), per
// group of 16 elements: scale = max |x| / 6 rounded to the scale's 4 significant bits, at
// most 10240; code = x / scale rounded to the nearest of the eight values; halfway cases to the
// even code, in both.
//
// A thread takes eight pairs of a row, two 16-byte pieces of bf16, and the same ones of
// several heads, so that it reads its angles once for all of them. New keys, values and
// queries are one launch.
//
// Measured (up to 4096 new tokens of 4 sequences, 32 query and 8 key heads of 128, bf16: 327 MB
// with the zeros behind ragged chunks): rotated 52 us, 6.3 TB/s (a plain copy: 6.8): the memory.
// Into 4-bit pages 71 us, 4.1 TB/s: rotating exactly and choosing codes take as many instructions
// as all else, 61% of the issue slots are used. Read back 17 us; 131072 rows of 128 with a third of
// them zeros 54 us, 5.7 TB/s. A single token of 64 sequences 4.5 and 5.2 us: launch. fp32: rotated 108 us
// (574 MB and zeros), into 4-bit pages 99; those 131072 rows as fp32 135 us (586 MB: a row's codes come in pieces
// of 4 bytes, the rows leave in pieces of 32), from plain pages 69 in bf16 (6.5 TB/s) and 144 in fp32 (6.2).
#include <cuda_bf16.h>

#include "internal.h"
#include "paged.h"
#include "paged_q4.cuh"

namespace sa {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWriteThreads = 128;

// a c - b s. fp32 rows: off by two roundings of the result, whatever cancels (Kahan's difference of
// products). bf16 rows: the product b s rounded to fp32 first, 2^-24 of it, is far below what is rounded off then.
template <typename T>
__device__ __forceinline__ float turn(float a, float c, float b, float s) {
    const float w = b * s, r = fmaf(a, c, -w);
    if (sizeof(T) == 2) return r;
    const float e = fmaf(b, s, -w);
    return r - (e == e ? e : 0.f);  // an infinite w has no error
}

// The same to fp32's last place (of a sum good to 2^-46: products and the difference
// with their rounding errors kept; Dekker, Knuth), and what is left over.
__device__ __forceinline__ float turn_exact(float a, float c, float b, float s, float &rest) {
    const float h = __fmul_rn(a, c), t = fmaf(a, c, -h);
    const float w = __fmul_rn(b, s), u = fmaf(b, s, -w);
    const float d = __fsub_rn(h, w), bb = __fsub_rn(d, h);
    const float e = __fsub_rn(__fsub_rn(h, __fsub_rn(d, bb)), __fadd_rn(w, bb));
    const float lo = __fadd_rn(e, __fsub_rn(t, u));
    const float r = __fadd_rn(d, lo);
    rest = __fsub_rn(lo, __fsub_rn(r, d));
    return r;
}

// Whether r's rounding to T depends on what is left over: halfway between two bf16 numbers.
template <typename T>
__device__ __forceinline__ bool halfway(float r) {
    return sizeof(T) == 2 && (__float_as_uint(r) & 0xffffu) == 0x8000u;
}

// Rounded once to the type of the new rows, as a float: what a code is chosen for. (By way of
// fp32 one number in 2^17 would come out differently, and one code in some millions.)
template <typename T>
__device__ __forceinline__ float rounded(float r) {
    return sizeof(T) == 2 ? __bfloat162float(__float2bfloat16_rn(r)) : r;
}
template <typename T>
__device__ __forceinline__ float rounded(float r, float rest) {
    if (halfway<T>(r) && rest != 0.f) r = __uint_as_float(__float_as_uint(r) + ((rest > 0.f) == (r > 0.f) ? 1u : ~0u));
    return rounded<T>(r);
}

// Eight pairs, exactly. Hardly ever is one halfway: then all of them again, with what is left over.
template <typename T, bool INTER>
__device__ __forceinline__ void turn8_exact(float (&va)[8], float (&vb)[8], const float (&c)[8], const float (&sn)[8]) {
    float ra[8], rb[8], rest;
    bool again = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float u = INTER ? (k < 4 ? va[2 * k & 7] : vb[2 * k & 7]) : va[k];
        const float v = INTER ? (k < 4 ? va[(2 * k + 1) & 7] : vb[(2 * k + 1) & 7]) : vb[k];
        ra[k] = turn_exact(u, c[k], v, sn[k], rest);
        rb[k] = turn_exact(v, c[k], u, -sn[k], rest);
        again |= halfway<T>(ra[k]) | halfway<T>(rb[k]);
    }
    if (again) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float u = INTER ? (k < 4 ? va[2 * k & 7] : vb[2 * k & 7]) : va[k];
            const float v = INTER ? (k < 4 ? va[(2 * k + 1) & 7] : vb[(2 * k + 1) & 7]) : vb[k];
            ra[k] = turn_exact(u, c[k], v, sn[k], rest);
            ra[k] = rounded<T>(ra[k], rest);
            rb[k] = turn_exact(v, c[k], u, -sn[k], rest);
            rb[k] = rounded<T>(rb[k], rest);
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (INTER) {
            (k < 4 ? va[2 * k & 7] : vb[2 * k & 7]) = rounded<T>(ra[k]);
            (k < 4 ? va[(2 * k + 1) & 7] : vb[(2 * k + 1) & 7]) = rounded<T>(rb[k]);
        } else {
            va[k] = rounded<T>(ra[k]);
            vb[k] = rounded<T>(rb[k]);
        }
    }
}

template <typename T, bool INTER>
__device__ __forceinline__ void turn8(float (&va)[8], float (&vb)[8], const float (&c)[8], const float (&sn)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float &u = INTER ? (k < 4 ? va[2 * k & 7] : vb[2 * k & 7]) : va[k];
        float &v = INTER ? (k < 4 ? va[(2 * k + 1) & 7] : vb[(2 * k + 1) & 7]) : vb[k];
        const float y = turn<T>(u, c[k], v, sn[k]);
        v = turn<T>(v, c[k], u, -sn[k]);
        u = y;
    }
}

// Eight consecutive elements of a row.
template <typename T>
struct Eight {
    uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const void *base, size_t at) {
    Eight<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(base) + at) + i);
    return r;
}
template <typename T>
__device__ __forceinline__ void floats8(const Eight<T> &v, float (&o)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 &q = v.w[sizeof(T) == 2 ? 0 : i >> 2];
        const int k = sizeof(T) == 2 ? i >> 1 : i & 3;
        const uint32_t w = k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w;
        o[i] = __uint_as_float(sizeof(T) == 4 ? w : i & 1 ? w & 0xffff0000u : w << 16);
    }
}
template <typename T>
__device__ __forceinline__ Eight<T> pack8(const float (&v)[8]) {
    Eight<T> r;
    uint32_t w[sizeof(T) * 2];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) * 2; ++i) {
        if (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
        else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[(2 * i + 1) & 7]), "f"(v[(2 * i) & 7]));
    }
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    return r;
}
template <typename T>
__device__ __forceinline__ void store8(void *base, size_t at, const Eight<T> &v) {
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(base) + at);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) out[i] = v.w[i];
}
template <typename T>
__device__ __forceinline__ void store8(void *base, size_t at, const float (&v)[8]) {
    store8<T>(base, at, pack8<T>(v));
}

// max |x| of eight numbers, NaN if one is NaN.
__device__ __forceinline__ float top8(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[i])));
    return m;
}

// x / y for a y of few bits and r near 1 / y: a product, corrected by its remainder, which is exact
// (Markstein 1990). Good to 2^-45 before its last rounding: halfway between two numbers of few bits only
// where x / y is, as no other fp32 x comes nearer to such a place times y than half of a quotient's unit.
__device__ __forceinline__ float quotient(float x, float y, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, y, x), r, q);
}

// The scale byte of a group whose largest magnitude is `top`.
__device__ __forceinline__ uint32_t scale_byte(float top) {
    if (!(top <= 3.402823466e38f)) return 255u;
    const float s = fminf(quotient(top, 6.f, 1.f / 6.f), 10240.f);
    const uint32_t b = __float_as_uint(s), normal = ((b + 0x7ffffu + ((b >> 20) & 1u)) >> 20) - (112u << 3);
    return s < 6.103515625e-5f ? (uint32_t)__float2int_rn(s * 131072.f) : normal;  // below: multiples of 2^-17
}

// Eight codes, by the nearest of their eight values to x / scale.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], uint32_t byte) {
    const float s = q4_scale(byte);
    float r, q[8];
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = byte == 0u ? 0.f : r;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], s, r);
    uint32_t w;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return w;
}

// Which elements thread `x` of a row's D / 16 holds: eight from `a` on and eight from `b` on.
// Rotated pairs come first: (8 x + i, rot / 2 + 8 x + i), or 16 consecutive elements in
// neighbouring pairs; then what is not rotated.
__device__ __forceinline__ void pieces_of(int x, int rot, bool inter, int &a, int &b) {
    const bool turned = 16 * x < rot;
    a = turned && !inter ? 8 * x : 16 * x;
    b = turned && !inter ? rot / 2 + 8 * x : 16 * x + 8;
}

// Of the Hkv keys, Hkv values and Hq queries laid end to end a CTA takes every gridDim.y-th head, so that
// each gets its share of every kind; threads take (sequence, token, eight pairs) and request
// the next head's elements before they work on one's.
template <typename T, int D, bool P4, bool INTER>
__global__ void __launch_bounds__(kWriteThreads, P4 ? 6 : 7) cache_write(const WriteProblem p) {
    constexpr int TPR = D / 16;  // threads of a row
    asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing is read before the launch in front has ended
    const int lane = threadIdx.x & 31;
    const int x = lane % TPR, first = lane - x;  // place in the row; the row's first lane
    const int rot = p.rot;
    const bool turned = 16 * x < rot;
    int pa, pb;
    pieces_of(x, rot, INTER, pa, pb);
    // 4 bits: the other half of a group of 16 elements may be any lane's first or second eight
    int la = 0, lb = 0;
    bool sa2 = false, sb2 = false;  // whether it is that lane's second eight
    if (P4) {
        for (int y = 0; y < TPR; ++y) {
            int qa, qb;
            pieces_of(y, rot, INTER, qa, qb);
            if (qa == (pa ^ 8)) la = first + y, sa2 = false;
            if (qb == (pa ^ 8)) la = first + y, sa2 = true;
            if (qa == (pb ^ 8)) lb = first + y, sb2 = false;
            if (qb == (pb ^ 8)) lb = first + y, sb2 = true;
        }
    }
    const long long total = (long long)p.B * p.m * TPR;
    for (long long i = (long long)blockIdx.x * kWriteThreads + threadIdx.x; i - lane < total;
         i += (long long)gridDim.x * kWriteThreads) {
        const bool in = i < total;
        const long long bt = (in ? i : total - 1) / TPR;
        const int b = (int)(bt / p.m), t = (int)(bt - (long long)b * p.m);
        int q = p.qlens ? __ldg(p.qlens + b) : p.m;
        const int s = __ldg(p.lens + b);
        if (q < 0 || q > p.m || s < q || (long long)s > ((long long)p.max_pages << p.log_page)) {
            if (in) atomicOr(p.status, kDevBadIndex);
            q = 0;
        }
        const int pos = s - q + t;
        bool live = in && t < q;
        int pg = -1;
        if (live && rot && pos >= p.rope_len) {  // no angles for it
            atomicOr(p.status, kDevBadIndex);
            live = false;
        }
        if (live) {
            pg = __ldg(p.table + (size_t)b * p.max_pages + (pos >> p.log_page));
            if (pg < 0 || pg >= p.num_pages) {  // nowhere to write the token
                atomicOr(p.status, kDevBadIndex);
                pg = -1;
            }
        }
        float c[8], sn[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            c[k] = 1.f;
            sn[k] = 0.f;
        }
        if (live && turned) {
            const float4 *cp = reinterpret_cast<const float4 *>(p.cos + (size_t)pos * (rot / 2) + 8 * x);
            const float4 *sp = reinterpret_cast<const float4 *>(p.sin + (size_t)pos * (rot / 2) + 8 * x);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 u = __ldg(cp + k), v = __ldg(sp + k);
                c[4 * k] = u.x, c[4 * k + 1] = u.y, c[4 * k + 2] = u.z, c[4 * k + 3] = u.w;
                sn[4 * k] = v.x, sn[4 * k + 1] = v.y, sn[4 * k + 2] = v.z, sn[4 * k + 3] = v.w;
            }
        }
        const int gy = (int)gridDim.y;
        // Heads h, h + gy, ... before `end` of one kind, rows of `from`; `done` gets each head's number and elements
        // (as they are: what is not rotated or coded keeps its bits, those of a NaN too).
        auto heads_of = [&](const void *from, int H, int h, int end, bool take, auto done) {
            Eight<T> na = {}, nb = {};
            const T *at = static_cast<const T *>(from) + (((size_t)b * H + h) * p.m + t) * D;
            const size_t step = (size_t)gy * p.m * D;
            if (take && h < end) {
                na = load8<T>(at, pa);
                nb = load8<T>(at, pb);
            }
#pragma unroll 1
            for (; h < end; h += gy) {
                const Eight<T> ea = na, eb = nb;
                at += step;
                if (take && h + gy < end) {
                    na = load8<T>(at, pa);
                    nb = load8<T>(at, pb);
                }
                done(h, ea, eb);
            }
        };
        const bool there = live && pg >= 0;
        const size_t page_at = there ? (size_t)pg * p.Hkv : 0;
        const int in_page = pos & (p.page - 1);
        auto put = [&](void *pool, int h, Eight<T> ea, Eight<T> eb, bool turn) {
            const size_t row = ((page_at + h) << p.log_page) + in_page;
            float va[8], vb[8];
            if constexpr (P4) {
                floats8<T>(ea, va);
                floats8<T>(eb, vb);
                if (turn) turn8_exact<T, INTER>(va, vb, c, sn);
                const float ta = top8(va), tb = top8(vb);
                const float a1 = __shfl_sync(kAll, ta, la), a2 = __shfl_sync(kAll, tb, la);
                const float b1 = __shfl_sync(kAll, ta, lb), b2 = __shfl_sync(kAll, tb, lb);
                float ga = sa2 ? a2 : a1, gb = sb2 ? b2 : b1;
                asm("max.NaN.f32 %0, %0, %1;" : "+f"(ga) : "f"(ta));
                asm("max.NaN.f32 %0, %0, %1;" : "+f"(gb) : "f"(tb));
                const uint32_t sa = scale_byte(ga), sb = scale_byte(gb);
                const uint32_t wa = codes8(va, sa), wb = codes8(vb, sb);
                if (!there) return;
                const Q4At at = q4_row<D>(row, p.page, p.log_page);
                uint8_t *bytes = static_cast<uint8_t *>(pool);
                *reinterpret_cast<uint32_t *>(bytes + at.codes + pa / 2) = wa;
                *reinterpret_cast<uint32_t *>(bytes + at.codes + pb / 2) = wb;
                if (!(pa & 8)) bytes[at.scales + pa / 16] = (uint8_t)sa;
                if (!(pb & 8)) bytes[at.scales + pb / 16] = (uint8_t)sb;
            } else if (there) {
                if (turn) {
                    floats8<T>(ea, va);
                    floats8<T>(eb, vb);
                    turn8<T, INTER>(va, vb, c, sn);
                    ea = pack8<T>(va);
                    eb = pack8<T>(vb);
                }
                store8<T>(pool, row * D + pa, ea);
                store8<T>(pool, row * D + pb, eb);
            }
        };
        int h = blockIdx.y;
        heads_of(p.Kn, p.Hkv, h, p.Hkv, there,
                 [&](int k, const Eight<T> &ea, const Eight<T> &eb) { put(p.K, k, ea, eb, turned); });
        while (h < p.Hkv) h += gy;
        h -= p.Hkv;
        heads_of(p.Vn, p.Hkv, h, p.Hkv, there,
                 [&](int k, const Eight<T> &ea, const Eight<T> &eb) { put(p.V, k, ea, eb, false); });
        while (h < p.Hkv) h += gy;
        h -= p.Hkv;
        if (!in) continue;
        heads_of(p.Qn, p.Hq, h, p.Hq, live, [&](int k, Eight<T> ea, Eight<T> eb) {
            if (turned) {
                float va[8], vb[8];
                floats8<T>(ea, va);
                floats8<T>(eb, vb);
                turn8<T, INTER>(va, vb, c, sn);
                ea = pack8<T>(va);
                eb = pack8<T>(vb);
            }
            const size_t dst = (((size_t)b * p.Hq + k) * p.m + t) * D;
            store8<T>(p.Qo, dst + pa, ea);
            store8<T>(p.Qo, dst + pb, eb);
        });
    }
}

// ------------------------------------------------------------------ reading
// Rows [B][Hkv][m][D] of the tokens [lens - q, lens): a thread takes eight elements of
// kReadRows rows each of K and V, all requested before the first is stored. Rows
// past q, and tokens whose page is missing, are zeros.
constexpr int kReadThreads = 256, kReadRows = 4;

template <typename T, int D, bool P4>
__global__ void __launch_bounds__(kReadThreads) cache_read(const WriteProblem p) {
    constexpr int TPR = D / 8;  // threads of a row
    constexpr int RPB = kReadThreads / TPR;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int x = threadIdx.x % TPR;
    for (long long bh = blockIdx.y; bh < (long long)p.B * p.Hkv; bh += gridDim.y) {
        const int h = (int)(bh % p.Hkv), b = (int)(bh / p.Hkv);
        int q = p.qlens ? __ldg(p.qlens + b) : p.m;
        const int s = __ldg(p.lens + b);
        if (q < 0 || q > p.m || s < q || (long long)s > ((long long)p.max_pages << p.log_page)) {
            if (threadIdx.x == 0) atomicOr(p.status, kDevBadIndex);
            q = 0;
        }
        const int32_t *trow = p.table + (size_t)b * p.max_pages;
        for (long long t0 = (long long)blockIdx.x * (RPB * kReadRows) + threadIdx.x / TPR; t0 < p.m;
             t0 += (long long)gridDim.x * (RPB * kReadRows)) {
            Eight<T> kw[kReadRows], vw[kReadRows];   // of ordinary pages
            uint32_t kc[kReadRows], vc[kReadRows], ks[kReadRows], vs[kReadRows];
#pragma unroll
            for (int r = 0; r < kReadRows; ++r) {
                const long long t = t0 + r * RPB;
                kc[r] = vc[r] = ks[r] = vs[r] = 0u;
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; ++i) kw[r].w[i] = vw[r].w[i] = make_uint4(0u, 0u, 0u, 0u);
                if (t >= q) continue;
                const int pos = s - q + (int)t;
                const int pg = __ldg(trow + (pos >> p.log_page));
                if (pg < 0 || pg >= p.num_pages) {
                    if (pg != -1) atomicOr(p.status, kDevBadIndex);
                    continue;
                }
                const size_t row = (((size_t)pg * p.Hkv + h) << p.log_page) + (pos & (p.page - 1));
                if constexpr (P4) {
                    const Q4At at = q4_row<D>(row, p.page, p.log_page);
                    const uint8_t *K = static_cast<const uint8_t *>(p.K), *V = static_cast<const uint8_t *>(p.V);
                    kc[r] = __ldcs(reinterpret_cast<const uint32_t *>(K + at.codes) + x);
                    vc[r] = __ldcs(reinterpret_cast<const uint32_t *>(V + at.codes) + x);
                    ks[r] = __ldg(K + at.scales + x / 2);
                    vs[r] = __ldg(V + at.scales + x / 2);
                } else {
                    kw[r] = load8<T>(p.K, row * D + x * 8);
                    vw[r] = load8<T>(p.V, row * D + x * 8);
                }
            }
#pragma unroll
            for (int r = 0; r < kReadRows; ++r) {
                const long long t = t0 + r * RPB;
                if (t >= p.m) continue;
                const size_t dst = ((size_t)bh * p.m + (size_t)t) * D + x * 8;
                if constexpr (P4) {
                    float kf[8], vf[8];
                    q4_floats(kc[r], ks[r], kf);
                    q4_floats(vc[r], vs[r], vf);
                    store8<T>(p.Ko, dst, kf);
                    store8<T>(p.Vo, dst, vf);
                } else {
                    store8<T>(p.Ko, dst, kw[r]);
                    store8<T>(p.Vo, dst, vw[r]);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ whole pages
// For chunks of many tiles, which would all turn the same codes into numbers again. Only pages
// that a row may see: from the first new token's reach on, those with a global
// position, all if a new token is global. The rest are marked missing, as nobody looks there.
// A CTA takes one key head of every gridDim.x-th page of a sequence. The attention is set up as
// the last CTAs run out, no earlier: started beside all of them it comes to sit badly (4096
// tokens of 4 sequences, window 512, 32 query and 4 key heads, d = 64: 183 us, 138 so).
constexpr int kUnpackThreads = 256, kUnpackWords = 4;

template <int D>
__global__ void __launch_bounds__(kUnpackThreads) paged_unpack(const PagedProblem p, uint4 *K, uint4 *V, int32_t *table) {
    __shared__ int s_stride, s_global;
    const int b = blockIdx.y, h = blockIdx.z, tid = threadIdx.x;
    int q = p.qlens ? __ldg(p.qlens + b) : p.m;
    const int s = __ldg(p.lens + b);
    // lengths that break the contract are latched by the attention
    if (q < 0 || q > p.m || s < q || (long long)s > ((long long)p.max_pages << p.log_page)) q = 0;
    if (p.dilation || p.ng > 0) {
        if (tid == 0) {
            s_stride = 1;
            s_global = 0;
        }
        __syncthreads();
        if (p.dilation) {
            int most = 1;
            for (int i = tid; i < p.Hq; i += kUnpackThreads) {
                const int v = __ldg(p.dilation + i);
                if (v > 0 && v <= kMaxDilation) most = max(most, v + 1);
            }
            atomicMax(&s_stride, most);
        }
        for (int i = tid; i < p.ng; i += kUnpackThreads) {
            const int g = __ldg(p.gidx + i);
            if (g >= s - q && g < s) s_global = 1;
        }
        __syncthreads();
    }
    const long long reach = (long long)p.half * (p.dilation ? s_stride : 1);
    const long long first = p.ng > 0 && s_global ? 0 : (long long)(s - q) - reach;
    const int words = p.page * (D / 8);
    const size_t page_bytes = q4_page_bytes(p.page, D);
    for (int c = blockIdx.x; c < p.max_pages; c += gridDim.x) {
        const long long lo = (long long)c << p.log_page, hi = lo + p.page;
        bool need = q > 0 && lo < s && hi > first;
        if (q > 0 && lo < s && !need && p.ng > 0) {
            bool mine = false;
            for (int i = tid; i < p.ng; i += kUnpackThreads) {
                const int g = __ldg(p.gidx + i);
                mine |= g >= lo && g < hi;
            }
            need = __syncthreads_or(mine);
        }
        const size_t slot = (size_t)b * p.max_pages + c;
        int pg = need ? __ldg(p.table + slot) : -1;
        if (pg < -1 || pg >= p.num_pages) {
            if (tid == 0) atomicOr(p.status, kDevBadIndex);
            pg = -1;
        }
        if (tid == 0 && h == 0) table[slot] = pg < 0 ? -1 : (int32_t)slot;
        if (pg < 0) continue;
        const size_t from = ((size_t)pg * p.Hkv + h) * page_bytes, to = (slot * p.Hkv + h) * words;
        const uint8_t *kp = static_cast<const uint8_t *>(p.K) + from, *vp = static_cast<const uint8_t *>(p.V) + from;
        for (int w0 = tid; w0 < words; w0 += kUnpackThreads * kUnpackWords) {
            uint32_t kc[kUnpackWords], vc[kUnpackWords], ks[kUnpackWords], vs[kUnpackWords];
#pragma unroll
            for (int x = 0; x < kUnpackWords; ++x) {
                const int w = w0 + x * kUnpackThreads;
                if (w >= words) break;
                kc[x] = __ldcs(reinterpret_cast<const uint32_t *>(kp) + w);
                vc[x] = __ldcs(reinterpret_cast<const uint32_t *>(vp) + w);
                ks[x] = __ldg(kp + words * 4 + (w >> 1));
                vs[x] = __ldg(vp + words * 4 + (w >> 1));
            }
#pragma unroll
            for (int x = 0; x < kUnpackWords; ++x) {
                const int w = w0 + x * kUnpackThreads;
                if (w >= words) break;
                float f[8];
                q4_floats(kc[x], ks[x], f);
                store8<__nv_bfloat16>(K, (to + w) * 8, f);
                q4_floats(vc[x], vs[x], f);
                store8<__nv_bfloat16>(V, (to + w) * 8, f);
            }
        }
    }
}

template <typename T, int D>
cudaError_t write_d(const WriteProblem &p, int num_sms, cudaStream_t stream) {
    const long long threads = (long long)p.B * p.m * (D / 16);
    const long long ctas = (threads + kWriteThreads - 1) / kWriteThreads;
    const int heads = 2 * p.Hkv + p.Hq;
    // heads to a thread: few where there are few tokens
    long long slices = 32ll * num_sms / ctas;
    slices = slices < 1 ? 1 : slices > heads ? heads : slices;
    const dim3 grid((unsigned)(ctas < (1 << 30) ? ctas : (1 << 30)), (unsigned)slices);
    void (*kern)(const WriteProblem) =
        p.packed ? (p.interleaved ? cache_write<T, D, true, true> : cache_write<T, D, true, false>)
                 : (p.interleaved ? cache_write<T, D, false, true> : cache_write<T, D, false, false>);
    return launch_behind(kern, grid, kWriteThreads, 0, stream, p);
}

template <typename T, int D>
cudaError_t read_d(const WriteProblem &p, cudaStream_t stream) {
    const long long rows = kReadThreads / (D / 8) * kReadRows;
    const long long ctas = (p.m + rows - 1) / rows, heads = (long long)p.B * p.Hkv;
    const dim3 grid((unsigned)ctas, (unsigned)(heads < 65535 ? heads : 65535));
    return launch_behind(p.packed ? cache_read<T, D, true> : cache_read<T, D, false>, grid, kReadThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_cache_write(const WriteProblem &p, sa_dtype dtype, int num_sms, cudaStream_t stream) {
    if (dtype == SA_FP32) return p.d == 64 ? write_d<float, 64>(p, num_sms, stream) : write_d<float, 128>(p, num_sms, stream);
    return p.d == 64 ? write_d<__nv_bfloat16, 64>(p, num_sms, stream) : write_d<__nv_bfloat16, 128>(p, num_sms, stream);
}

cudaError_t launch_cache_read(const WriteProblem &p, sa_dtype dtype, cudaStream_t stream) {
    if (dtype == SA_FP32) return p.d == 64 ? read_d<float, 64>(p, stream) : read_d<float, 128>(p, stream);
    return p.d == 64 ? read_d<__nv_bfloat16, 64>(p, stream) : read_d<__nv_bfloat16, 128>(p, stream);
}

cudaError_t launch_paged_unpack(const PagedProblem &p, void *K, void *V, int32_t *table, int num_sms, cudaStream_t stream) {
    const long long rows = (long long)p.B * p.Hkv, per_row = 16ll * num_sms / rows + 1;
    const dim3 grid((unsigned)(p.max_pages < per_row ? p.max_pages : per_row), (unsigned)p.B, (unsigned)p.Hkv);
    (p.d == 64 ? paged_unpack<64> : paged_unpack<128>)<<<grid, kUnpackThreads, 0, stream>>>(
        p, static_cast<uint4 *>(K), static_cast<uint4 *>(V), table);
    return cudaGetLastError();
}

}  // namespace sa
