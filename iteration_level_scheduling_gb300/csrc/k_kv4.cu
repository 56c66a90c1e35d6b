// A K/V cache held in 4 bits: quantising rows as they are written, reading
// slots back, and attention over the held codes.
//
// A component x of a group of min(32, head_dim) components of one head of one
// slot is held as code c with the group's scale s and minimum m (both bf16):
//   s = bf16((max - min) / 15), m = bf16(min),
//   c = the integer nearest to (x - m) / s (ties to even) within 0 .. 15,
// and stands for m + s c.  The differences and the quotient of the scale are
// taken in fp32; the code is the one real arithmetic gives (below), so it does
// not depend on how the division rounds.  s = 0 holds c = 0.  A group whose
// scale or minimum is not finite (an infinity or NaN among its values, or a
// range beyond fp32) holds s = m = NaN and reads back as NaN.
//
// Layout of a layer (S = kv_slots rounded up to 16, G groups per head):
//   K codes  [head][S][D / 2]      component 2b in the low, 2b + 1 in the high bits of byte b
//   V codes  [head][S / 2][D / 4]  32-bit words: four components of the even slot in the low
//                                  half, the same four of the odd slot in the high half
//   K params [head][S][G]          s in the low, m in the high 16 bits
//   V params [head][S / 2][G][2]   the same, even slot first
// K's codes are read along a key (the reduction of q k runs over components);
// V's reduction runs over keys, so a word pairs the two keys that a tensor-core
// operand register wants side by side.  A slot is written in 16-bit pieces at
// least, so no two slots' writers ever share a word to be merged.
#include <algorithm>
#include <cfloat>
#include <cstring>
#include <type_traits>
#include <vector>

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.cuh"

namespace orca {

namespace {

constexpr float kLow = -FLT_MAX;

struct Kv4View {
    uint8_t *kc, *vc;
    uint32_t *kp, *vp;
    int64_t S;  // slots, padded
};

Kv4View kv4_view(const void *layer, int n_heads, int d, int64_t kv_slots) {
    Kv4View v;
    const int G = kv4_groups(d);
    v.S = (kv_slots + 15) / 16 * 16;
    const int64_t codes = (int64_t)n_heads * v.S * d / 2, params = (int64_t)n_heads * v.S * G;
    v.kc = (uint8_t *)layer;
    v.vc = v.kc + codes;
    v.kp = (uint32_t *)(v.vc + codes);
    v.vp = v.kp + params;
    return v;
}

// min / max that return NaN if either operand is NaN
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_bits(float x) { return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// The code of x for scale s > 0 and minimum m.  The fp32 quotient may round
// onto or across a border k + 1/2, so the candidate is put right with the
// residual x - m - c s, which is exact: a + e = x - m (a rounded, e its
// error), and r = a - c s is a difference of near multiples of one grid.
__device__ __forceinline__ uint32_t kv4_code(float x, float m, float s) {
    const float a = __fsub_rn(x, m);
    const float bb = __fsub_rn(x, a);                                            // m as the subtraction saw it
    const float e = __fadd_rn(__fsub_rn(x, __fadd_rn(a, bb)), __fsub_rn(bb, m));  // x - m = a + e
    float c = rintf(__fdiv_rn(a, s));
    c = fminf(fmaxf(c, 0.f), 15.f);
    const float r = __fmaf_rn(-c, s, a), h = 0.5f * s;
    const bool odd = ((int)c & 1) != 0;
    if (r > h || (r == h && (e > 0.f || (e == 0.f && odd)))) c += 1.f;
    else if (r < -h || (r == -h && (e < 0.f || (e == 0.f && odd)))) c -= 1.f;
    return (uint32_t)fminf(fmaxf(c, 0.f), 15.f);
}

// Eight components' codes, component i in bits 4 i ..  The candidate from a
// product with 1 / s is right if what it leaves is less than half a step (the
// residual is exact, as above).  Halves, which bf16 data meet about once in 256,
// are settled one after the other, by the error of x - m or to the even code;
// what is further off (a minimum that rounded up by more than half a step) is
// done the long way.  Digits are put together in fp32, four at a time.
__device__ __forceinline__ uint32_t kv4_codes(const float *x, float m, float s, float inv) {
    constexpr float kRound = 12582912.f;  // 1.5 2^23: the integer in the low bits
    const float h = 0.5f * s, inv15 = inv * (1.f / 15.f);
    uint32_t open = 0;
    float d[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        const float a = __fsub_rn(x[i], m);
        const float c = __fmaf_rn(__saturatef(a * inv15), 15.f, kRound) - kRound;  // clamped to 0 .. 15
        const float r = __fmaf_rn(-c, s, a);
        if (!(fabsf(r) < h)) open |= 1u << i;
        d[i >> 2] = __fmaf_rn(d[i >> 2], 16.f, c);
    }
    if (!(s > 0.f)) return 0u;
    uint32_t w = (__float_as_uint(d[0] + 8388608.f) & 0xffffu) | (__float_as_uint(d[1] + 8388608.f) << 16);
    while (open) {
        const int i = __ffs(open) - 1;
        open &= open - 1;
        float xi = x[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) xi = i == e ? x[e] : xi;  // (x stays in registers)
        const uint32_t c = (w >> (4 * i)) & 15u;
        const float a = __fsub_rn(xi, m), r = __fmaf_rn(-(float)c, s, a);
        uint32_t to;
        if (fabsf(r) == h) {
            const float bb = __fsub_rn(xi, a);
            const float e = __fadd_rn(__fsub_rn(xi, __fadd_rn(a, bb)), __fsub_rn(bb, m));  // x - m = a + e
            const bool away = e == 0.f ? (c & 1u) != 0 : (e > 0.f) == (r > 0.f);
            to = !away ? c : r > 0.f ? min(c + 1, 15u) : max(c, 1u) - 1;
        } else {
            to = kv4_code(xi, m, s);
        }
        w = (w & ~(15u << (4 * i))) | to << (4 * i);
    }
    return w;
}

// Scale and minimum (packed, bf16) and the codes of a group's share of 8 components, GT neighbouring threads each
// holding 8; every thread of the warp takes part.
template <int GT>
__device__ __forceinline__ uint32_t kv4_quantise(const float *x, uint32_t *par) {
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) lo = min_nan(lo, x[i]), hi = max_nan(hi, x[i]);
#pragma unroll
    for (int o = 1; o < GT; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    uint32_t sb = bf_bits(__fdiv_rn(__fsub_rn(hi, lo), 15.f)), mb = bf_bits(lo);
    if ((sb & 0x7f80u) == 0x7f80u || (mb & 0x7f80u) == 0x7f80u) sb = mb = 0x7fc0u;
    *par = sb | (mb << 16);
    const float s = bf_lo(sb);
    float inv;
    asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
    return kv4_codes(x, bf_lo(mb), s, inv);
}

// ---------------------------------------------------------------------------
// write: one thread per 8 components of k and of v, of one row or of two whose
// slots share a pair (then V goes out in whole words)
//
// Bound by issue (84 % of active cycles; 25 warp instructions per 32 components,
// 5 of them for halves): 10.5 k rows of 40 heads of 128, bf16, 81 us for 215 MB
// read and 67 MB written (42 us at the copy rate); with an IEEE quotient per
// component 189.
// ---------------------------------------------------------------------------
constexpr int kApThreads = 128;

template <typename T>
__device__ __forceinline__ void load8_stream(const T *p, float *x) {
#pragma unroll
    for (int i = 0; i < 8; i += Elem<T>::kPer16) load16_stream(p + i, x + i);
}

// Flat: the threads of a block run on from unit to unit (a row whose H / 8 is no multiple of the block's threads would
// leave the rest of them idle; 5 x <= 333 rows of 12 heads of 32, fp32: 4.2 -> 3.0 us).  A group's threads stay in one
// unit.
template <typename T, int D, bool Flat>
__global__ void __launch_bounds__(kApThreads) kv4_append_kernel(const T *qkv, const int32_t *units, int n_units, Kv4View v,
                                                                int H) {
    constexpr int G = D >= 32 ? D / 32 : 1, GT = D / G / 8;
    pdl_trigger();
    pdl_wait();
    int unit, c;  // c: component of the row
    if constexpr (Flat) {
        const int64_t i = (int64_t)blockIdx.x * kApThreads + threadIdx.x;
        unit = (int)(i / (H / 8)), c = (int)(i - (int64_t)unit * (H / 8)) * 8;
    } else {
        unit = blockIdx.x, c = (blockIdx.y * kApThreads + threadIdx.x) * 8;
    }
    const bool on = unit < n_units;
    const int4 un = on ? reinterpret_cast<const int4 *>(units)[unit] : make_int4(0, 0, 0, 0);  // first row, its slot,
    const int64_t slot = un.y;                                                                 // rows (1, or 2 in one pair)
    const bool two = un.z == 2;
    float x[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // k, v of the first row; of the second
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
        if (on && (i < 2 || two)) load8_stream(qkv + ((size_t)un.x + (i >> 1)) * 3 * H + (1 + (i & 1)) * (size_t)H + c, x[i]);
    }
    const int h = c / D, dd = c % D;
    const int64_t row = (int64_t)h * v.S + slot, pair = row >> 1;  // (S is even)
    const bool lead = dd % (8 * GT) == 0;
    const int g = dd / (8 * GT);
    uint32_t par[2], w[2];
    w[0] = kv4_quantise<GT>(x[0], &par[0]);
    if (on) {
        *reinterpret_cast<uint32_t *>(v.kc + row * (D / 2) + dd / 2) = w[0];
        if (lead) v.kp[row * G + g] = par[0];
    }
    if (!Flat ? two : __any_sync(0xffffffffu, two)) {
        w[0] = kv4_quantise<GT>(x[2], &par[0]);
        if (two) {
            *reinterpret_cast<uint32_t *>(v.kc + (row + 1) * (D / 2) + dd / 2) = w[0];
            if (lead) v.kp[(row + 1) * G + g] = par[0];
        }
        w[0] = kv4_quantise<GT>(x[1], &par[0]);
        w[1] = kv4_quantise<GT>(x[3], &par[1]);
        if (two) {
            *reinterpret_cast<uint2 *>(v.vc + pair * D + dd) =
                make_uint2((w[0] & 0xffffu) | (w[1] << 16), (w[0] >> 16) | (w[1] & 0xffff0000u));
            if (lead) *reinterpret_cast<uint2 *>(v.vp + (pair * G + g) * 2) = make_uint2(par[0], par[1]);
        }
    } else {
        w[0] = kv4_quantise<GT>(x[1], &par[0]);
    }
    if (on && !two) {
        uint16_t *dst = reinterpret_cast<uint16_t *>(v.vc + pair * D + dd) + (slot & 1);
        dst[0] = (uint16_t)w[0];
        dst[2] = (uint16_t)(w[0] >> 16);
        if (lead) v.vp[(pair * G + g) * 2 + (slot & 1)] = par[0];
    }
}

// ---------------------------------------------------------------------------
// read back: tiles of up to 64 slots of one range, one head's K and V per CTA
//
// Bound by memory: the same 10.5 k slots, 67 MB read and 215 MB written, in 44 us
// (96 % of the copy rate; part of the writes is still in L2).
// ---------------------------------------------------------------------------
constexpr int kRdThreads = 128;
constexpr int kReadTile = 64;  // slots per tile
// heads that a CTA of kv4_read_few_kernel takes
__host__ __device__ constexpr int kv4_few_heads(int d, int per) { return 2 * kRdThreads / (d / 8) / per; }

// nibbles N and N + 4 of w as floats, through bf16's 128 + c (conversions run at an eighth of the rate)
template <int N>
__device__ __forceinline__ void code_floats(uint32_t w, float &a, float &b) {
    const uint32_t u = ((w >> (4 * N)) & 0x000f000fu) | 0x43004300u;
    a = bf_lo(u) - 128.f, b = bf_hi(u) - 128.f;
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float *x) {
#pragma unroll
    for (int i = 0; i < 8; i += Elem<T>::kPer16) store16(p + i, x + i);
}
__device__ __forceinline__ void store8(__half *p, const float *x) {
    uint4 u;
    __half2 *h = reinterpret_cast<__half2 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = u;
}

// Scaled (prompts, below): scale holds the inverses of the powers of two that the values are to be multiplied by,
// [request][head][K|V].  Every load of a thread is issued before the first is used.
template <typename T, int D, bool Scaled>
__global__ void __launch_bounds__(kRdThreads) kv4_read_kernel(Kv4View v, const int32_t *tiles, T *out, int64_t out_slots,
                                                              int n_heads, const float *scale) {
    constexpr int G = D >= 32 ? D / 32 : 1, GS = D / G, U = D / 8;  // 8-component units per row
    constexpr int KN = kReadTile * U / kRdThreads, VN = (KN + 1) / 2;  // units of K per thread, pairs of V
    pdl_trigger();
    pdl_wait();
    const int4 tl = reinterpret_cast<const int4 *>(tiles)[blockIdx.x];  // first slot, slots, first output index, request
    const int h = blockIdx.y;
    const int64_t s0 = tl.x, s1 = s0 + tl.y;
    float kf = 1.f, vf = 1.f;
    if constexpr (Scaled) {
        const float *f = scale + 2 * ((size_t)tl.w * n_heads + h);
        kf = 1.f / f[0], vf = 1.f / f[1];
    }
    T *ko = out + ((int64_t)h * out_slots + tl.z) * D, *vo = ko + (int64_t)n_heads * out_slots * D;
    const int u = threadIdx.x % U, gr = u * 8 / GS;
    uint32_t kw[KN], kp[KN], pv[KN];
#pragma unroll
    for (int n = 0; n < KN; ++n) {
        const int j = (threadIdx.x + n * kRdThreads) / U;
        if (j < tl.y) {
            const int64_t row = (int64_t)h * v.S + s0 + j;
            kw[n] = __ldcs(reinterpret_cast<const uint32_t *>(v.kc + row * (D / 2)) + u);
            kp[n] = v.kp[row * G + gr];
            if constexpr (Scaled) pv[n] = v.vp[((row >> 1) * G + gr) * 2 + ((s0 + j) & 1)];
        }
    }
    const int64_t p0 = s0 >> 1;
    const int np = (int)(((s1 + 1) >> 1) - p0);  // up to 33 pairs: the 33rd is left to a second round
    uint2 vw[VN], vp[VN];
    auto load_v = [&](int n, int j) {
        if (j < np) {
            const int64_t pair = (int64_t)h * (v.S / 2) + p0 + j;
            vw[n] = __ldcs(reinterpret_cast<const uint2 *>(v.vc + pair * D) + u);
            vp[n] = *reinterpret_cast<const uint2 *>(v.vp + (pair * G + gr) * 2);
        }
    };
#pragma unroll
    for (int n = 0; n < VN; ++n) load_v(n, (threadIdx.x + n * kRdThreads) / U);
#pragma unroll
    for (int n = 0; n < KN; ++n) {
        const int j = (threadIdx.x + n * kRdThreads) / U;
        if (j >= tl.y) continue;
        float s = bf_lo(kp[n]) * kf, m = bf_hi(kp[n]) * kf;
        if constexpr (Scaled) {
            // a NaN among the values is moved to the key: a weight of 0 times it would reach rows that do not see
            // the key, while a masked score is dropped whatever it is
            const float sv = bf_lo(pv[n]);
            if (sv != sv) m = sv;
        }
        float x[8];
        code_floats<0>(kw[n], x[0], x[4]);
        code_floats<1>(kw[n], x[1], x[5]);
        code_floats<2>(kw[n], x[2], x[6]);
        code_floats<3>(kw[n], x[3], x[7]);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = fmaf(s, x[k], m);
        store8(ko + (int64_t)j * D + u * 8, x);
    }
    auto store_v = [&](int n, int j) {
        if (j >= np) return;
        float xe[8], xo[8];  // even and odd slot
        code_floats<0>(vw[n].x, xe[0], xo[0]);
        code_floats<1>(vw[n].x, xe[1], xo[1]);
        code_floats<2>(vw[n].x, xe[2], xo[2]);
        code_floats<3>(vw[n].x, xe[3], xo[3]);
        code_floats<0>(vw[n].y, xe[4], xo[4]);
        code_floats<1>(vw[n].y, xe[5], xo[5]);
        code_floats<2>(vw[n].y, xe[6], xo[6]);
        code_floats<3>(vw[n].y, xe[7], xo[7]);
        const int64_t slot = 2 * (p0 + j);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            if (slot + o < s0 || slot + o >= s1) continue;
            const uint32_t pp = o ? vp[n].y : vp[n].x;
            float s = bf_lo(pp) * vf, m = bf_hi(pp) * vf;
            if (Scaled && s != s) s = m = 0.f;
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = fmaf(s, o ? xo[k] : xe[k], m);
            store8(vo + (slot + o - s0) * D + u * 8, x);
        }
    };
#pragma unroll
    for (int n = 0; n < VN; ++n) store_v(n, (threadIdx.x + n * kRdThreads) / U);
    for (int j = (threadIdx.x + VN * kRdThreads) / U; j < np; j += kRdThreads / U) load_v(0, j), store_v(0, j);
}

// The same for a plan whose ranges are all short (increments): a CTA takes `per` slots of several heads, two units of
// K and V per thread.  64 ranges, 40 heads of 128, against a CTA per range and head: one slot 1.7 us and 4.8, four
// slots 2.8 and 5.2, eight 4.5 and 5.8; 12 heads of 32 in fp32: 1.25 and 1.7, 1.5 and 1.7, 2.1 and 1.7.
constexpr int kFewSlots = 4;
template <typename T, int D>
__global__ void __launch_bounds__(kRdThreads) kv4_read_few_kernel(Kv4View v, const int32_t *tiles, T *out,
                                                                  int64_t out_slots, int n_heads, int per) {
    constexpr int G = D >= 32 ? D / 32 : 1, GS = D / G, U = D / 8, N = 2;
    pdl_trigger();
    pdl_wait();
    const int4 tl = reinterpret_cast<const int4 *>(tiles)[blockIdx.x];
    const int u = threadIdx.x % U, gr = u * 8 / GS, heads = kv4_few_heads(D, per);  // heads per CTA
    uint32_t kw[N], kp[N], pv[N];
    uint2 vw[N];
    int h[N], s[N];
    bool on[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int j = (threadIdx.x + n * kRdThreads) / U, hh = j / per;
        h[n] = blockIdx.y * heads + hh, s[n] = j - hh * per;
        on[n] = hh < heads && h[n] < n_heads && s[n] < tl.y;
        if (on[n]) {
            const int64_t row = h[n] * v.S + tl.x + s[n], pair = row >> 1;
            kw[n] = __ldcs(reinterpret_cast<const uint32_t *>(v.kc + row * (D / 2)) + u);
            kp[n] = v.kp[row * G + gr];
            vw[n] = reinterpret_cast<const uint2 *>(v.vc + pair * D)[u];
            pv[n] = v.vp[(pair * G + gr) * 2 + (row & 1)];
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (!on[n]) continue;
        const bool odd = (tl.x + s[n]) & 1;
        const uint32_t w = odd ? (vw[n].x >> 16) | (vw[n].y & 0xffff0000u) : (vw[n].x & 0xffffu) | (vw[n].y << 16);
        T *dst = out + ((int64_t)h[n] * out_slots + tl.z + s[n]) * D + u * 8;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const uint32_t c = o ? w : kw[n], p = o ? pv[n] : kp[n];
            float x[8];
            code_floats<0>(c, x[0], x[4]);
            code_floats<1>(c, x[1], x[5]);
            code_floats<2>(c, x[2], x[6]);
            code_floats<3>(c, x[3], x[7]);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = fmaf(bf_lo(p), x[k], bf_hi(p));
            store8(dst + (o ? (int64_t)n_heads * out_slots * D : 0), x);
        }
    }
}

// ---------------------------------------------------------------------------
// prompts on the tcgen05 prefill kernel: q, K and V as fp16 in a workspace
// ---------------------------------------------------------------------------
// fp16 rather than bf16: K and V come from codes and not from bf16 values, so
// rounding them to 8 bits would add an error as large as the output's own.
// fp16 keeps 11 bits; its narrow range is met by powers of two, one per row and
// head for q and one per request and head for K and V, that bring the largest
// magnitude to [2^14, 2^15).  Groups below 2^-28 of the largest would lose bits
// and those below 2^-40 everything, also for rows that do not see the largest:
// a request and head with such a group is marked, and its rows are attended in
// groups on the codes themselves behind the prefill kernel (kv4_rows_wide_kernel;
// without marks the launch costs 1 us: the prompt chunks below 189.2 and 190.2).
// Four prompts of 900 rows over 1000 keys, 40 heads of 128: scales and q 25 us, K
// and V 42 us, the attention 168 us under the profiler (tensor pipe 36 % of active
// cycles, as on a bf16 cache); against rows one by one 4968 us.

// The power of two for a largest magnitude, as its inverse; 1 where that is zero or subnormal.
__device__ __forceinline__ float kv4_inverse_scale(float amax) {
    const int e = (int)(__float_as_uint(amax) >> 23);  // (amax >= 0)
    if (e == 0) return 1.f;
    return __uint_as_float((uint32_t)max(e - 14, 27) << 23);  // 2^(e - 127 - 14), not below 2^-100
}

struct Kv4Prep {
    const bf16 *qkv;
    __half *q16;
    float *q_scale, *kv_scale;
    int32_t *wide;  // [prompt][head]: fp16 does not hold the range of its K or V
    Kv4View v;
    int H, n_heads, d, G, n_rows, n_pre;  // G is 2 or 4
    const int32_t *pre;  // 4 words per prompt: request, first slot, slots, 0
};
constexpr int kPrepThreads = 256, kPrepQ = 4;

// Blocks 0 .. n_pre * n_heads - 1: the scales of K and V of one prompt and head, from the parameters (a component lies
// between m and m + 15 s).  The others scale and round q.
__global__ void __launch_bounds__(kPrepThreads) kv4_prep_kernel(const Kv4Prep a) {
    __shared__ float red[4][kPrepThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = a.n_pre * a.n_heads;
    if ((int)blockIdx.x < first) {
        const int i = blockIdx.x / a.n_heads, h = blockIdx.x - i * a.n_heads;
        const int4 pr = reinterpret_cast<const int4 *>(a.pre)[i];
        const int64_t s0 = pr.y, s1 = s0 + pr.z;
        // (fmaxf and fminf drop NaN: a group that reads back as NaN does so whatever the scale)
        auto size = [](uint32_t p) { return fmaxf(fabsf(bf_hi(p)), fabsf(fmaf(15.f, bf_lo(p), bf_hi(p)))); };
        const uint32_t *kp = a.v.kp + (int64_t)h * a.v.S * a.G, *vp = a.v.vp + (int64_t)h * a.v.S * a.G;
        // words of K: s0 G .. s1 G; of V, whose pairs hold group by group the even and the odd slot, those of the
        // pairs, less the even slot of the first or the odd one of the last.  16 bytes at a time: the 16 slots' words
        // of a head are whole vectors, what lies outside is dropped.
        const int64_t k0 = s0 * a.G, k1 = s1 * a.G, v0 = (s0 >> 1) * 2 * a.G, v1 = ((s1 + 1) >> 1) * 2 * a.G;
        auto take = [&](const uint32_t *base, int64_t lo, int64_t hi, auto in) {
            float2 r = make_float2(0.f, INFINITY);  // the largest group, and the smallest that is not all zeros
            for (int64_t j = (lo & ~int64_t(3)) + 4 * threadIdx.x; j < hi; j += 4 * 8 * kPrepThreads) {
                uint4 p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    p[e] = j + 4 * e * kPrepThreads < hi
                               ? *reinterpret_cast<const uint4 *>(base + j + 4 * e * kPrepThreads)
                               : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t w[4] = {p[e].x, p[e].y, p[e].z, p[e].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int64_t at = j + 4 * e * kPrepThreads + q;
                        if (at >= lo && at < hi && in(at)) {
                            const float x = size(w[q]);
                            r.x = fmaxf(r.x, x);
                            if (x > 0.f) r.y = fminf(r.y, x);
                        }
                    }
                }
            }
            return r;
        };
        float2 km = take(kp, k0, k1, [](int64_t) { return true; });
        float2 vm = take(vp, v0, v1, [&](int64_t at) {
            const int64_t slot = (at >> (a.G == 4 ? 3 : 2)) * 2 + (at & 1);
            return slot >= s0 && slot < s1;
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            km.x = fmaxf(km.x, __shfl_xor_sync(0xffffffffu, km.x, o));
            vm.x = fmaxf(vm.x, __shfl_xor_sync(0xffffffffu, vm.x, o));
            km.y = fminf(km.y, __shfl_xor_sync(0xffffffffu, km.y, o));
            vm.y = fminf(vm.y, __shfl_xor_sync(0xffffffffu, vm.y, o));
        }
        if (lane == 0) red[0][warp] = km.x, red[1][warp] = vm.x, red[2][warp] = km.y, red[3][warp] = vm.y;
        __syncthreads();
        if (threadIdx.x < 32) {
            bool wide = false;
            if (threadIdx.x < 2) {
                float big = 0.f, small = INFINITY;
                for (int w = 0; w < kPrepThreads / 32; ++w)
                    big = fmaxf(big, red[threadIdx.x][w]), small = fminf(small, red[2 + threadIdx.x][w]);
                const float inv = kv4_inverse_scale(big);
                a.kv_scale[2 * ((size_t)pr.x * a.n_heads + h) + threadIdx.x] = inv;
                wide = small < inv * 6.103515625e-05f;  // 2^-14, fp16's smallest normal number
            }
            wide = __any_sync(0xffffffffu, wide);
            if (threadIdx.x == 0) a.wide[blockIdx.x] = wide;
        }
        return;
    }
    // q: a thread's units of 8 components, kPrepQ of them in flight; d / 8 neighbouring threads hold a head
    const int upr = a.H / 8, per_head = a.d / 8;
    const int64_t units = (int64_t)a.n_rows * upr;
    const int64_t u0 = ((int64_t)blockIdx.x - first) * (kPrepThreads * kPrepQ) + threadIdx.x;
    float x[kPrepQ][8];
#pragma unroll
    for (int n = 0; n < kPrepQ; ++n) {
        const int64_t u = u0 + n * kPrepThreads;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[n][e] = 0.f;
        if (u < units) {
            const int64_t r = u / upr;
            load16_stream(a.qkv + r * 3 * a.H + (u - r * upr) * 8, x[n]);
        }
    }
#pragma unroll
    for (int n = 0; n < kPrepQ; ++n) {
        const int64_t u = u0 + n * kPrepThreads;
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(x[n][e]));
        for (int o = per_head / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float inv = kv4_inverse_scale(m), f = 1.f / inv;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[n][e] *= f;
        if (u < units) {
            store8(a.q16 + u * 8, x[n]);
            if (u % per_head == 0) a.q_scale[u / per_head] = inv;  // [row][head]
        }
    }
}

// ---------------------------------------------------------------------------
// attention of single rows: item = (row, chunk of its keys) x head, four warps
// ---------------------------------------------------------------------------
constexpr int kKvThreads = 128, kKvWarps = 4;

struct Kv4Attn {
    const void *qkv;
    void *out;
    Kv4View v;
    int H, n_heads;
    float scale_log2;
    const int32_t *items;  // block = item * n_heads + head; 8 words: first slot, keys, row, chunks of the row, this chunk, the row's first partial, its counter
    int *counters;         // [row counter][head], zero between launches
    float *part;           // [partial][head][D + 2]
    const int32_t *row_items;  // the same for groups of rows (kv4_rows_mma_kernel), 12 words an item
    const int32_t *row_joins;
    float *row_part;  // [partial][head][16][D + 2]
    const int32_t *wide, *wide_items;  // prompts' heads beyond fp16's range, and the prompts' rows in groups
    int n_wide, n_wide_items;          // prompts x heads, items
};

// Join the partials of `nch` chunks, `stride` floats apart, in chunk order: component `at`, the maximum at D and the
// sum at D + 1.  Eight chunks' loads are in flight at a time.
template <int D>
__device__ __forceinline__ float kv4_join(const float *part, size_t stride, int nch, int at) {
    float Mt = kLow, Lt = 0.f, Ot = 0.f;
    for (int c = 0; c < nch; c += 8) {
        float pm[8], pl[8], po[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float *p = part + (size_t)min(c + j, nch - 1) * stride;
            pm[j] = __ldcg(p + D), pl[j] = __ldcg(p + D + 1), po[j] = __ldcg(p + at);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < nch) {
                const float mn = fmaxf(Mt, pm[j]), co = exp2f(Mt - mn), cn = exp2f(pm[j] - mn);
                Lt = Lt * co + pl[j] * cn;
                Ot = Ot * co + po[j] * cn;
                Mt = mn;
            }
    }
    return Ot / Lt;
}

template <int D>
struct Kv4Merge {
    float m[kKvWarps], l[kKvWarps], o[kKvWarps][D];
    int last;
};

// 2^x by the SFU's approximation (x <= 0 here; results below 2^-126 are zero)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The four warps' states (each already in sm) -> the row's output, or this
// chunk's partial; the last chunk to arrive joins all of them in chunk order,
// so the result does not depend on which that is.
template <typename T, int D>
__device__ __forceinline__ void kv4_finish(const Kv4Attn &a, Kv4Merge<D> &sm, const int4 &r0, const int4 &r1, int h) {
    __syncthreads();
    const int tid = threadIdx.x;
    float M = kLow, L = 0.f, O = 0.f, c[kKvWarps];
#pragma unroll
    for (int w = 0; w < kKvWarps; ++w) M = fmaxf(M, sm.m[w]);
#pragma unroll
    for (int w = 0; w < kKvWarps; ++w) c[w] = exp2f(sm.m[w] - M), L += sm.l[w] * c[w];
    if (tid < D) {
#pragma unroll
        for (int w = 0; w < kKvWarps; ++w) O += sm.o[w][tid] * c[w];
    }
    T *dst = (T *)a.out + (size_t)r0.z * a.H + h * D;
    const int nch = r0.w;
    if (nch == 1) {
        if (tid < D) dst[tid] = Elem<T>::from_f(O / L);
        return;
    }
    float *mine = a.part + ((size_t)(r1.y + r1.x) * a.n_heads + h) * (D + 2);
    if (tid < D) mine[tid] = O;
    if (tid == 0) mine[D] = M, mine[D + 1] = L;
    __syncthreads();
    if (tid == 0) {
        int *cnt = a.counters + (size_t)r1.z * a.n_heads + h;
        __threadfence();
        const int last = atom_add_acq_rel(cnt, 1) == nch - 1;
        if (last) *cnt = 0;
        sm.last = last;
    }
    __syncthreads();
    if (!sm.last) return;
    __threadfence();
    if (tid < D)
        dst[tid] = Elem<T>::from_f(kv4_join<D>(a.part + ((size_t)r1.y * a.n_heads + h) * (D + 2),
                                               (size_t)a.n_heads * (D + 2), nch, tid));
}

// W consecutive words
template <int W>
__device__ __forceinline__ void get_words(const void *p, uint32_t *w) {
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// W consecutive words, streamed
template <int W>
__device__ __forceinline__ void load_words(const void *p, uint32_t *w) {
    if constexpr (W == 4) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (W == 2) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
    }
}

// Single rows of any type and head_dim, fp32 arithmetic (fp32 models; head_dim 16).  A warp
// takes 32 slots at a time: for the scores a lane owns a key and walks its
// components against q in shared memory; for the values a lane owns four
// components and walks the keys, two per word.  A code is used as the fp32
// subnormal that its bits are in place (nibble n of a word: c 2^(4n - 149), for
// n <= 4), times a factor that carries the power of two -- q's, scaled -- or, for
// the values, added to 2^23 and taken around code 8: an AND or two instead of a
// shift, an AND and a conversion at an eighth of the rate.  Bound by latency and
// issue: 64 requests of 4000 keys, 12 heads of 64, fp32: 123 us (277 with the
// conversions, 139 without the values' early loads); 17 of <= 900 keys 11.6.
__device__ __forceinline__ float nibble_bits(uint32_t w, int n) { return __uint_as_float(w & (15u << (4 * n))); }

template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads, 4) kv4_decode_kernel(const Kv4Attn a) {
    constexpr int G = D / 32 > 0 ? D / 32 : 1, GS = D / G, GW = GS / 8;  // words of a group and key
    constexpr int LP = D / 4, PP = 32 / LP;  // lanes per pair of keys, pairs per step
    __shared__ Kv4Merge<D> sm;
    __shared__ __align__(16) float q[D];
    __shared__ float qs[G], big[kKvWarps];
    pdl_trigger();
    pdl_wait();
    const int item = blockIdx.x / a.n_heads, h = blockIdx.x - item * a.n_heads;
    const int4 r0 = reinterpret_cast<const int4 *>(a.items)[2 * item],
               r1 = reinterpret_cast<const int4 *>(a.items)[2 * item + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // q brought to 2^14 by a power of two and on to 2^100, by nibble (5 .. 7 are used two places to the right)
    float k_unit;
    {
        const float x = threadIdx.x < D
                            ? Elem<T>::to_f(((const T *)a.qkv)[(size_t)r0.z * 3 * a.H + h * D + threadIdx.x]) : 0.f;
        float m = fabsf(x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) big[warp] = m;
        if (threadIdx.x < D) q[threadIdx.x] = x;
        __syncthreads();
        m = 0.f;
#pragma unroll
        for (int w = 0; w < kKvWarps; ++w) m = max_nan(m, big[w]);
        if (threadIdx.x < G) {
            float s = 0.f;
            for (int i = 0; i < GS; ++i) s += q[threadIdx.x * GS + i];
            qs[threadIdx.x] = s * a.scale_log2;
        }
        const float inv = kv4_inverse_scale(m);
        const int n = threadIdx.x & 7, place = n < 5 ? n : n - 3;
        __syncthreads();
        if (threadIdx.x < D) q[threadIdx.x] = x * (1.f / inv) * __uint_as_float((127u + 86u - 4u * place) << 23);
        k_unit = inv * a.scale_log2;  // of the scores' sums, with 2^(149 - 86) in two steps below
        __syncthreads();
    }
    const int64_t s0 = r0.x, s1 = s0 + r0.y;
    const int sub = lane % LP, grp = lane / LP;
    float m = kLow, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f}, zero = 0.f;
    for (int64_t b = (s0 & ~int64_t(1)) + 32 * warp; b < s1; b += 32 * kKvWarps) {
        const int64_t slot = b + lane;
        const bool valid = slot >= s0 && slot < s1;
        if (b + 32 * kKvWarps + 32 <= s1) {  // the warp's next 32 slots into L1, line by line
            constexpr int kCode = 32 * D / 2 / 128, kPar = 32 * G * 4 / 128;
            const int64_t next = (int64_t)h * a.v.S + b + 32 * kKvWarps;
#pragma unroll
            for (int c = 0; c < 2 * (kCode + kPar); c += 32) {
                const int n = c + lane;
                const uint8_t *at = n < kCode              ? a.v.kc + next * (D / 2) + n * 128
                                    : n < 2 * kCode        ? a.v.vc + next * (D / 2) + (n - kCode) * 128
                                    : n < 2 * kCode + kPar ? (const uint8_t *)(a.v.kp + next * G) + (n - 2 * kCode) * 128
                                                           : (const uint8_t *)(a.v.vp + next * G) + (n - 2 * kCode - kPar) * 128;
                if (n < 2 * (kCode + kPar)) prefetch_l1(at);
            }
        }
        // the values' words of the first steps, in flight with the keys
        constexpr int kSteps = 16 / PP, kEarly = kSteps < 8 ? kSteps : 8;
        uint32_t vx[kEarly];
        uint2 vpp[kEarly];
        auto load_v = [&](int j, uint32_t &x, uint2 &pp) {
            const int64_t se = b + 2 * (j * PP + grp);
            x = 0u, pp = make_uint2(0u, 0u);
            if (se + 1 >= s0 && se < s1) {
                const int64_t pair = (int64_t)h * (a.v.S / 2) + (se >> 1);
                x = reinterpret_cast<const uint32_t *>(a.v.vc + pair * D)[sub];
                pp = *reinterpret_cast<const uint2 *>(a.v.vp + (pair * G + sub * 4 / GS) * 2);
            }
        };
#pragma unroll
        for (int j = 0; j < kEarly; ++j) load_v(j, vx[j], vpp[j]);
        float sc = kLow;
        if (valid) {
            const int64_t row = (int64_t)h * a.v.S + slot;
            uint32_t w[G * GW];
            const uint32_t *kc = reinterpret_cast<const uint32_t *>(a.v.kc + row * (D / 2));
            if constexpr (D >= 32) {
#pragma unroll
                for (int g = 0; g < G; ++g) get_words<4>(kc + 4 * g, w + 4 * g);
            } else {
                get_words<2>(kc, w);
            }
            sc = 0.f;
            float acc = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t p = a.v.kp[row * G + g];
                float e[2] = {0.f, 0.f};
#pragma unroll
                for (int x = 0; x < GW; ++x) {
                    const float4 qa = *reinterpret_cast<const float4 *>(&q[(g * GW + x) * 8]),
                                 qb = *reinterpret_cast<const float4 *>(&q[(g * GW + x) * 8 + 4]);
                    const uint32_t lo = w[g * GW + x], hi = lo >> 12;
                    e[0] = fmaf(qa.x, nibble_bits(lo, 0), e[0]), e[1] = fmaf(qa.y, nibble_bits(lo, 1), e[1]);
                    e[0] = fmaf(qa.z, nibble_bits(lo, 2), e[0]), e[1] = fmaf(qa.w, nibble_bits(lo, 3), e[1]);
                    e[0] = fmaf(qb.x, nibble_bits(lo, 4), e[0]), e[1] = fmaf(qb.y, nibble_bits(hi, 2), e[1]);
                    e[0] = fmaf(qb.z, nibble_bits(hi, 3), e[0]), e[1] = fmaf(qb.w, nibble_bits(hi, 4), e[1]);
                }
                acc = fmaf(bf_lo(p), (e[0] + e[1]) * __uint_as_float((127u + 63u) << 23), acc);
                sc = fmaf(bf_hi(p), qs[g], sc);
            }
            sc = fmaf(acc, k_unit, sc);
        }
        float mx = sc;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        mx = fmaxf(mx, m);
        const float corr = exp2f(m - mx);
        m = mx;
        const float p = valid ? exp2f(sc - m) : 0.f;
        l = l * corr + p;
        zero *= corr;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] *= corr;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const int pr = j * PP + grp;  // this lane's pair
            const float pe = __shfl_sync(0xffffffffu, p, 2 * pr), po = __shfl_sync(0xffffffffu, p, 2 * pr + 1);
            const int64_t se = b + 2 * pr;
            const bool ve = se >= s0 && se < s1, vo = se + 1 >= s0 && se + 1 < s1;
            uint32_t x;
            uint2 pp;
            if (j < kEarly) x = vx[j < kEarly ? j : 0], pp = vpp[j < kEarly ? j : 0];
            else load_v(j, x, pp);
            // around code 8, as the sums run over all keys; an unused slot's parameters may be anything
            const float we = ve ? pe * bf_lo(pp.x) : 0.f, wo = vo ? po * bf_lo(pp.y) : 0.f;
            zero += (ve ? pe * fmaf(8.f, bf_lo(pp.x), bf_hi(pp.x)) : 0.f) +
                    (vo ? po * fmaf(8.f, bf_lo(pp.y), bf_hi(pp.y)) : 0.f);
            const uint32_t y = x >> 16;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // (2^23 + c 2^(4k)) - (2^23 + 8 2^(4k)): exact
                const float eight = 8388608.f + (float)(8u << (4 * k));
                const float ce = __uint_as_float((x & (15u << (4 * k))) | 0x4b000000u) - eight;
                const float co = __uint_as_float((y & (15u << (4 * k))) | 0x4b000000u) - eight;
                o[k] = fmaf(we, ce, fmaf(wo, co, o[k]));
            }
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
    for (int off = LP; off < 32; off <<= 1) {
        zero += __shfl_xor_sync(0xffffffffu, zero, off);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] += __shfl_xor_sync(0xffffffffu, o[k], off);
    }
    if (grp == 0)
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 2^(-4k)
            sm.o[warp][4 * sub + k] = fmaf(o[k], __uint_as_float((127u - 4u * k) << 23), zero);
    if (lane == 0) sm.m[warp] = m, sm.l[warp] = l;
    kv4_finish<T, D>(a, sm, r0, r1, h);
}

// bf16, head_dim 32 and more: both products on mma.sync m16n8k16 with the
// codes as the A operand, unpacked in registers straight from 16-byte loads.
//   scores   rows = 16 keys.  A lane's loads of one key are components of one
//            group; q enters column g of B only where the component's group is
//            g, so the columns of S gather sum q c group by group and s, m
//            apply afterwards.  A = the codes as fp16 subnormals, q in fp16.
//            (128 + c in bf16 with the accumulator started at -128 sum q took
//            two more shifts per word and four more products per block.)
//   values   rows = 16 components, k = 16 keys.  A = c - 8, exact; column g of
//            B is p s_g rounded to bf16, column 4 + g what the rounding left,
//            so the weights keep 16 bits; sum p (m + 8 s) is added in fp32.
// Bound by issue and the integer pipe (each 66 % of their peak): 64 requests of <= 4000 keys, 40 heads of 128, 1.04 GB, in
// 197 us, 78 % of the copy rate; 378 warp instructions per 16 keys and head, a third of them to unpack.
// Codes are centred for the values because those sums run over all keys:
// taken around 0 .. 15 the accumulator would grow with every key and cancel
// against the minima at the end.
__device__ __forceinline__ void kv4_mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// {128 + nibble n, 128 + nibble n + 4} of w as two bf16
template <int N>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    return ((w >> (4 * N)) & 0x000f000fu) | 0x43004300u;
}
// the same less 136: {nibble n - 8, nibble n + 4 - 8}
template <int N>
__device__ __forceinline__ uint32_t code_pair_centred(uint32_t w) {
    const uint32_t u = code_pair<N>(w);
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&u), __float2bfloat162_rn(136.f));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}
// One block of 16 slots as a lane (g, t) = (lane / 4, lane % 4) of a warp holds it.
template <int D>
struct Kv4Block {
    static constexpr int W = D / 32;  // words per lane and row, and groups
    uint32_t k[2][W];                 // keys g, g + 8: components 8 W t ..
    uint32_t v[2][W];                 // pairs t, t + 4: components 4 W g ..
    uint32_t kp[2][2];                // keys g, g + 8: groups 2t, 2t + 1
    uint32_t vp[2][2];                // pairs t, t + 4: group g % 4, even and odd slot
};
// A warp's ring of blocks in shared memory, filled by 16-byte asynchronous copies kRing - 1 blocks ahead: the loads in
// flight cost no registers (with one block ahead in registers, 41 KB per SM, the 64-request case ran at 62 % of the copy
// rate).  Each block is four pieces that lie together in the layer: 16 rows of K codes, 8 pairs of V codes, their
// parameters.
constexpr int kRing = 4;  // (5 blocks: 216 us, 6: 235, 3: 222 at five CTAs per SM)
template <int D>
struct Kv4Ring {
    static constexpr int W = D / 32;
    uint8_t kc[kRing][16][D / 2];
    uint8_t vc[kRing][8][D];
    uint32_t kp[kRing][16][W];
    uint32_t vp[kRing][8][W][2];
};
__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Where a lane's copies come from; the warp's next block is a constant step.
template <int D>
struct Kv4Source {
    static constexpr int W = D / 32, kCode = D / 2, kPar = D / 8;  // 16-byte pieces of codes (K or V), of parameters
    const uint8_t *kc, *vc, *par;
    __device__ __forceinline__ Kv4Source(const Kv4View &v, int h, int64_t b, int lane) {
        const int64_t row = (int64_t)h * v.S + b;
        kc = v.kc + row * (D / 2) + lane * 16;
        vc = v.vc + row * (D / 2) + lane * 16;
        par = lane < kPar ? (const uint8_t *)(v.kp + row * W) + lane * 16
                          : (const uint8_t *)(v.vp + row * W) + (lane - kPar) * 16;
    }
    __device__ __forceinline__ void copy(Kv4Ring<D> &r, int stage, int lane) {
#pragma unroll
        for (int c = 0; c < kCode; c += 32)
            if (kCode >= 32 || lane < kCode) {
                copy16(&r.kc[stage][0][0] + (c + lane) * 16, kc + c * 16);
                copy16(&r.vc[stage][0][0] + (c + lane) * 16, vc + c * 16);
            }
        if (lane < kPar) copy16((uint8_t *)&r.kp[stage][0][0] + lane * 16, par);
        else if (lane < 2 * kPar) copy16((uint8_t *)&r.vp[stage][0][0][0] + (lane - kPar) * 16, par);
        kc += 8 * D * kKvWarps, vc += 8 * D * kKvWarps, par += 64 * W * kKvWarps;
    }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Nibbles N and N + 4 of a word as fp16: N even, the value c 2^-24 (a subnormal: the bits themselves); N odd, c 2^-20.
// Two of the four pairs need no shift, and nothing is added that the product would have to lose again.
template <int N>
__device__ __forceinline__ uint32_t code_pair_f16(uint32_t w) {
    return (N < 2 ? w : w >> 8) & (N % 2 ? 0x00f000f0u : 0x000f000fu);
}
__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ void kv4_mma_f16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kDecodeCtas = 4;  // per SM (the 64-request case: four 213 us, five 223, six 233)
template <int D>
__global__ void __launch_bounds__(kKvThreads, kDecodeCtas) kv4_decode_mma_kernel(const Kv4Attn a) {
    constexpr int W = D / 32;
    constexpr unsigned kAll = 0xffffffffu;
    __shared__ __align__(16) union {
        Kv4Ring<D> ring[kKvWarps];
        Kv4Merge<D> merge;  // once the rings are done with
    } shared;
    Kv4Merge<D> &sm = shared.merge;
    pdl_trigger();
    pdl_wait();
    const int item = blockIdx.x / a.n_heads, h = blockIdx.x - item * a.n_heads;
    const int4 r0 = reinterpret_cast<const int4 *>(a.items)[2 * item],
               r1 = reinterpret_cast<const int4 *>(a.items)[2 * item + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // slots relative to the chunk's first block of 16 (S is a multiple of 16: a block never leaves the layer)
    const int64_t base = r0.x & ~15;
    const int s0 = r0.x & 15, s1 = s0 + r0.y;
    int b = 16 * warp, ahead = b;
    constexpr int kStep = 16 * kKvWarps;
    Kv4Ring<D> &ring = shared.ring[warp];
    Kv4Source<D> src(a.v, h, base + b, lane);
#pragma unroll
    for (int n = 0; n < kRing - 1; ++n, ahead += kStep) {
        if (ahead < s1) src.copy(ring, n, lane);
        copies_commit();
    }

    // q in fp16, its largest magnitude brought to 2^14 by a power of two (bf16 has fewer bits: nothing is lost down to
    // 2^-28 of that).  Word w of a lane covers components 8 (W t + w) ..; pairs (n, n + 4), those of odd n over 16.
    uint32_t qf[W][4];
    float qsum[2], q_inv;  // sums of q over groups 2t and 2t + 1
    {
        const bf16 *q = (const bf16 *)a.qkv + (size_t)r0.z * 3 * a.H + h * D + 8 * W * t;
        const bool mine = g == (t * W) / 4;
        float x[W][8], sum = 0.f, big = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            load16(q + 8 * w, x[w]);
#pragma unroll
            for (int n = 0; n < 8; ++n) sum += x[w][n], big = max_nan(big, fabsf(x[w][n]));
        }
        big = max_nan(big, __shfl_xor_sync(kAll, big, 1));
        big = max_nan(big, __shfl_xor_sync(kAll, big, 2));
        q_inv = kv4_inverse_scale(big);
        const float f = 1.f / q_inv;
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float fn = n % 2 ? f * 0.0625f : f;
                qf[w][n] = mine ? pack2_f16(x[w][n] * fn, x[w][n + 4] * fn) : 0u;
            }
        float of[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) of[j] = __shfl_sync(kAll, sum, j);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            qsum[j] = 0.f;
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
                if ((tt * W) / 4 == 2 * t + j) qsum[j] += of[tt];
            qsum[j] *= a.scale_log2;
        }
        q_inv *= a.scale_log2;
    }
    float m = kLow, l = 0.f, zero = 0.f, o[2 * W][4];
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    auto step = [&](const Kv4Block<D> &x, int here) {
        // scores of keys g and g + 8
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w) {
            kv4_mma_f16(c, code_pair_f16<0>(x.k[0][w]), code_pair_f16<0>(x.k[1][w]), code_pair_f16<1>(x.k[0][w]),
                        code_pair_f16<1>(x.k[1][w]), qf[w][0], qf[w][1]);
            kv4_mma_f16(c, code_pair_f16<2>(x.k[0][w]), code_pair_f16<2>(x.k[1][w]), code_pair_f16<3>(x.k[0][w]),
                        code_pair_f16<3>(x.k[1][w]), qf[w][2], qf[w][3]);
        }
        float sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float s = 0.f;
            if (2 * t < W) {  // (the other lanes' columns hold no group)
                const float u = fmaf(bf_lo(x.kp[i][0]), c[2 * i], bf_lo(x.kp[i][1]) * c[2 * i + 1]) * 16777216.f;
                s = fmaf(u, q_inv, fmaf(bf_hi(x.kp[i][0]), qsum[0], bf_hi(x.kp[i][1]) * qsum[1]));
            }
            if (W == 4) s += __shfl_xor_sync(kAll, s, 1);
            sc[i] = s;
        }
        // from lanes t = 0 to the key's other lanes: for W = 4 lanes 0 and 1 have the sum
#pragma unroll
        for (int i = 0; i < 2; ++i) sc[i] = __shfl_sync(kAll, sc[i], lane & ~3);
        const bool whole = here >= s0 && here + 16 <= s1;  // warp-uniform
        bool v_lo = true, v_hi = true;
        if (!whole) {
            v_lo = here + g >= s0 && here + g < s1;
            v_hi = here + g + 8 >= s0 && here + g + 8 < s1;
            if (!v_lo) sc[0] = kLow;
            if (!v_hi) sc[1] = kLow;
        }
        float mx = fmaxf(sc[0], sc[1]);
        if (__any_sync(kAll, mx > m)) {
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
            const float corr = ex2(m - mx);
            m = mx;
            l *= corr, zero *= corr;
#pragma unroll
            for (int i = 0; i < 2 * W; ++i) o[i][0] *= corr, o[i][1] *= corr, o[i][2] *= corr, o[i][3] *= corr;
        }
        const float p_lo = v_lo ? ex2(sc[0] - m) : 0.f, p_hi = v_hi ? ex2(sc[1] - m) : 0.f;
        l += p_lo + p_hi;
        // weights of keys 2t, 2t + 1, 2t + 8, 2t + 9 in group g % 4
        uint32_t bw[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float pe = __shfl_sync(kAll, i ? p_hi : p_lo, 8 * t), po = __shfl_sync(kAll, i ? p_hi : p_lo, 8 * t + 4);
            float se = bf_lo(x.vp[i][0]), me = bf_hi(x.vp[i][0]), so = bf_lo(x.vp[i][1]), mo = bf_hi(x.vp[i][1]);
            if (!whole) {  // an unused slot's parameters may be anything
                const int slot = here + 8 * i + 2 * t;
                if (slot < s0 || slot >= s1) se = me = 0.f;
                if (slot + 1 < s0 || slot + 1 >= s1) so = mo = 0.f;
            }
            const float we = pe * se, wo = po * so;
            zero = fmaf(8.f, we + wo, fmaf(pe, me, fmaf(po, mo, zero)));
            const uint32_t hi = pack2(we, wo);
            const uint32_t left = pack2(we - bf_lo(hi), wo - bf_hi(hi));
            bw[i] = (g & 3) >= W ? 0u : g < 4 ? hi : left;
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
            kv4_mma(o[2 * w], code_pair_centred<0>(x.v[0][w]), code_pair_centred<1>(x.v[0][w]),
                    code_pair_centred<0>(x.v[1][w]), code_pair_centred<1>(x.v[1][w]), bw[0], bw[1]);
            kv4_mma(o[2 * w + 1], code_pair_centred<2>(x.v[0][w]), code_pair_centred<3>(x.v[0][w]),
                    code_pair_centred<2>(x.v[1][w]), code_pair_centred<3>(x.v[1][w]), bw[0], bw[1]);
        }
    };
    for (int stage = 0; b < s1; b += kStep, ahead += kStep) {
        copies_wait<kRing - 2>();
        __syncwarp();  // the block is there for every lane, and every lane is done with the one before
        if (ahead < s1) src.copy(ring, stage == 0 ? kRing - 1 : stage - 1, lane);
        copies_commit();
        Kv4Block<D> x;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            get_words<W>(&ring.kc[stage][g + 8 * i][t * 4 * W], x.k[i]);
            get_words<W>(&ring.vc[stage][t + 4 * i][g * 4 * W], x.v[i]);
            if constexpr (W > 1) get_words<2>(&ring.kp[stage][g + 8 * i][W == 4 ? 2 * (t & 1) : 0], x.kp[i]);
            else x.kp[i][0] = ring.kp[stage][g + 8 * i][0], x.kp[i][1] = 0u;
            get_words<2>(&ring.vp[stage][t + 4 * i][g & (W - 1)][0], x.vp[i]);
        }
        step(x, b);
        stage = stage == kRing - 1 ? 0 : stage + 1;
    }
    __syncthreads();  // the merge takes the rings' place
    // l over the keys of a lane's column; the minima's part over the keys of its group
    l += __shfl_xor_sync(kAll, l, 4);
    l += __shfl_xor_sync(kAll, l, 8);
    l += __shfl_xor_sync(kAll, l, 16);
    zero += __shfl_xor_sync(kAll, zero, 1);
    zero += __shfl_xor_sync(kAll, zero, 2);
    // row g of o[2w + j] is component 4 (W g + w) + 2j of group W g / 8, row g + 8 the one after it; that
    // group's column and its remainder's are 2t + (group & 1) at t = group / 2 and t = group / 2 + 2
    const int gr = W * g / 8;
    const float z = __shfl_sync(kAll, zero, 4 * gr);
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float *c = o[2 * w + j];
            float e0 = (gr & 1) ? c[1] : c[0], e1 = (gr & 1) ? c[3] : c[2];
            e0 += __shfl_xor_sync(kAll, e0, 2);
            e1 += __shfl_xor_sync(kAll, e1, 2);
            if (t == gr / 2) {
                float *dst = &sm.o[warp][4 * (W * g + w) + 2 * j];
                dst[0] = e0 + z, dst[1] = e1 + z;
            }
        }
    if (lane == 0) sm.m[warp] = m, sm.l[warp] = l;
    kv4_finish<bf16, D>(a, sm, r0, r1, h);
}

// Up to 16 rows of one request at a time: the rows are the A operand's 16 rows, so 16 keys are unpacked once for all
// of them.  Item = (16 rows, chunk of keys) x head, four warps taking 16 keys each in turn.  A head of 16 components
// is half a group, the rest of it zero.
//   S    A = q, B = 128 + c of 8 keys; two MMAs per group of components, whose sums the key's s and m then apply to.
//   O    A = p s of the group, as two bf16 (16 bits kept), B = c - 8 of 8 components of that group; the part of the
//        minima, sum p (m + 8 s), in fp32.
// fp32: q and the weights in three bf16 parts (24 bits), K's codes centred too, each 16 keys' sum added in fp32: errors
// as in fp32 throughout.  4 requests of <= 200 rows over <= 500 keys, 30 heads of 128: 84 us, against 578 row by row
// on kv4_decode_kernel; 30 heads of 16, 4 x <= 1000 rows over <= 800 keys, bf16: 198 and 1109.
// P leaves the first product in the very registers that the second one takes it from.
// Bound by issue and latency: 9 requests of <= 7 rows over <= 1500 keys, 32 heads of 128, 39 us (row by row 65), 51 MB:
// 7.6 us at the copy rate; the schedulers issue in 52 % of active cycles, three CTAs of 168 registers per SM.
constexpr int kRowsPerItem = 16;

template <typename T, int D>
struct Kv4RowsMerge {
    static constexpr int Q = std::is_same<T, float>::value ? 3 : 1;  // bf16 parts of q
    float m[kKvWarps][kRowsPerItem], l[kKvWarps][kRowsPerItem];
    float o[kKvWarps][kRowsPerItem][D];
    uint4 q[Q][D >= 32 ? D / 32 : 1][2][32];  // q as the A operand: part, group, half of it, lane
};

// The bf16 nearest to two floats; what it leaves of them stays.
__device__ __forceinline__ uint32_t bf_part(float &a, float &b) {
    const uint32_t u = pack2(a, b);
    a -= bf_lo(u), b -= bf_hi(u);
    return u;
}

// Half: every item of the launch has at most 8 rows, and the A operand's rows 8 .. 15 are zero.
template <typename T, int D, bool Half>
__device__ __forceinline__ void kv4_rows_item(const Kv4Attn &a, Kv4RowsMerge<T, D> &sm, const int4 r0, const int4 *rec,
                                              int h) {
    constexpr bool F32 = std::is_same<T, float>::value;
    constexpr int W = D >= 32 ? D / 32 : 1;  // groups
    constexpr int R = Half ? 1 : 2;  // row g, and g + 8
    constexpr unsigned kAll = 0xffffffffu;
    using Merge = Kv4RowsMerge<T, D>;
    // r0: first slot, keys, first row, rows; then the rows' chunks, this chunk, first partial, prompt (wide items) (read
    // late: registers); r2.x: keys that row 0 sees
    const int4 r2 = rec[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t s0 = r0.x, s1 = s0 + r0.y;
    const int rows = r0.w;

    float qsum[W][2];  // rows g and g + 8
#pragma unroll
    for (int y = 0; y < W; ++y) {
        float x[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
            if (i < R && g + 8 * i < rows && 32 * y + 8 * t < D) {
                const T *q = (const T *)a.qkv + (size_t)(r0.z + g + 8 * i) * 3 * a.H + h * D + 32 * y + 8 * t;
#pragma unroll
                for (int e = 0; e < 8; e += Elem<T>::kPer16) load16(q + e, x[i] + e);
            }
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += x[i][e];
            s += __shfl_xor_sync(kAll, s, 1);
            s += __shfl_xor_sync(kAll, s, 2);
            qsum[y][i] = s;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (warp == (2 * y + k) % kKvWarps) {
#pragma unroll
                for (int n = 0; n < Merge::Q; ++n)
                    sm.q[n][y][k][lane] = make_uint4(bf_part(x[0][2 * k], x[0][2 * k + 4]), bf_part(x[1][2 * k], x[1][2 * k + 4]),
                                                     bf_part(x[0][2 * k + 1], x[0][2 * k + 5]),
                                                     bf_part(x[1][2 * k + 1], x[1][2 * k + 5]));
            }
    }
    __syncthreads();
    float m[2] = {kLow, kLow}, l[2] = {0.f, 0.f}, zero[W][2], o[W][4][4];
#pragma unroll
    for (int y = 0; y < W; ++y) {
        zero[y][0] = zero[y][1] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[y][j][0] = o[y][j][1] = o[y][j][2] = o[y][j][3] = 0.f;
    }
    for (int64_t b = (s0 & ~int64_t(15)) + 16 * warp; b < s1; b += 16 * kKvWarps) {
        const int64_t row = (int64_t)h * a.v.S + b, pair = row >> 1;
        if (b + 16 * kKvWarps < s1) {  // the warp's next 16 slots into L1, a line per lane (16 slots are whole lines)
            constexpr int kCode = 16 * D / 2 / 128, kPar = 16 * W * 4 / 128 > 0 ? 16 * W * 4 / 128 : 1;
            const int64_t next = row + 16 * kKvWarps;
            const uint8_t *p = lane < kCode               ? a.v.kc + next * (D / 2) + lane * 128
                               : lane < 2 * kCode         ? a.v.vc + next * (D / 2) + (lane - kCode) * 128
                               : lane < 2 * kCode + kPar  ? (const uint8_t *)(a.v.kp + next * W) + (lane - 2 * kCode) * 128
                                                          : (const uint8_t *)(a.v.vp + next * W) + (lane - 2 * kCode - kPar) * 128;
            if (lane < 2 * (kCode + kPar)) prefetch_l1(p);
        }
        uint32_t kw[2][W], vw[2][W], kp[4][W], vp[2][2 * W];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t *kc = reinterpret_cast<const uint32_t *>(a.v.kc + (row + g + 8 * i) * (D / 2)) + t;
            const uint32_t *vc = reinterpret_cast<const uint32_t *>(a.v.vc + (pair + t + 4 * i) * D) + g;
#pragma unroll
            for (int y = 0; y < W; ++y) {
                kw[i][y] = D >= 32 || t < D / 8 ? kc[4 * y] : 0u;  // (q is zero there)
                vw[i][y] = D >= 32 || g < D / 4 ? vc[8 * y] : 0u;  // (columns that are not used)
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) load_words<W>(a.v.kp + (row + 8 * i + 2 * t + e) * W, kp[2 * i + e]);
            if constexpr (W == 4) {
                load_words<4>(a.v.vp + (pair + t + 4 * i) * 8, vp[i]);
                load_words<4>(a.v.vp + (pair + t + 4 * i) * 8 + 4, vp[i] + 4);
            } else {
                load_words<2 * W>(a.v.vp + (pair + t + 4 * i) * (2 * W), vp[i]);
            }
        }
        // scores: c[i][..] = keys 8 i + 2 t, + 1 of rows g (0, 1) and g + 8 (2, 3)
        float sc[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
            for (int y = 0; y < W; ++y) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t w = kw[i][y];
                if constexpr (F32) {
                    const uint32_t b[4] = {code_pair_centred<0>(w), code_pair_centred<1>(w), code_pair_centred<2>(w),
                                           code_pair_centred<3>(w)};
#pragma unroll
                    for (int n = Merge::Q - 1; n >= 0; --n) {
                        const uint4 qa = sm.q[n][y][0][lane], qb = sm.q[n][y][1][lane];
                        kv4_mma(c, qa.x, qa.y, qa.z, qa.w, b[0], b[1]);
                        kv4_mma(c, qb.x, qb.y, qb.z, qb.w, b[2], b[3]);
                    }
                } else {
                    c[0] = c[1] = -128.f * qsum[y][0], c[2] = c[3] = -128.f * qsum[y][1];
                    const uint4 qa = sm.q[0][y][0][lane], qb = sm.q[0][y][1][lane];
                    kv4_mma(c, qa.x, qa.y, qa.z, qa.w, code_pair<0>(w), code_pair<1>(w));
                    kv4_mma(c, qb.x, qb.y, qb.z, qb.w, code_pair<2>(w), code_pair<3>(w));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float s = bf_lo(kp[2 * i + e][y]), z0 = bf_hi(kp[2 * i + e][y]), z = F32 ? fmaf(8.f, s, z0) : z0;
                    sc[i][e] = fmaf(s, c[e], fmaf(z, qsum[y][0], sc[i][e]));
                    if (!Half) sc[i][2 + e] = fmaf(s, c[2 + e], fmaf(z, qsum[y][1], sc[i][2 + e]));
                }
            }
        }
        // causal: row j of the item sees the chunk's first r2.x + j keys (the chunk itself ends at s1)
        const bool whole = b >= s0 && b + 16 <= s1 && b + 16 - s0 <= r2.x;
        const int first = (int)(b - s0) + 2 * t;  // this lane's first key, in the chunk
        float mx[2] = {kLow, kLow};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 2 * R; ++e) {
                sc[i][e] *= a.scale_log2;
                if (!whole) {
                    const int key = first + 8 * i + (e & 1), j = g + 8 * (e >> 1);
                    if (key < 0 || key >= r0.y || key >= r2.x + j) sc[i][e] = -INFINITY;
                }
                mx[e >> 1] = fmaxf(mx[e >> 1], sc[i][e]);
            }
        bool grown = false;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(kAll, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(kAll, mx[i], 2));
            grown |= mx[i] > m[i];
        }
        if (__any_sync(kAll, grown)) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float n = fmaxf(m[i], mx[i]), corr = ex2(m[i] - n);
                m[i] = n;
                l[i] *= corr;
#pragma unroll
                for (int y = 0; y < W; ++y) {
                    zero[y][i] *= corr;
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[y][j][2 * i] *= corr, o[y][j][2 * i + 1] *= corr;
                }
            }
        }
        float p[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 2 * R; ++e) {
                p[i][e] = ex2(sc[i][e] - m[e >> 1]);  // (-inf: 0)
                if (!whole && sc[i][e] == -INFINITY) p[i][e] = -0.f;  // marks what the row does not see
                l[e >> 1] += p[i][e];
            }
#pragma unroll
        for (int y = 0; y < W; ++y) {
            // A: rows g, g + 8 at keys 2t, 2t + 1 (a0, a1) and 2t + 8, 2t + 9 (a2, a3)
            uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u}, rest[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float se = bf_lo(vp[i][2 * y]), me = bf_hi(vp[i][2 * y]), so = bf_lo(vp[i][2 * y + 1]),
                            mo = bf_hi(vp[i][2 * y + 1]);
                const float ze = fmaf(8.f, se, me), zo = fmaf(8.f, so, mo);
#pragma unroll
                for (int x = 0; x < R; ++x) {  // row g + 8 x
                    const float pe = p[i][2 * x], po = p[i][2 * x + 1];
                    float we = pe * se, wo = po * so, ye = pe * ze, yo = po * zo;
                    if (!whole) {  // what a row does not see may hold anything, 0 times which may be NaN
                        if (__float_as_uint(pe) == 0x80000000u) we = ye = 0.f;
                        if (__float_as_uint(po) == 0x80000000u) wo = yo = 0.f;
                    }
                    zero[y][x] += ye + yo;
                    hi[2 * i + x] = bf_part(we, wo);
                    lo[2 * i + x] = bf_part(we, wo);
                    if (F32) rest[2 * i + x] = pack2(we, wo);
                }
            }
            const uint32_t c0[4] = {code_pair_centred<0>(vw[0][y]), code_pair_centred<1>(vw[0][y]),
                                    code_pair_centred<2>(vw[0][y]), code_pair_centred<3>(vw[0][y])};
            const uint32_t c1[4] = {code_pair_centred<0>(vw[1][y]), code_pair_centred<1>(vw[1][y]),
                                    code_pair_centred<2>(vw[1][y]), code_pair_centred<3>(vw[1][y])};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (F32) {  // (these 16 keys' sum by itself: the tensor core cuts off where fp32 rounds)
                    float n[4] = {0.f, 0.f, 0.f, 0.f};
                    kv4_mma(n, rest[0], rest[1], rest[2], rest[3], c0[j], c1[j]);
                    kv4_mma(n, lo[0], lo[1], lo[2], lo[3], c0[j], c1[j]);
                    kv4_mma(n, hi[0], hi[1], hi[2], hi[3], c0[j], c1[j]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[y][j][e] += n[e];
                } else {
                    kv4_mma(o[y][j], hi[0], hi[1], hi[2], hi[3], c0[j], c1[j]);
                    kv4_mma(o[y][j], lo[0], lo[1], lo[2], lo[3], c0[j], c1[j]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        l[i] += __shfl_xor_sync(kAll, l[i], 1);
        l[i] += __shfl_xor_sync(kAll, l[i], 2);
        if (t == 0) sm.m[warp][g + 8 * i] = m[i], sm.l[warp][g + 8 * i] = l[i];
#pragma unroll
        for (int y = 0; y < W; ++y) {
            float z = zero[y][i];
            z += __shfl_xor_sync(kAll, z, 1);
            z += __shfl_xor_sync(kAll, z, 2);
            // columns 2t and 2t + 1 of o[y][j]: components 32 y + 8 t + j and + 4
            if (8 * t >= D) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sm.o[warp][g + 8 * i][32 * y + 8 * t + j] = o[y][j][2 * i] + z;
                sm.o[warp][g + 8 * i][32 * y + 8 * t + 4 + j] = o[y][j][2 * i + 1] + z;
            }
        }
    }
    __syncthreads();
    // join the warps; of several chunks, the partials are joined by the next kernel
    const int4 r1 = rec[1];
    const int nch = r1.x;
    for (int x = 2 * threadIdx.x; x < rows * D; x += 2 * kKvThreads) {  // two components
        const int j = x / D, d = x - j * D;
        float M = kLow, L = 0.f, O[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kKvWarps; ++w) M = fmaxf(M, sm.m[w][j]);
#pragma unroll
        for (int w = 0; w < kKvWarps; ++w) {
            const float c = ex2(sm.m[w][j] - M);
            const float2 o2 = *reinterpret_cast<const float2 *>(&sm.o[w][j][d]);
            L += sm.l[w][j] * c, O[0] += o2.x * c, O[1] += o2.y * c;
        }
        if (nch == 1) {
            T *dst = (T *)a.out + (size_t)(r0.z + j) * a.H + h * D + d;
            if constexpr (F32) *reinterpret_cast<float2 *>(dst) = make_float2(O[0] / L, O[1] / L);
            else *reinterpret_cast<uint32_t *>(dst) = pack2(O[0] / L, O[1] / L);
        } else {
            float *mine = a.row_part + (((size_t)(r1.z + r1.y) * a.n_heads + h) * kRowsPerItem + j) * (D + 2);
            *reinterpret_cast<float2 *>(mine + d) = make_float2(O[0], O[1]);
            if (d == 0) mine[D] = M, mine[D + 1] = L;
        }
    }
}

template <typename T, int D, bool Half>
__global__ void __launch_bounds__(kKvThreads, 3) kv4_rows_mma_kernel(const Kv4Attn a) {
    __shared__ Kv4RowsMerge<T, D> sm;
    pdl_trigger();
    pdl_wait();
    const int item = blockIdx.x / a.n_heads, h = blockIdx.x - item * a.n_heads;
    const int4 *rec = reinterpret_cast<const int4 *>(a.row_items) + 3 * item;
    kv4_rows_item<T, D, Half>(a, sm, rec[0], rec, h);
}

// The rows of the prompts' marked heads again, over what the prefill kernel made of them.  As many blocks as run at
// once: a call without marks costs one look at them.
template <int D>
__global__ void __launch_bounds__(kKvThreads, 3) kv4_rows_wide_kernel(const Kv4Attn a) {
    __shared__ Kv4RowsMerge<bf16, D> sm;
    pdl_trigger();
    int any = 0;  // (the marks are there: the prefill kernel triggers behind its wait)
    for (int i = threadIdx.x; i < a.n_wide; i += kKvThreads) any |= __ldcg(a.wide + i);
    pdl_wait();
    if (!__syncthreads_or(any)) return;
    for (int64_t j = blockIdx.x; j < (int64_t)a.n_wide_items * a.n_heads; j += gridDim.x) {
        const int item = (int)(j / a.n_heads), h = (int)(j - (int64_t)item * a.n_heads);
        const int4 *rec = reinterpret_cast<const int4 *>(a.wide_items) + 3 * (int64_t)item;
        if (!a.wide[rec[1].w * a.n_heads + h]) continue;
        kv4_rows_item<bf16, D, false>(a, sm, rec[0], rec, h);
        __syncthreads();
    }
}

// The chunks' partials of one group of rows and head, a warp per row.  (A launch of its own: the last block of a group
// joining them alone took longer than the attention, 16 rows of 130 floats for every chunk.)
template <typename T, int D>
__global__ void __launch_bounds__(32 * kRowsPerItem) kv4_rows_join_kernel(const Kv4Attn a) {
    pdl_trigger();
    pdl_wait();
    const int4 r = reinterpret_cast<const int4 *>(a.row_joins)[blockIdx.x];  // first row, rows, chunks, first partial
    const int h = blockIdx.y, j = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (j >= r.y) return;
    const float *part = a.row_part + (((size_t)r.w * a.n_heads + h) * kRowsPerItem + j) * (D + 2);
    T *dst = (T *)a.out + (size_t)(r.x + j) * a.H + h * D;
#pragma unroll
    for (int d = lane; d < D; d += 32)
        dst[d] = Elem<T>::from_f(kv4_join<D>(part, (size_t)a.n_heads * kRowsPerItem * (D + 2), r.z, d));
}

// f(head_dim as a constant)
template <typename F>
cudaError_t for_dim(int d, F f) {
    switch (d) {
        case 16: return f(std::integral_constant<int, 16>());
        case 32: return f(std::integral_constant<int, 32>());
        case 64: return f(std::integral_constant<int, 64>());
        case 128: return f(std::integral_constant<int, 128>());
        default: return cudaErrorInvalidValue;
    }
}

template <typename T>
cudaError_t launch_decode(const Kv4Attn &a, int d, int n_items, cudaStream_t st) {
    const dim3 grid((unsigned)n_items * a.n_heads), block(kKvThreads);
    return for_dim(d, [&](auto dim) {
        if constexpr (std::is_same<T, bf16>::value && dim() >= 32)
            return launch_pdl(kv4_decode_mma_kernel<dim()>, grid, block, 0, st, a);
        else
            return launch_pdl(kv4_decode_kernel<T, dim()>, grid, block, 0, st, a);
    });
}

// ---------------------------------------------------------------------------
// plans
// ---------------------------------------------------------------------------
constexpr int32_t kKv4Magic = 0x4B563450;
constexpr int kKv4Hdr = 64;
enum : int {
    Q_MAGIC = 0,
    Q_DTYPE,
    Q_HEADS,
    Q_DIM,
    Q_SLOTS,
    Q_ROWS,
    Q_ITEMS,     // work items of single rows
    Q_SPLITS,    // rows whose keys span several items
    Q_PARTS,     // partials of those rows
    Q_TILES,     // read-back tiles
    Q_KEYS,      // keys of all requests
    Q_TWICE,     // a slot is written by two rows of the batch
    Q_TOTAL,
    Q_UNITS,     // rows to write, by ones and by twos that share a pair of slots
    Q_O_UNITS,   // word offsets of the tables
    Q_O_ITEMS,
    Q_O_COUNT,
    Q_O_TILES,
    Q_PRE,       // prompts: requests whose rows run on the prefill kernel
    Q_PRETILES,  // their (request, 128 rows) tiles
    Q_PREREAD,   // read-back tiles of their slots
    Q_PREKEYS,   // their slots
    Q_REQS,
    Q_O_PRE,
    Q_O_PRETILES,
    Q_O_PREREAD,
    Q_O_REQOFF,
    Q_O_REQCTX,
    Q_RITEMS,   // work items of groups of rows, their partials and the groups that have some
    Q_RPARTS,
    Q_RJOINS,
    Q_RHALF,  // no group has more than 8 rows
    Q_O_RITEMS,
    Q_O_RJOINS,
    Q_O_REQWS,  // a prompt's first slot in the workspace's pool
    Q_TILEMOST,  // slots of the longest read-back tile
    Q_WIDE,      // the prompts' rows in groups, for heads that fp16 does not hold
    Q_O_WIDE,
};
int64_t up4(int64_t w) { return (w + 3) & ~int64_t(3); }

// How a request's rows are attended: on the prefill kernel, in groups of rows, or row by row.
enum Kv4Form { kPromptForm, kGroupForm, kRowForm };
enum Kv4Several { kAllGroups, kAllPrompts, kByRequest };  // requests of several rows
struct Kv4Policy {
    Kv4Several several = kAllGroups;
    bool singles_grouped = false;
};
bool prompts_possible(const Kv4Batch &b) { return b.dtype == 1 && b.head_dim >= 64; }

// Time of the two forms (us), by a model of their launches: a start (prompts: of three more), a time per key of the
// longest request (its chunks, or the walk of one tile of 128 rows over it), and a time per key, head and group of 16
// rows, or tile of 128, that reads it.  Measured at 152 SMs, 4 requests of <= 20 / 40 / 60 / 100 / 200 rows over <= 1500
// keys, 30 heads: of 64, in groups 22 / 31 / 44 / 59 / 108 us and as prompts 33 / 35 / 35 / 35 / 49; of 128, 37 / 52 / 75 /
// 100 / 185 and 49 / 54 / 55 / 56 / 75; one request of 200 rows alone, 5 heads of 128, 10 and 16.
struct Kv4Cost {
    struct {
        double start, longest, each;
    } group, tile;
};
Kv4Cost cost_of(const Kv4Batch &b) {
    return b.head_dim == 64 ? Kv4Cost{{4.5, 0.0045, 65e-6}, {11, 0.0085, 90e-6}}
                            : Kv4Cost{{5, 0.0085, 110e-6}, {13, 0.011, 210e-6}};
}
double group_time(const Kv4Batch &b, int i) {
    const double n = b.n_input[i], g = (b.n_input[i] + kRowsPerItem - 1) / kRowsPerItem;
    return cost_of(b).group.each * b.n_heads * (g * b.ctx_len[i] + kRowsPerItem / 2 * g * (g - 1) + n);
}
double tile_time(const Kv4Batch &b, int i) {
    const double n = b.n_input[i], t = (b.n_input[i] + kPrefillRowsPerTile - 1) / kPrefillRowsPerTile;
    return cost_of(b).tile.each * b.n_heads * (t * b.ctx_len[i] + kPrefillRowsPerTile / 2 * t * (t - 1) + n);
}
Kv4Form form_of(const Kv4Batch &b, int i, const Kv4Policy &p) {
    if (b.n_input[i] == 1) return p.singles_grouped ? kGroupForm : kRowForm;
    return p.several == kAllPrompts || (p.several == kByRequest && tile_time(b, i) < group_time(b, i)) ? kPromptForm
                                                                                                     : kGroupForm;
}

// Single rows among groups of rows: in a launch of their own, or, while that would take longer to start and to end than
// its keys are worth, as groups of one row.  One request of 5 rows and single rows of so many keys x heads in all, bf16,
// as groups and apart: head_dim 64, 23k 8.1 and 14.5 us, 187k 15.9 and 18.1, 316k 23.9 and 21.2, 1220k 62 and 39;
// head_dim 128, 187k 24.4 and 24.8, 316k 37 and 31; fp32, 64: 187k 18.4 and 22.8, 316k 28 and 27.
constexpr int64_t kGroupedKeys = 200000;
Kv4Policy policy_of(const Kv4Batch &b) {
    Kv4Policy p;
    if (prompts_possible(b)) {
        const Kv4Cost c = cost_of(b);
        double groups = 0, tiles = 0, longest = 0;  // of all
        double some_groups = 0, some_tiles = 0, longest_group = 0, longest_tile = 0;  // each request as it is cheaper
        for (int i = 0; i < b.n_req; ++i) {
            if (b.n_input[i] == 1) continue;
            const double g = group_time(b, i), t = tile_time(b, i), keys = (double)b.ctx_len[i] + b.n_input[i];
            groups += g, tiles += t, longest = std::max(longest, keys);
            if (t < g) some_tiles += t, longest_tile = std::max(longest_tile, keys);
            else some_groups += g, longest_group = std::max(longest_group, keys);
        }
        const double as_groups = c.group.start + c.group.longest * longest + groups,
                     as_prompts = c.tile.start + c.tile.longest * longest + tiles,
                     split = c.group.start + c.group.longest * longest_group + some_groups + c.tile.start +
                             c.tile.longest * longest_tile + some_tiles;
        if (std::min(as_prompts, split) < as_groups) p.several = as_prompts <= split ? kAllPrompts : kByRequest;
    }
    int64_t keys = 0;
    bool any = false;
    for (int i = 0; i < b.n_req; ++i) {
        if (b.n_input[i] == 1) keys += b.ctx_len[i] + (int64_t)1;
        else any |= form_of(b, i, p) == kGroupForm;
    }
    p.singles_grouped = any && keys * b.n_heads <= kGroupedKeys;
    return p;
}

struct Kv4Sizes {
    int64_t rows = 0, units = 0, items = 0, splits = 0, parts = 0, tiles = 0, keys = 0;
    int64_t ritems = 0, rsplits = 0, rparts = 0;
    int64_t pre = 0, pre_tiles = 0, pre_read = 0, pre_keys = 0, wide = 0;
    int chunk = 0;
    int64_t rchunk = 0;
    Kv4Policy policy;
    int64_t off_ritems, off_rjoins, off_units, off_items, off_count, off_tiles, off_pre, off_pretiles, off_preread, off_reqoff, off_reqctx,
        off_reqws, off_wide, total;
};

// Keys per work item of rows one by one: the largest chunk (a power of two,
// 128 .. 2048 keys) that still gives every SM three blocks of four warps.  Short
// chunks cost a join: 16 requests of 300 keys, 40 heads of 128, took 18.2 us at
// six blocks per SM and 11.5 at three, one of 100 keys 5.1 us in chunks of 64 and
// 3.2 in one; one of 4000 keys 17.1 us at six, 13.8 at three, 19.7 at one.
// A row of few keys stays whole whatever the chunk.  One row, in chunks / whole, us at 350, 400, 450, 500, 550 and 600 keys
// (replayed from a graph): 20 heads of 64 5.0/4.3 5.0/4.7 5.0/5.1 5.0/5.3 5.3/5.6 5.4/6.0; 40 heads of 64 6.0/4.3 6.3/4.8
// 6.2/5.3 6.2/5.3 6.4/5.7 6.6/6.0; 40 heads of 128 6.9/5.5 7.1/5.9 7.1/6.5 7.2/6.5 6.9/7.2 6.4/7.7; two rows 7.9/6.6
// 7.9/7.6 7.9/8.3 7.8/8.5; 5 heads of 128 5.2/5.1 5.2/5.6; fp32, 12 heads of 64 4.9/5.1 4.9/6.1, 40 heads 6.3/5.2 6.4/6.1
// 6.5/6.3 6.5/6.3 5.7/7.6.  They cross between 350 and 620 keys by heads and type, in the middle at the value below.
constexpr int kWholeRow = 400;
int64_t row_items(int64_t keys, int chunk) { return keys <= kWholeRow ? 1 : (keys + chunk - 1) / chunk; }
int kv4_row_chunk(const Kv4Batch &b, const Kv4Policy &policy, int num_sms) {
    const int64_t most = 3LL * num_sms;
    int chunk = 2048;
    while (chunk > 128) {
        int64_t items = 0;
        for (int i = 0; i < b.n_req && items * b.n_heads < most; ++i)
            if (form_of(b, i, policy) == kRowForm)
                items += row_items(b.ctx_len[i] + (int64_t)1, chunk);
        if (items * b.n_heads >= most) break;
        chunk /= 2;
    }
    return chunk;
}

// The same for groups of rows, whose blocks are fewer and longer: the chunk with
// the least time by a simple model, in units of a key's time in a block -- the
// blocks' keys, 60 more for each block, over the blocks that run at once, half of
// the longest block (the last ones to start are the shortest), and 120 for the
// launch that joins chunks.  (9 requests of <= 7 rows over <= 1500 keys, 32 heads:
// 43.0 us in chunks of 512, 38.3 of 256, 51.2 of 1024; 8 requests of 2 rows over
// 300 keys, 40 heads: 13.4 us whole, 18.6 in chunks of 256.)  Partial outputs are
// written and read again, and what they take beyond 64 MiB is charged at the copy
// rate (a key's time in a block is about 0.05 us): a long prompt's many groups
// nearly fill the GPU whole (fp32, 32 heads of 128, 8192 rows behind 24576 keys:
// 52.5 ms and 1885 MiB in chunks of 2048, 49.3 ms and 260 MiB in 16384; 2048
// rows behind 30000: 14.2 ms and 509 MiB, 13.6 and 130).
int64_t kv4_group_chunk(const Kv4Batch &b, const Kv4Policy &policy, int num_sms) {
    const int64_t at_once = 3LL * num_sms;
    int64_t largest = 2048, best = 0;
    for (int i = 0; i < b.n_req; ++i)
        while (form_of(b, i, policy) == kGroupForm && largest < b.ctx_len[i] + (int64_t)b.n_input[i]) largest *= 2;
    double best_time = 0;
    for (int64_t chunk = largest; chunk >= 128; chunk /= 2) {
        int64_t keys = 0, items = 0, longest = 0, parts = 0;
        bool split = false;
        for (int i = 0; i < b.n_req; ++i) {
            if (form_of(b, i, policy) != kGroupForm) continue;
            const int64_t groups = (b.n_input[i] + kRowsPerItem - 1) / kRowsPerItem, k = b.ctx_len[i] + (int64_t)b.n_input[i];
            keys += groups * k;
            items += groups * ((k + chunk - 1) / chunk);
            longest = std::max(longest, std::min(k, chunk));
            split |= k > chunk;
            if (k > chunk) parts += groups * ((k + chunk - 1) / chunk);
        }
        const double bytes = 4.0 * parts * b.n_heads * kRowsPerItem * (b.head_dim + 2);
        const double time = (double)(keys + 60 * items) * b.n_heads / at_once + 0.5 * (longest + 60) + (split ? 120 : 0) +
                            2 * std::max(0.0, bytes - (64 << 20)) / (6.7e6 * 0.05);
        if (chunk == largest || time < best_time) best = chunk, best_time = time;
    }
    return best;
}

bool kv4_sizes(const Kv4Batch &b, int num_sms, Kv4Sizes *z) {
    int64_t rows = 0;
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t n = b.n_input[i], c = b.ctx_len[i], o = b.kv_offset[i];
        if (n < 1 || c < 0 || o < 0 || o > b.kv_slots || o + c + n > b.kv_slots) return false;
        rows += n;
        if (rows > INT32_MAX / 8) return false;
    }
    const Kv4Policy policy = z->policy = policy_of(b);
    z->chunk = kv4_row_chunk(b, policy, num_sms);
    z->rchunk = kv4_group_chunk(b, policy, num_sms);
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t n = b.n_input[i], c = b.ctx_len[i];
        z->rows += n;
        z->keys += c + n;
        z->units += n / 2 + (n % 2 || (b.kv_offset[i] + c) % 2 ? 1 : 0);
        z->tiles += (c + n + kReadTile - 1) / kReadTile;
        const Kv4Form form = form_of(b, i, policy);
        if (form == kPromptForm) {
            z->pre++;
            z->pre_tiles += (n + kPrefillRowsPerTile - 1) / kPrefillRowsPerTile;
            z->pre_read += (c + n + kReadTile - 1) / kReadTile;
            z->pre_keys += c + n;
            z->wide += (n + kRowsPerItem - 1) / kRowsPerItem;
            continue;
        }
        if (form == kGroupForm) {
            for (int64_t r = 0; r < n; r += kRowsPerItem) {
                const int64_t nch = (c + std::min<int64_t>(n, r + kRowsPerItem) + z->rchunk - 1) / z->rchunk;
                z->ritems += nch;
                if (nch > 1) z->rsplits++, z->rparts += nch;
            }
            continue;
        }
        const int64_t nch = row_items(c + 1, z->chunk);
        z->items += nch;
        if (nch > 1) z->splits++, z->parts += nch;
    }
    int64_t w = kKv4Hdr;
    z->off_units = w, w = up4(w + 4 * z->units);
    z->off_items = w, w = up4(w + 8 * z->items);
    z->off_count = w, w = up4(w + z->splits * b.n_heads);
    z->off_tiles = w, w = up4(w + 4 * z->tiles);
    z->off_ritems = w, w = up4(w + 12 * z->ritems);
    z->off_rjoins = w, w = up4(w + 4 * z->rsplits);
    z->off_pre = w, w = up4(w + 4 * z->pre);
    z->off_pretiles = w, w = up4(w + 2 * z->pre_tiles);
    z->off_preread = w, w = up4(w + 4 * z->pre_read);
    z->off_reqoff = w, w = up4(w + b.n_req + 1);
    z->off_reqctx = w, w = up4(w + b.n_req);
    z->off_reqws = w, w = up4(w + b.n_req);
    z->off_wide = w, w = up4(w + 12 * z->wide);
    z->total = w;
    // 32-bit table entries and grid sizes
    return w <= INT32_MAX && z->keys <= INT32_MAX && (z->items + z->ritems) * b.n_heads <= INT32_MAX && z->pre_tiles * b.n_heads <= INT32_MAX &&
           (z->pre + z->rows) * b.n_heads <= INT32_MAX;
}

}  // namespace

int kv4_groups(int head_dim) { return head_dim >= 32 ? head_dim / 32 : 1; }

int64_t kv4_layer_bytes(int n_heads, int head_dim, int64_t kv_slots) {
    const int64_t S = (kv_slots + 15) / 16 * 16;
    return n_heads * S * (head_dim + 8 * (int64_t)kv4_groups(head_dim));
}

int64_t kv4_plan_words(const Kv4Batch &b, int num_sms) {
    Kv4Sizes z;
    return kv4_sizes(b, num_sms, &z) ? z.total : -1;
}

namespace {
// Order records of N words by their second, largest first (stable).
template <int N>
void longest_first(int32_t *rec, int64_t n) {
    struct R {
        int32_t w[N];
    };
    R *r = reinterpret_cast<R *>(rec);
    std::stable_sort(r, r + n, [](const R &x, const R &y) { return x.w[1] > y.w[1]; });
}
}  // namespace

bool kv4_plan_build(const Kv4Batch &b, int num_sms, int32_t *buf, int64_t cap) {
    Kv4Sizes z;
    if (!kv4_sizes(b, num_sms, &z) || cap < z.total) return false;
    std::memset(buf, 0, sizeof(int32_t) * (size_t)z.total);  // (the device copy's counters start at zero)
    int32_t *un = buf + z.off_units, *it = buf + z.off_items, *tl = buf + z.off_tiles;
    int32_t *pre = buf + z.off_pre, *pt = buf + z.off_pretiles, *pd = buf + z.off_preread;
    int32_t *req_off = buf + z.off_reqoff, *req_ctx = buf + z.off_reqctx, *req_ws = buf + z.off_reqws;
    int32_t *ri = buf + z.off_ritems, *rj = buf + z.off_rjoins, *wd = buf + z.off_wide;
    int64_t row = 0, split = 0, part = 0, key = 0, ws = 0, rpart = 0;
    bool half = true;
    int32_t most = 0;
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t n = b.n_input[i], c = b.ctx_len[i], o = b.kv_offset[i];
        const Kv4Form form = form_of(b, i, z.policy);
        const bool prompt = form == kPromptForm;
        req_off[i] = (int32_t)row;
        req_ctx[i] = (int32_t)c;
        req_ws[i] = (int32_t)ws;
        for (int64_t j = 0; j < n; un += 4) {
            un[0] = (int32_t)(row + j);
            un[1] = (int32_t)(o + c + j);
            un[2] = (o + c + j) % 2 == 0 && j + 1 < n ? 2 : 1;
            j += un[2];
        }
        if (form == kRowForm) {
            const int64_t keys = c + 1, nch = row_items(keys, z.chunk), per = nch == 1 ? keys : z.chunk;
            for (int64_t k = 0; k < nch; ++k, it += 8) {
                it[0] = (int32_t)(o + k * per);
                it[1] = (int32_t)std::min<int64_t>(per, keys - k * per);
                it[2] = (int32_t)row;
                it[3] = (int32_t)nch;
                it[4] = (int32_t)k;
                it[5] = (int32_t)part;
                it[6] = (int32_t)split;
            }
            if (nch > 1) ++split, part += nch;
        }
        row += n;
        for (int64_t r = 0; form == kGroupForm && r < n; r += kRowsPerItem) {
            const int64_t rows = std::min<int64_t>(kRowsPerItem, n - r), keys = c + r + rows;
            const int64_t nch = (keys + z.rchunk - 1) / z.rchunk;
            for (int64_t k = 0; k < nch; ++k, ri += 12) {
                ri[0] = (int32_t)(o + k * z.rchunk);
                ri[1] = (int32_t)std::min<int64_t>(z.rchunk, keys - k * z.rchunk);
                ri[2] = (int32_t)(req_off[i] + r);
                ri[3] = (int32_t)rows;
                half &= rows <= 8;
                ri[4] = (int32_t)nch;
                ri[5] = (int32_t)k;
                ri[6] = (int32_t)rpart;
                ri[8] = (int32_t)(c + r + 1 - k * z.rchunk);
            }
            if (nch > 1) {
                rj[0] = (int32_t)(req_off[i] + r), rj[1] = (int32_t)rows, rj[2] = (int32_t)nch, rj[3] = (int32_t)rpart;
                rj += 4, rpart += nch;
            }
        }
        for (int64_t t = 0; t < c + n; t += kReadTile, tl += 4) {
            tl[0] = (int32_t)(o + t);
            tl[1] = (int32_t)std::min<int64_t>(kReadTile, c + n - t);
            most = std::max(most, tl[1]);
            tl[2] = (int32_t)(key + t);
            if (prompt) {
                std::memcpy(pd, tl, 4 * sizeof(int32_t));
                pd[2] = (int32_t)(ws + t);
                pd[3] = i;
                pd += 4;
            }
        }
        key += c + n;
        if (prompt) {
            const int32_t index = (int32_t)((pre - (buf + z.off_pre)) / 4);
            for (int64_t r = 0; r < n; r += kRowsPerItem, wd += 12) {
                const int64_t rows = std::min<int64_t>(kRowsPerItem, n - r);
                wd[0] = (int32_t)o, wd[1] = (int32_t)(c + r + rows), wd[2] = (int32_t)(req_off[i] + r), wd[3] = (int32_t)rows;
                wd[4] = 1, wd[7] = index, wd[8] = (int32_t)(c + r + 1);
            }
            pre[0] = i, pre[1] = (int32_t)o, pre[2] = (int32_t)(c + n);
            pre += 4;
            for (int64_t q = 0; q < n; q += kPrefillRowsPerTile, pt += 2) pt[0] = i, pt[1] = (int32_t)q;
            ws += c + n;
        }
    }
    req_off[b.n_req] = (int32_t)row;
    // blocks are dealt in order, all heads of an item after one another: the longest first, so that none starts late
    longest_first<8>(buf + z.off_items, z.items);
    longest_first<12>(buf + z.off_ritems, z.ritems);
    longest_first<12>(buf + z.off_wide, z.wide);
    prefill_order(buf + z.off_pretiles, (int)z.pre_tiles, req_off, req_ctx);
    // slots written by two rows
    std::vector<std::pair<int64_t, int64_t>> w((size_t)b.n_req);
    for (int i = 0; i < b.n_req; ++i)
        w[i] = {b.kv_offset[i] + b.ctx_len[i], b.kv_offset[i] + b.ctx_len[i] + b.n_input[i]};
    std::sort(w.begin(), w.end());
    bool twice = false;
    for (int i = 1; i < b.n_req; ++i) twice |= w[i].first < w[i - 1].second;
    buf[Q_MAGIC] = kKv4Magic;
    buf[Q_DTYPE] = b.dtype;
    buf[Q_HEADS] = b.n_heads;
    buf[Q_DIM] = b.head_dim;
    buf[Q_SLOTS] = (int32_t)b.kv_slots;
    buf[Q_ROWS] = (int32_t)z.rows;
    buf[Q_UNITS] = (int32_t)z.units;
    buf[Q_ITEMS] = (int32_t)z.items;
    buf[Q_SPLITS] = (int32_t)z.splits;
    buf[Q_PARTS] = (int32_t)z.parts;
    buf[Q_TILES] = (int32_t)z.tiles;
    buf[Q_KEYS] = (int32_t)z.keys;
    buf[Q_TWICE] = twice;
    buf[Q_TOTAL] = (int32_t)z.total;
    buf[Q_O_UNITS] = (int32_t)z.off_units;
    buf[Q_O_ITEMS] = (int32_t)z.off_items;
    buf[Q_O_COUNT] = (int32_t)z.off_count;
    buf[Q_O_TILES] = (int32_t)z.off_tiles;
    buf[Q_RITEMS] = (int32_t)z.ritems;
    buf[Q_RPARTS] = (int32_t)z.rparts;
    buf[Q_RJOINS] = (int32_t)z.rsplits;
    buf[Q_RHALF] = half;
    buf[Q_O_RITEMS] = (int32_t)z.off_ritems;
    buf[Q_O_RJOINS] = (int32_t)z.off_rjoins;
    buf[Q_PRE] = (int32_t)z.pre;
    buf[Q_PRETILES] = (int32_t)z.pre_tiles;
    buf[Q_PREREAD] = (int32_t)z.pre_read;
    buf[Q_PREKEYS] = (int32_t)z.pre_keys;
    buf[Q_REQS] = b.n_req;
    buf[Q_O_PRE] = (int32_t)z.off_pre;
    buf[Q_O_PRETILES] = (int32_t)z.off_pretiles;
    buf[Q_O_PREREAD] = (int32_t)z.off_preread;
    buf[Q_O_REQOFF] = (int32_t)z.off_reqoff;
    buf[Q_O_REQCTX] = (int32_t)z.off_reqctx;
    buf[Q_O_REQWS] = (int32_t)z.off_reqws;
    buf[Q_TILEMOST] = most;
    buf[Q_WIDE] = (int32_t)z.wide;
    buf[Q_O_WIDE] = (int32_t)z.off_wide;
    return true;
}

bool kv4_plan_ok(const int32_t *hp) { return hp && hp[Q_MAGIC] == kKv4Magic; }
bool kv4_plan_writes_once(const int32_t *hp) { return !hp[Q_TWICE]; }

namespace {
// byte offsets in the workspace
struct Kv4Work {
    int64_t row_part, q16, pool16, q_scale, kv_scale, wide, total;
};
Kv4Work kv4_work(const int32_t *hp) {
    const int64_t nh = hp[Q_HEADS], d = hp[Q_DIM];
    Kv4Work w;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    take((int64_t)hp[Q_PARTS] * nh * (d + 2) * 4);
    w.row_part = take((int64_t)hp[Q_RPARTS] * nh * kRowsPerItem * (d + 2) * 4);
    const bool pre = hp[Q_PRE] > 0;
    w.q16 = take(pre ? (int64_t)hp[Q_ROWS] * nh * d * 2 : 0);
    w.pool16 = take(2 * nh * hp[Q_PREKEYS] * d * 2);
    w.q_scale = take(pre ? (int64_t)hp[Q_ROWS] * nh * 4 : 0);
    w.kv_scale = take(pre ? (int64_t)hp[Q_REQS] * nh * 2 * 4 : 0);
    w.wide = take(hp[Q_PRE] * nh * 4);
    w.total = at;
    return w;
}
}  // namespace

int64_t kv4_workspace_bytes(const int32_t *hp) { return kv4_work(hp).total; }

namespace {
template <typename T>
cudaError_t append(const void *qkv, const Kv4View &v, const int32_t *hp, const int32_t *dp, cudaStream_t st) {
    const int H = hp[Q_HEADS] * hp[Q_DIM];
    const int per = H / 8, n = hp[Q_UNITS];  // threads of a unit
    return for_dim(hp[Q_DIM], [&](auto d) {
        if (per % kApThreads == 0)
            return launch_pdl(kv4_append_kernel<T, d(), false>, dim3(n, per / kApThreads), dim3(kApThreads), 0, st,
                              (const T *)qkv, dp + hp[Q_O_UNITS], n, v, H);
        return launch_pdl(kv4_append_kernel<T, d(), true>, dim3((unsigned)(((int64_t)n * per + kApThreads - 1) / kApThreads)),
                          dim3(kApThreads), 0, st, (const T *)qkv, dp + hp[Q_O_UNITS], n, v, H);
    });
}

template <typename T>
cudaError_t read(const Kv4View &v, const int32_t *hp, const int32_t *dp, void *out, cudaStream_t st) {
    const int per = hp[Q_TILEMOST];
    return for_dim(hp[Q_DIM], [&](auto d) {
        if (per <= kFewSlots) {
            const int heads = kv4_few_heads(d(), per);
            return launch_pdl(kv4_read_few_kernel<T, d()>, dim3(hp[Q_TILES], (hp[Q_HEADS] + heads - 1) / heads),
                              dim3(kRdThreads), 0, st, v, dp + hp[Q_O_TILES], (T *)out, (int64_t)hp[Q_KEYS], hp[Q_HEADS],
                              per);
        }
        return launch_pdl(kv4_read_kernel<T, d(), false>, dim3(hp[Q_TILES], hp[Q_HEADS]), dim3(kRdThreads), 0, st, v,
                          dp + hp[Q_O_TILES], (T *)out, (int64_t)hp[Q_KEYS], hp[Q_HEADS], (const float *)nullptr);
    });
}
}  // namespace

cudaError_t kv4_append(const void *qkv, void *layer, const int32_t *hp, const int32_t *dp, cudaStream_t st) {
    const Kv4View v = kv4_view(layer, hp[Q_HEADS], hp[Q_DIM], hp[Q_SLOTS]);
    return hp[Q_DTYPE] == 1 ? append<bf16>(qkv, v, hp, dp, st) : append<float>(qkv, v, hp, dp, st);
}

cudaError_t kv4_read(const void *layer, const int32_t *hp, const int32_t *dp, void *out, cudaStream_t st) {
    const Kv4View v = kv4_view(layer, hp[Q_HEADS], hp[Q_DIM], hp[Q_SLOTS]);
    return hp[Q_DTYPE] == 1 ? read<bf16>(v, hp, dp, out, st) : read<float>(v, hp, dp, out, st);
}

namespace {
template <typename T>
cudaError_t launch_rows(const Kv4Attn &a, int d, int items, bool half, int joins, int *launches, cudaStream_t st) {
    const dim3 grid((unsigned)items * a.n_heads), block(kKvThreads);
    return for_dim(d, [&](auto dim) {
        const cudaError_t e = half ? launch_pdl(kv4_rows_mma_kernel<T, dim(), true>, grid, block, 0, st, a)
                                   : launch_pdl(kv4_rows_mma_kernel<T, dim(), false>, grid, block, 0, st, a);
        ++*launches;
        if (e != cudaSuccess || joins == 0) return e;
        ++*launches;
        return launch_pdl(kv4_rows_join_kernel<T, dim()>, dim3(joins, a.n_heads), dim3(32 * kRowsPerItem), 0, st, a);
    });
}
}  // namespace

cudaError_t kv4_attention(const void *qkv, const void *layer, const int32_t *hp, int32_t *dp, void *workspace,
                          void *out, unsigned *err, int *launches, cudaStream_t st) {
    const int nh = hp[Q_HEADS], d = hp[Q_DIM];
    Kv4Attn a;
    a.qkv = qkv;
    a.out = out;
    a.v = kv4_view(layer, nh, d, hp[Q_SLOTS]);
    a.H = nh * d;
    a.n_heads = nh;
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)d);
    a.items = dp + hp[Q_O_ITEMS];
    a.counters = dp + hp[Q_O_COUNT];
    const Kv4Work w = kv4_work(hp);
    uint8_t *ws = (uint8_t *)workspace;
    a.part = (float *)workspace;
    a.row_items = dp + hp[Q_O_RITEMS];
    a.row_joins = dp + hp[Q_O_RJOINS];
    a.row_part = (float *)(ws + w.row_part);
    cudaError_t e = cudaSuccess;
    *launches = 0;
    if (hp[Q_ITEMS] > 0) {
        e = hp[Q_DTYPE] == 1 ? launch_decode<bf16>(a, d, hp[Q_ITEMS], st) : launch_decode<float>(a, d, hp[Q_ITEMS], st);
        ++*launches;
    }
    if (e == cudaSuccess && hp[Q_RITEMS] > 0) {
        auto run = [&](auto type) {
            return launch_rows<decltype(type)>(a, d, hp[Q_RITEMS], hp[Q_RHALF] != 0, hp[Q_RJOINS], launches, st);
        };
        e = hp[Q_DTYPE] == 1 ? run(bf16()) : run(0.f);
    }
    if (e != cudaSuccess || hp[Q_PRE] == 0) return e;
    Kv4Prep pr;
    pr.qkv = (const bf16 *)qkv;
    pr.q16 = (__half *)(ws + w.q16);
    pr.q_scale = (float *)(ws + w.q_scale);
    pr.kv_scale = (float *)(ws + w.kv_scale);
    pr.wide = (int32_t *)(ws + w.wide);
    pr.v = a.v;
    pr.H = a.H, pr.n_heads = nh, pr.d = d, pr.G = kv4_groups(d);
    pr.n_rows = hp[Q_ROWS], pr.n_pre = hp[Q_PRE];
    pr.pre = dp + hp[Q_O_PRE];
    constexpr int kPer = kPrepThreads * kPrepQ;
    const int64_t blocks = (int64_t)pr.n_pre * nh + ((int64_t)pr.n_rows * (a.H / 8) + kPer - 1) / kPer;
    e = launch_pdl(kv4_prep_kernel, dim3((unsigned)blocks), dim3(kPrepThreads), 0, st, pr);
    if (e == cudaSuccess)
        e = launch_pdl(d == 64 ? kv4_read_kernel<__half, 64, true> : kv4_read_kernel<__half, 128, true>,
                       dim3(hp[Q_PREREAD], nh), dim3(kRdThreads), 0, st, a.v, dp + hp[Q_O_PREREAD],
                       (__half *)(ws + w.pool16), (int64_t)hp[Q_PREKEYS], nh, (const float *)pr.kv_scale);
    AttnPlan ap{};
    ap.req_off = dp + hp[Q_O_REQOFF];
    ap.req_ctx = dp + hp[Q_O_REQCTX];
    ap.req_kvoff = dp + hp[Q_O_REQWS];
    ap.pre_tiles = dp + hp[Q_O_PRETILES];
    ap.n_pre_tiles = hp[Q_PRETILES];
    ap.n_rows = hp[Q_ROWS];
    if (e == cudaSuccess)
        e = attention_prefill_f16(pr.q16, hp[Q_ROWS], ws + w.pool16, hp[Q_PREKEYS], (bf16 *)out, ap, a.H, nh, pr.q_scale,
                                  pr.kv_scale, err, st);
    *launches += 3;
    if (e != cudaSuccess) return e;
    a.wide = pr.wide, a.n_wide = hp[Q_PRE] * nh;
    a.wide_items = dp + hp[Q_O_WIDE], a.n_wide_items = hp[Q_WIDE];
    int sms = 0, dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const dim3 grid((unsigned)std::min<int64_t>((int64_t)a.n_wide_items * nh, 3LL * sms));
    ++*launches;
    return launch_pdl(d == 64 ? kv4_rows_wide_kernel<64> : kv4_rows_wide_kernel<128>, grid, dim3(kKvThreads), 0, st, a);
}

}  // namespace orca
