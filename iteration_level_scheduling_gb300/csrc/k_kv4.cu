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

// ---------------------------------------------------------------------------
// write: k and v of every row, one thread per 8 components
// ---------------------------------------------------------------------------
constexpr int kApThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kApThreads) kv4_append_kernel(const T *qkv, const int32_t *row_slot, Kv4View v, int H,
                                                                int d, int G, int gt) {
    pdl_trigger();
    pdl_wait();
    const int r = blockIdx.x;
    const int64_t slot = row_slot[r];
    const int u = blockIdx.y * kApThreads + threadIdx.x;  // 8-component unit of k, then v
    const bool on = u * 8 < 2 * H;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (on) {
        const T *src = qkv + (size_t)r * 3 * H + H + (size_t)u * 8;
#pragma unroll
        for (int i = 0; i < 8; i += Elem<T>::kPer16) load16_stream(src + i, x + i);
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) lo = min_nan(lo, x[i]), hi = max_nan(hi, x[i]);
    // the group's 2 or 4 threads (gt) are neighbours; units of k and v and of heads never share a group
    for (int o = 1; o < gt; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (!on) return;
    uint32_t sb = bf_bits(__fdiv_rn(__fsub_rn(hi, lo), 15.f)), mb = bf_bits(lo);
    const bool fine = (sb & 0x7f80u) != 0x7f80u && (mb & 0x7f80u) != 0x7f80u;
    if (!fine) sb = mb = 0x7fc0u;
    const float s = bf_lo(sb), m = bf_lo(mb);
    uint32_t w = 0;
    if (fine && s > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= kv4_code(x[i], m, s) << (4 * i);
    }
    const int c = u * 8, which = c >= H, cc = c - which * H, h = cc / d, dd = cc - h * d;
    const uint32_t par = sb | (mb << 16);
    const bool lead = (u % gt) == 0;
    const int g = dd / (8 * gt);
    if (!which) {
        *reinterpret_cast<uint32_t *>(v.kc + ((int64_t)h * v.S + slot) * (d / 2) + dd / 2) = w;
        if (lead) v.kp[((int64_t)h * v.S + slot) * G + g] = par;
    } else {
        const int64_t pair = (int64_t)h * (v.S / 2) + (slot >> 1);
        uint16_t *dst = reinterpret_cast<uint16_t *>(v.vc + (pair * (d / 4) + dd / 4) * 4) + (slot & 1);
        dst[0] = (uint16_t)w;
        dst[2] = (uint16_t)(w >> 16);
        if (lead) v.vp[(pair * G + g) * 2 + (slot & 1)] = par;
    }
}

// ---------------------------------------------------------------------------
// read back: tiles of up to 64 slots of one range, one head's K and V per CTA
// ---------------------------------------------------------------------------
constexpr int kRdThreads = 128;

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

// scale: the inverses of the powers of two that the values are to be multiplied by ([request][head][K|V]), or null
template <typename T>
__global__ void __launch_bounds__(kRdThreads) kv4_read_kernel(Kv4View v, const int32_t *tiles, T *out, int64_t out_slots,
                                                              int n_heads, int d, int G, const float *scale) {
    pdl_trigger();
    pdl_wait();
    const int4 tl = reinterpret_cast<const int4 *>(tiles)[blockIdx.x];  // first slot, slots, first output index, request
    const int h = blockIdx.y, gs = d / G, upr = d / 8;                  // 8-component units per row
    const int64_t s0 = tl.x, s1 = s0 + tl.y;
    float kf = 1.f, vf = 1.f;
    if (scale) {
        const float *f = scale + 2 * ((size_t)tl.w * n_heads + h);
        kf = 1.f / f[0], vf = 1.f / f[1];
    }
    T *ko = out + ((int64_t)h * out_slots + tl.z) * d, *vo = ko + (int64_t)n_heads * out_slots * d;
    for (int i = threadIdx.x; i < tl.y * upr; i += kRdThreads) {
        const int j = i / upr, u = i - j * upr;
        const int64_t row = (int64_t)h * v.S + s0 + j;
        const uint32_t w = *reinterpret_cast<const uint32_t *>(v.kc + row * (d / 2) + u * 4);
        const uint32_t p = v.kp[row * G + u * 8 / gs];
        float s = bf_lo(p) * kf, m = bf_hi(p) * kf;
        if (scale) {
            // a NaN among the values is moved to the key: a weight of 0 times it would reach rows that do not see
            // the key, while a masked score is dropped whatever it is
            const int64_t slot = s0 + j;
            const uint32_t pv = v.vp[(((int64_t)h * (v.S / 2) + (slot >> 1)) * G + u * 8 / gs) * 2 + (slot & 1)];
            if (bf_lo(pv) != bf_lo(pv)) m = bf_lo(pv);
        }
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = fmaf(s, (float)((w >> (4 * k)) & 15u), m);
        store8(ko + (int64_t)j * d + u * 8, x);
    }
    const int64_t p0 = s0 >> 1, np = ((s1 + 1) >> 1) - p0;
    for (int i = threadIdx.x; i < (int)np * upr; i += kRdThreads) {
        const int j = i / upr, u = i - j * upr;
        const int64_t pair = (int64_t)h * (v.S / 2) + p0 + j;
        const uint2 w = *reinterpret_cast<const uint2 *>(v.vc + (pair * (d / 4) + u * 2) * 4);
        const uint2 p = *reinterpret_cast<const uint2 *>(v.vp + (pair * G + u * 8 / gs) * 2);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int64_t slot = 2 * (p0 + j) + o;
            if (slot < s0 || slot >= s1) continue;
            const uint32_t a = w.x >> (16 * o), b = w.y >> (16 * o), pp = o ? p.y : p.x;
            float s = bf_lo(pp) * vf, m = bf_hi(pp) * vf;
            if (scale && s != s) s = m = 0.f;
            float x[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[k] = fmaf(s, (float)((a >> (4 * k)) & 15u), m);
                x[4 + k] = fmaf(s, (float)((b >> (4 * k)) & 15u), m);
            }
            store8(vo + (slot - s0) * d + u * 8, x);
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
// magnitude to [2^14, 2^15) (values 2^-28 of it and below lose bits).

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
    Kv4View v;
    int H, n_heads, d, G, n_rows, n_pre;
    const int32_t *pre;  // 4 words per prompt: request, first slot, slots, 0
};
constexpr int kPrepThreads = 256;

// Blocks 0 .. n_pre * n_heads - 1: the scales of K and V of one prompt and head, from the parameters (a component lies
// between m and m + 15 s).  The others: a warp scales and rounds q of one row and head.
__global__ void __launch_bounds__(kPrepThreads) kv4_prep_kernel(const Kv4Prep a) {
    __shared__ float red[2][kPrepThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = a.n_pre * a.n_heads;
    if ((int)blockIdx.x < first) {
        const int i = blockIdx.x / a.n_heads, h = blockIdx.x - i * a.n_heads;
        const int4 pr = reinterpret_cast<const int4 *>(a.pre)[i];
        const int64_t s0 = pr.y, s1 = s0 + pr.z;
        float km = 0.f, vm = 0.f;
        // (fmaxf drops NaN: a group that reads back as NaN does so whatever the scale)
        auto size = [](uint32_t p) { return fmaxf(fabsf(bf_hi(p)), fabsf(fmaf(15.f, bf_lo(p), bf_hi(p)))); };
        const uint32_t *kp = a.v.kp + ((int64_t)h * a.v.S + s0) * a.G;
        const int64_t nk = (s1 - s0) * a.G;
#pragma unroll 4
        for (int64_t j = threadIdx.x; j < nk; j += kPrepThreads) km = fmaxf(km, size(kp[j]));
        const int64_t p0 = s0 >> 1, np = ((s1 + 1) >> 1) - p0;
        const uint2 *vp = reinterpret_cast<const uint2 *>(a.v.vp) + ((int64_t)h * (a.v.S / 2) + p0) * a.G;
#pragma unroll 4
        for (int64_t j = threadIdx.x; j < np * a.G; j += kPrepThreads) {
            const uint2 p = vp[j];
            const int64_t slot = 2 * (p0 + j / a.G);
            if (slot >= s0) vm = fmaxf(vm, size(p.x));
            if (slot + 1 < s1) vm = fmaxf(vm, size(p.y));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
            vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
        }
        if (lane == 0) red[0][warp] = km, red[1][warp] = vm;
        __syncthreads();
        if (threadIdx.x < 2) {
            float m = 0.f;
            for (int w = 0; w < kPrepThreads / 32; ++w) m = fmaxf(m, red[threadIdx.x][w]);
            a.kv_scale[2 * ((size_t)pr.x * a.n_heads + h) + threadIdx.x] = kv4_inverse_scale(m);
        }
        return;
    }
    const int64_t unit = ((int64_t)blockIdx.x - first) * (kPrepThreads / 32) + warp;  // (row, head)
    if (unit >= (int64_t)a.n_rows * a.n_heads) return;
    const int64_t r = unit / a.n_heads;
    const int h = (int)(unit - r * a.n_heads);
    const bool on = lane * 8 < a.d;  // 8 components per lane
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (on) load16_stream(a.qkv + r * 3 * a.H + h * a.d + lane * 8, x);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(x[e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float inv = kv4_inverse_scale(m), f = 1.f / inv;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= f;
    if (on) store8(a.q16 + r * a.H + h * a.d + lane * 8, x);
    if (lane == 0) a.q_scale[r * a.n_heads + h] = inv;
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
    const int32_t *items;  // 8 words: first slot, keys, row, chunks of the row, this chunk, the row's first partial, its counter
    int *counters;         // [row counter][head], zero between launches
    float *part;           // [partial][head][D + 2]
};

template <int D>
struct Kv4Merge {
    float m[kKvWarps], l[kKvWarps], o[kKvWarps][D];
    int last;
};

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
    float Mt = kLow, Lt = 0.f, Ot = 0.f;
    for (int j = 0; j < nch; ++j) {
        const float *pj = a.part + ((size_t)(r1.y + j) * a.n_heads + h) * (D + 2);
        const float pm = __ldcg(pj + D), pl = __ldcg(pj + D + 1), po = tid < D ? __ldcg(pj + tid) : 0.f;
        const float mn = fmaxf(Mt, pm), co = exp2f(Mt - mn), cn = exp2f(pm - mn);
        Lt = Lt * co + pl * cn;
        Ot = Ot * co + po * cn;
        Mt = mn;
    }
    if (tid < D) dst[tid] = Elem<T>::from_f(Ot / Lt);
}

// Any type and head_dim, fp32 arithmetic.  A warp takes 32 slots at a time:
// for the scores a lane owns a key and walks its components against q in
// shared memory; for the values a lane owns four components and walks the
// keys, two per word.
template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads) kv4_decode_kernel(const Kv4Attn a) {
    constexpr int G = D / 32 > 0 ? D / 32 : 1, GS = D / G;
    constexpr int LP = D / 4, PP = 32 / LP;  // lanes per pair of keys, pairs per step
    __shared__ Kv4Merge<D> sm;
    __shared__ float q[D];
    __shared__ float qs[G];
    pdl_trigger();
    pdl_wait();
    const int4 r0 = reinterpret_cast<const int4 *>(a.items)[2 * blockIdx.x],
               r1 = reinterpret_cast<const int4 *>(a.items)[2 * blockIdx.x + 1];
    const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < D)
        q[threadIdx.x] = Elem<T>::to_f(((const T *)a.qkv)[(size_t)r0.z * 3 * a.H + h * D + threadIdx.x]) * a.scale_log2;
    __syncthreads();
    if (threadIdx.x < G) {
        float s = 0.f;
        for (int i = 0; i < GS; ++i) s += q[threadIdx.x * GS + i];
        qs[threadIdx.x] = s;
    }
    __syncthreads();
    const int64_t s0 = r0.x, s1 = s0 + r0.y;
    const int sub = lane % LP, grp = lane / LP;
    float m = kLow, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t b = (s0 & ~int64_t(1)) + 32 * warp; b < s1; b += 32 * kKvWarps) {
        const int64_t slot = b + lane;
        const bool valid = slot >= s0 && slot < s1;
        float sc = kLow;
        if (valid) {
            const int64_t row = (int64_t)h * a.v.S + slot;
            sc = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t p = a.v.kp[row * G + g];
                float acc = 0.f;
#pragma unroll
                for (int w = 0; w < GS / 8; ++w) {
                    const uint32_t x =
                        *reinterpret_cast<const uint32_t *>(a.v.kc + row * (D / 2) + g * (GS / 2) + w * 4);
#pragma unroll
                    for (int k = 0; k < 8; ++k) acc = fmaf(q[g * GS + w * 8 + k], (float)((x >> (4 * k)) & 15u), acc);
                }
                sc += bf_lo(p) * acc + bf_hi(p) * qs[g];
            }
        }
        float mx = sc;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        mx = fmaxf(mx, m);
        const float corr = exp2f(m - mx);
        m = mx;
        const float p = valid ? exp2f(sc - m) : 0.f;
        l = l * corr + p;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] *= corr;
#pragma unroll 4
        for (int j = 0; j < 16; j += PP) {
            const int pr = j + grp;  // this lane's pair
            const float pe = __shfl_sync(0xffffffffu, p, 2 * pr), po = __shfl_sync(0xffffffffu, p, 2 * pr + 1);
            const int64_t se = b + 2 * pr;
            const bool ve = se >= s0 && se < s1, vo = se + 1 >= s0 && se + 1 < s1;
            if (!ve && !vo) continue;
            const int64_t pair = (int64_t)h * (a.v.S / 2) + (se >> 1);
            const uint32_t x = *reinterpret_cast<const uint32_t *>(a.v.vc + (pair * (D / 4) + sub) * 4);
            const uint2 pp = *reinterpret_cast<const uint2 *>(a.v.vp + (pair * G + sub * 4 / GS) * 2);
            // (an unused slot's parameters may be anything)
            const float ws = ve ? pe * bf_lo(pp.x) : 0.f, wm = ve ? pe * bf_hi(pp.x) : 0.f;
            const float xs = vo ? po * bf_lo(pp.y) : 0.f, xm = vo ? po * bf_hi(pp.y) : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] += fmaf(ws, (float)((x >> (4 * k)) & 15u), wm) + fmaf(xs, (float)((x >> (16 + 4 * k)) & 15u), xm);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
    for (int off = LP; off < 32; off <<= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] += __shfl_xor_sync(0xffffffffu, o[k], off);
    if (grp == 0)
#pragma unroll
        for (int k = 0; k < 4; ++k) sm.o[warp][4 * sub + k] = o[k];
    if (lane == 0) sm.m[warp] = m, sm.l[warp] = l;
    kv4_finish<T, D>(a, sm, r0, r1, h);
}

// bf16, head_dim 32 and more: both products on mma.sync m16n8k16 with the
// codes as the A operand, unpacked in registers straight from 16-byte loads.
//   scores   rows = 16 keys.  A lane's loads of one key are components of one
//            group; q enters column g of B only where the component's group is
//            g, so the columns of S gather sum q c group by group and s, m
//            apply afterwards.  A = 128 + c (the bits of c in the mantissa of
//            bf16's 128); -128 sum q is the accumulator's start.
//   values   rows = 16 components, k = 16 keys.  A = c - 8, exact; column g of
//            B is p s_g rounded to bf16, column 4 + g what the rounding left,
//            so the weights keep 16 bits; sum p (m + 8 s) is added in fp32.
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

// One block of 16 slots as a lane (g, t) = (lane / 4, lane % 4) of a warp holds it.
template <int D>
struct Kv4Block {
    static constexpr int W = D / 32;  // words per lane and row, and groups
    uint32_t k[2][W];                 // keys g, g + 8: components 8 W t ..
    uint32_t v[2][W];                 // pairs t, t + 4: components 4 W g ..
    uint32_t kp[2][2];                // keys g, g + 8: groups 2t, 2t + 1
    uint32_t vp[2][2];                // pairs t, t + 4: group g % 4, even and odd slot
    __device__ __forceinline__ void load(const Kv4View &v4, int h, int64_t b, int g, int t) {
        const int64_t row = (int64_t)h * v4.S + b, pair = row >> 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            load_words<W>(v4.kc + (row + g + 8 * i) * (D / 2) + t * (4 * W), k[i]);
            load_words<W>(v4.vc + (pair + t + 4 * i) * D + g * (4 * W), v[i]);
            const uint32_t *p = v4.kp + (row + g + 8 * i) * W;
            if constexpr (W == 4) load_words<2>(p + 2 * (t & 1), kp[i]);
            else if constexpr (W == 2) load_words<2>(p, kp[i]);
            else kp[i][0] = __ldcs(p), kp[i][1] = 0u;
            load_words<2>(v4.vp + ((pair + t + 4 * i) * W + (g & (W - 1))) * 2, vp[i]);
        }
    }
};

template <int D>
__global__ void __launch_bounds__(kKvThreads, 4) kv4_decode_mma_kernel(const Kv4Attn a) {
    constexpr int W = D / 32;
    constexpr unsigned kAll = 0xffffffffu;
    __shared__ Kv4Merge<D> sm;
    pdl_trigger();
    pdl_wait();
    const int4 r0 = reinterpret_cast<const int4 *>(a.items)[2 * blockIdx.x],
               r1 = reinterpret_cast<const int4 *>(a.items)[2 * blockIdx.x + 1];
    const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t s0 = r0.x, s1 = s0 + r0.y;
    int64_t b = (s0 & ~int64_t(15)) + 16 * warp;  // (S is a multiple of 16: a block never leaves the layer)
    Kv4Block<D> nx;
    if (b < s1) nx.load(a.v, h, b, g, t);

    // q: word w of a lane covers components 8 (W t + w) ..; pairs (n, n + 4)
    uint32_t qf[W][4];
    float qsum[2];  // sum of q over groups 2t and 2t + 1
    {
        const bf16 *q = (const bf16 *)a.qkv + (size_t)r0.z * 3 * a.H + h * D + 8 * W * t;
        const bool mine = g == (t * W) / 4;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            float x[8];
            load16(q + 8 * w, x);
#pragma unroll
            for (int n = 0; n < 8; ++n) sum += x[n];
#pragma unroll
            for (int n = 0; n < 4; ++n) qf[w][n] = mine ? pack2(x[n], x[n + 4]) : 0u;
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
        }
    }
    float m = kLow, l = 0.f, zero = 0.f, o[2 * W][4];
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    while (b < s1) {
        const Kv4Block<D> x = nx;
        const int64_t here = b;
        b += 16 * kKvWarps;
        if (b < s1) nx.load(a.v, h, b, g, t);
        // scores of keys g and g + 8
        float c[4] = {-128.f * qsum[0], -128.f * qsum[1], -128.f * qsum[0], -128.f * qsum[1]};
#pragma unroll
        for (int w = 0; w < W; ++w) {
            kv4_mma(c, code_pair<0>(x.k[0][w]), code_pair<0>(x.k[1][w]), code_pair<1>(x.k[0][w]),
                    code_pair<1>(x.k[1][w]), qf[w][0], qf[w][1]);
            kv4_mma(c, code_pair<2>(x.k[0][w]), code_pair<2>(x.k[1][w]), code_pair<3>(x.k[0][w]),
                    code_pair<3>(x.k[1][w]), qf[w][2], qf[w][3]);
        }
        float sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // (lanes whose columns hold no group have c = qsum = 0 but may have read another's parameters)
            float s = 0.f;
            if (2 * t < W)
                s = bf_lo(x.kp[i][0]) * c[2 * i] + bf_hi(x.kp[i][0]) * qsum[0] + bf_lo(x.kp[i][1]) * c[2 * i + 1] +
                    bf_hi(x.kp[i][1]) * qsum[1];
            s += __shfl_xor_sync(kAll, s, 1);
            s += __shfl_xor_sync(kAll, s, 2);
            sc[i] = s * a.scale_log2;
        }
        const bool whole = here >= s0 && here + 16 <= s1;  // warp-uniform
        bool v_lo = true, v_hi = true;
        if (!whole) {
            v_lo = here + g >= s0 && here + g < s1;
            v_hi = here + g + 8 >= s0 && here + g + 8 < s1;
            if (!v_lo) sc[0] = kLow;
            if (!v_hi) sc[1] = kLow;
        }
        float mx = fmaxf(sc[0], sc[1]);
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
        if (mx > m) {  // warp-uniform
            const float corr = exp2f(m - mx);
            m = mx;
            l *= corr, zero *= corr;
#pragma unroll
            for (int i = 0; i < 2 * W; ++i) o[i][0] *= corr, o[i][1] *= corr, o[i][2] *= corr, o[i][3] *= corr;
        }
        const float p_lo = v_lo ? exp2f(sc[0] - m) : 0.f, p_hi = v_hi ? exp2f(sc[1] - m) : 0.f;
        l += p_lo + p_hi;
        // weights of keys 2t, 2t + 1, 2t + 8, 2t + 9 in group g % 4
        uint32_t bw[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float pe = __shfl_sync(kAll, i ? p_hi : p_lo, 8 * t), po = __shfl_sync(kAll, i ? p_hi : p_lo, 8 * t + 4);
            float se = bf_lo(x.vp[i][0]), me = bf_hi(x.vp[i][0]), so = bf_lo(x.vp[i][1]), mo = bf_hi(x.vp[i][1]);
            if (!whole) {  // an unused slot's parameters may be anything
                const int64_t slot = here + 8 * i + 2 * t;
                if (slot < s0 || slot >= s1) se = me = 0.f;
                if (slot + 1 < s0 || slot + 1 >= s1) so = mo = 0.f;
            }
            const float we = pe * se, wo = po * so;
            zero += pe * fmaf(8.f, se, me) + po * fmaf(8.f, so, mo);
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
    }
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

template <typename T>
cudaError_t launch_decode(const Kv4Attn &a, int d, int n_items, cudaStream_t st) {
    const dim3 grid(n_items, a.n_heads), block(kKvThreads);
    if constexpr (std::is_same<T, bf16>::value) {
        if (d == 32) return launch_pdl(kv4_decode_mma_kernel<32>, grid, block, 0, st, a);
        if (d == 64) return launch_pdl(kv4_decode_mma_kernel<64>, grid, block, 0, st, a);
        if (d == 128) return launch_pdl(kv4_decode_mma_kernel<128>, grid, block, 0, st, a);
    }
    switch (d) {
        case 16: return launch_pdl(kv4_decode_kernel<T, 16>, grid, block, 0, st, a);
        case 32: return launch_pdl(kv4_decode_kernel<T, 32>, grid, block, 0, st, a);
        case 64: return launch_pdl(kv4_decode_kernel<T, 64>, grid, block, 0, st, a);
        case 128: return launch_pdl(kv4_decode_kernel<T, 128>, grid, block, 0, st, a);
        default: return cudaErrorInvalidValue;
    }
}

// ---------------------------------------------------------------------------
// plans
// ---------------------------------------------------------------------------
constexpr int32_t kKv4Magic = 0x4B563450;
constexpr int kKv4Hdr = 32;
constexpr int kReadTile = 64;  // slots per read-back tile
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
    Q_O_ROWSLOT,  // word offsets of the tables
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
    Q_O_REQWS,  // a prompt's first slot in the workspace's pool
};
// Requests of at least this many rows run on the prefill kernel (bf16, head_dim 64 or 128).
constexpr int kPromptRows = 16;

int64_t up4(int64_t w) { return (w + 3) & ~int64_t(3); }

struct Kv4Sizes {
    int64_t rows = 0, items = 0, splits = 0, parts = 0, tiles = 0, keys = 0;
    int64_t pre = 0, pre_tiles = 0, pre_read = 0, pre_keys = 0;
    int chunk = 0;
    int64_t off_rowslot, off_items, off_count, off_tiles, off_pre, off_pretiles, off_preread, off_reqoff, off_reqctx,
        off_reqws, total;
};

// Keys per work item: the largest chunk (a power of two, 64 .. 2048 keys) that
// still gives every SM several blocks of four warps; short chunks cost a join,
// long ones leave SMs idle.
bool is_prompt(const Kv4Batch &b, int i) {
    return b.dtype == 1 && (b.head_dim == 64 || b.head_dim == 128) && b.n_input[i] >= kPromptRows;
}

int kv4_chunk(const Kv4Batch &b, int num_sms) {
    int chunk = 2048;
    while (chunk > 64) {
        int64_t items = 0;
        for (int i = 0; i < b.n_req && items * b.n_heads < 6LL * num_sms; ++i)
            if (!is_prompt(b, i))
                items += (int64_t)b.n_input[i] * ((b.ctx_len[i] + (int64_t)b.n_input[i] + chunk - 1) / chunk);
        if (items * b.n_heads >= 6LL * num_sms) break;
        chunk /= 2;
    }
    return chunk;
}

bool kv4_sizes(const Kv4Batch &b, int num_sms, Kv4Sizes *z) {
    int64_t rows = 0;
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t n = b.n_input[i], c = b.ctx_len[i], o = b.kv_offset[i];
        if (n < 1 || c < 0 || o < 0 || o > b.kv_slots || o + c + n > b.kv_slots) return false;
        rows += n;
        if (rows > INT32_MAX / 8) return false;
    }
    z->chunk = kv4_chunk(b, num_sms);
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t n = b.n_input[i], c = b.ctx_len[i];
        z->rows += n;
        z->keys += c + n;
        z->tiles += (c + n + kReadTile - 1) / kReadTile;
        if (is_prompt(b, i)) {
            z->pre++;
            z->pre_tiles += (n + kPrefillRowsPerTile - 1) / kPrefillRowsPerTile;
            z->pre_read += (c + n + kReadTile - 1) / kReadTile;
            z->pre_keys += c + n;
            continue;
        }
        for (int64_t j = 0; j < n; ++j) {
            const int64_t nch = (c + j + 1 + z->chunk - 1) / z->chunk;
            z->items += nch;
            if (nch > 1) z->splits++, z->parts += nch;
        }
    }
    int64_t w = kKv4Hdr;
    z->off_rowslot = w, w = up4(w + z->rows);
    z->off_items = w, w = up4(w + 8 * z->items);
    z->off_count = w, w = up4(w + z->splits * b.n_heads);
    z->off_tiles = w, w = up4(w + 4 * z->tiles);
    z->off_pre = w, w = up4(w + 4 * z->pre);
    z->off_pretiles = w, w = up4(w + 2 * z->pre_tiles);
    z->off_preread = w, w = up4(w + 4 * z->pre_read);
    z->off_reqoff = w, w = up4(w + b.n_req + 1);
    z->off_reqctx = w, w = up4(w + b.n_req);
    z->off_reqws = w, w = up4(w + b.n_req);
    z->total = w;
    // 32-bit table entries and grid sizes
    return w <= INT32_MAX && z->keys <= INT32_MAX && z->pre_tiles * b.n_heads <= INT32_MAX &&
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

bool kv4_plan_build(const Kv4Batch &b, int num_sms, int32_t *buf, int64_t cap) {
    Kv4Sizes z;
    if (!kv4_sizes(b, num_sms, &z) || cap < z.total) return false;
    std::memset(buf, 0, sizeof(int32_t) * (size_t)z.total);  // (the device copy's counters start at zero)
    int32_t *slot = buf + z.off_rowslot, *it = buf + z.off_items, *tl = buf + z.off_tiles;
    int32_t *pre = buf + z.off_pre, *pt = buf + z.off_pretiles, *pd = buf + z.off_preread;
    int32_t *req_off = buf + z.off_reqoff, *req_ctx = buf + z.off_reqctx, *req_ws = buf + z.off_reqws;
    int64_t row = 0, split = 0, part = 0, key = 0, ws = 0;
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t n = b.n_input[i], c = b.ctx_len[i], o = b.kv_offset[i];
        const bool prompt = is_prompt(b, i);
        req_off[i] = (int32_t)row;
        req_ctx[i] = (int32_t)c;
        req_ws[i] = (int32_t)ws;
        for (int64_t j = 0; j < n; ++j, ++row) {
            slot[row] = (int32_t)(o + c + j);
            if (prompt) continue;
            const int64_t keys = c + j + 1, nch = (keys + z.chunk - 1) / z.chunk;
            for (int64_t k = 0; k < nch; ++k, it += 8) {
                it[0] = (int32_t)(o + k * z.chunk);
                it[1] = (int32_t)std::min<int64_t>(z.chunk, keys - k * z.chunk);
                it[2] = (int32_t)row;
                it[3] = (int32_t)nch;
                it[4] = (int32_t)k;
                it[5] = (int32_t)part;
                it[6] = (int32_t)split;
            }
            if (nch > 1) ++split, part += nch;
        }
        for (int64_t t = 0; t < c + n; t += kReadTile, tl += 4) {
            tl[0] = (int32_t)(o + t);
            tl[1] = (int32_t)std::min<int64_t>(kReadTile, c + n - t);
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
            pre[0] = i, pre[1] = (int32_t)o, pre[2] = (int32_t)(c + n);
            pre += 4;
            for (int64_t q = 0; q < n; q += kPrefillRowsPerTile, pt += 2) pt[0] = i, pt[1] = (int32_t)q;
            ws += c + n;
        }
    }
    req_off[b.n_req] = (int32_t)row;
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
    buf[Q_ITEMS] = (int32_t)z.items;
    buf[Q_SPLITS] = (int32_t)z.splits;
    buf[Q_PARTS] = (int32_t)z.parts;
    buf[Q_TILES] = (int32_t)z.tiles;
    buf[Q_KEYS] = (int32_t)z.keys;
    buf[Q_TWICE] = twice;
    buf[Q_TOTAL] = (int32_t)z.total;
    buf[Q_O_ROWSLOT] = (int32_t)z.off_rowslot;
    buf[Q_O_ITEMS] = (int32_t)z.off_items;
    buf[Q_O_COUNT] = (int32_t)z.off_count;
    buf[Q_O_TILES] = (int32_t)z.off_tiles;
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
    return true;
}

bool kv4_plan_ok(const int32_t *hp) { return hp && hp[Q_MAGIC] == kKv4Magic; }
bool kv4_plan_writes_once(const int32_t *hp) { return !hp[Q_TWICE]; }

namespace {
// byte offsets in the workspace
struct Kv4Work {
    int64_t q16, pool16, q_scale, kv_scale, total;
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
    const bool pre = hp[Q_PRE] > 0;
    w.q16 = take(pre ? (int64_t)hp[Q_ROWS] * nh * d * 2 : 0);
    w.pool16 = take(2 * nh * hp[Q_PREKEYS] * d * 2);
    w.q_scale = take(pre ? (int64_t)hp[Q_ROWS] * nh * 4 : 0);
    w.kv_scale = take(pre ? (int64_t)hp[Q_REQS] * nh * 2 * 4 : 0);
    w.total = at;
    return w;
}
}  // namespace

int64_t kv4_workspace_bytes(const int32_t *hp) { return kv4_work(hp).total; }

cudaError_t kv4_append(const void *qkv, void *layer, const int32_t *hp, const int32_t *dp, cudaStream_t st) {
    const int nh = hp[Q_HEADS], d = hp[Q_DIM], H = nh * d, G = kv4_groups(d), gt = d / G / 8;
    const Kv4View v = kv4_view(layer, nh, d, hp[Q_SLOTS]);
    const dim3 grid(hp[Q_ROWS], (2 * H / 8 + kApThreads - 1) / kApThreads);
    if (hp[Q_DTYPE] == 1)
        return launch_pdl(kv4_append_kernel<bf16>, grid, dim3(kApThreads), 0, st, (const bf16 *)qkv,
                          dp + hp[Q_O_ROWSLOT], v, H, d, G, gt);
    return launch_pdl(kv4_append_kernel<float>, grid, dim3(kApThreads), 0, st, (const float *)qkv, dp + hp[Q_O_ROWSLOT],
                      v, H, d, G, gt);
}

cudaError_t kv4_read(const void *layer, const int32_t *hp, const int32_t *dp, void *out, cudaStream_t st) {
    const int nh = hp[Q_HEADS], d = hp[Q_DIM], G = kv4_groups(d);
    const Kv4View v = kv4_view(layer, nh, d, hp[Q_SLOTS]);
    const dim3 grid(hp[Q_TILES], nh);
    if (hp[Q_DTYPE] == 1)
        return launch_pdl(kv4_read_kernel<bf16>, grid, dim3(kRdThreads), 0, st, v, dp + hp[Q_O_TILES], (bf16 *)out,
                          (int64_t)hp[Q_KEYS], nh, d, G, (const float *)nullptr);
    return launch_pdl(kv4_read_kernel<float>, grid, dim3(kRdThreads), 0, st, v, dp + hp[Q_O_TILES], (float *)out,
                      (int64_t)hp[Q_KEYS], nh, d, G, (const float *)nullptr);
}

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
    a.part = (float *)workspace;
    cudaError_t e = cudaSuccess;
    *launches = 0;
    if (hp[Q_ITEMS] > 0) {
        e = hp[Q_DTYPE] == 1 ? launch_decode<bf16>(a, d, hp[Q_ITEMS], st) : launch_decode<float>(a, d, hp[Q_ITEMS], st);
        ++*launches;
    }
    if (e != cudaSuccess || hp[Q_PRE] == 0) return e;
    const Kv4Work w = kv4_work(hp);
    uint8_t *ws = (uint8_t *)workspace;
    Kv4Prep pr;
    pr.qkv = (const bf16 *)qkv;
    pr.q16 = (__half *)(ws + w.q16);
    pr.q_scale = (float *)(ws + w.q_scale);
    pr.kv_scale = (float *)(ws + w.kv_scale);
    pr.v = a.v;
    pr.H = a.H, pr.n_heads = nh, pr.d = d, pr.G = kv4_groups(d);
    pr.n_rows = hp[Q_ROWS], pr.n_pre = hp[Q_PRE];
    pr.pre = dp + hp[Q_O_PRE];
    constexpr int kWarps = kPrepThreads / 32;
    const int64_t blocks = (int64_t)pr.n_pre * nh + ((int64_t)pr.n_rows * nh + kWarps - 1) / kWarps;
    e = launch_pdl(kv4_prep_kernel, dim3((unsigned)blocks), dim3(kPrepThreads), 0, st, pr);
    if (e == cudaSuccess)
        e = launch_pdl(kv4_read_kernel<__half>, dim3(hp[Q_PREREAD], nh), dim3(kRdThreads), 0, st, a.v,
                       dp + hp[Q_O_PREREAD], (__half *)(ws + w.pool16), (int64_t)hp[Q_PREKEYS], nh, d, pr.G,
                       (const float *)pr.kv_scale);
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
    return e;
}

}  // namespace orca
