// Token sampling: temperature, top-k, top-p and min-p, then the inverse of the
// cumulative distribution at a given uniform number.
//
// For a row of logits l with largest value m, w_i = exp((l_i - m) / T).  The
// kept tokens are, by (w descending, id ascending): the first k; of those the
// shortest prefix whose mass reaches p times theirs; of those the ones with
// w_i >= min_p.  The token is the first id, in the order of the ids, whose
// cumulative kept weight exceeds u times the total.
//
// Every weight is rounded once to fixed point with 42 fraction bits and all
// sums are 64-bit integers: exact, whatever their order, so the result does
// not depend on how the work is spread, and 2^20 weights of at most 1 fit.
// (In fp32 the running sums of 50257 probabilities are off by more than many
// of the tokens weigh; the token drawn would then often be a neighbour.)
//
// A row is read from memory once and kept in shared memory; a cluster of CTAs
// shares it when there are few rows or one SM cannot hold it, meeting in
// distributed shared memory.  Which tokens a filter keeps is decided from a
// histogram (counts or exact masses) of 2048 bins, linear in the logit over the
// 43 octaves below m that carry weight: the bins down to the one in which the
// count or the mass is reached hold every token that can be kept.  Up to 1024
// of them are gathered, sorted and settled by one CTA; more are settled by
// selecting the last kept logit and passing over the row in the order of the
// ids.
//
// Bound by barriers and latency, then by issue: 192 rows of 50257 with mixed
// parameters take 61 to 64 us (38.6 MB: 5.8 us of reading), the schedulers issuing in
// 44 % of their active cycles, barriers the first stall; a weight is about 95
// warp instructions per 32 logits with its comparison and sum, two thirds of
// them integer.  One row at T 0.8, top-k 50, top-p 0.95 takes 11.0 us on four
// CTAs: a quarter to load, a quarter to gather, the rest in barriers and in sums
// over the block (12.1 us, and the batch 73, with every logit in the histogram).
// With weights by fp64 exp, masses by a radix selection over the row in global
// memory, these were 2453 and 142 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cstddef>

#include "common.cuh"
#include "kernels.cuh"

namespace orca {

namespace {

namespace cg = cooperative_groups;

constexpr int kSpThreads = 512, kSpWarps = kSpThreads / 32;
constexpr int kFrac = 42;     // fraction bits of a weight
constexpr int kBins = 2048;   // histogram bins (four per thread)
constexpr int kList = 1024;   // tokens settled by sorting (two per thread)
constexpr int kMaxCluster = 8;
static_assert(kSpWarps / 2 + 1 >= kMaxCluster, "two warps fetch a CTA's list");

using u64 = unsigned long long;
static_assert(kBins == 4 * kSpThreads && kList == 2 * kSpThreads, "bins and list per thread");

struct SampleArgs {
    const void *logits;
    int64_t ld;
    int V, per;     // ids of one CTA (a multiple of four)
    int n_rows;
    bool by_work;  // rows are taken by the work that their parameters mean, the most first
    const float *temperature, *top_p, *min_p, *uniform;
    const int32_t *top_k;
    int32_t *out;
    unsigned *err;
};

// A logit as it is held: NaN as -inf (neither is ever drawn), -0 as +0.
__device__ __forceinline__ float sp_logit(float l) { return l == l ? l + 0.f : -INFINITY; }
// Keys ordered as the logits are.
__device__ __forceinline__ uint32_t sp_key(float l) {
    const uint32_t u = __float_as_uint(l);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float sp_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// ---------------------------------------------------------------------------
// 2^-t in fixed point, table-driven (P. T. P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point
// arithmetic", 1989): t = n - j / 8 - g with j = 0 .. 7 and |g| <= 1/16, so
// 2^-t = 2^-n 2^(j/8) 2^g, 2^g by its Taylor polynomial.  In pairs of floats,
// since fp64 runs at 1/64 of the fp32 rate here: relative error below 2^-37
// (the worst of 2 million random arguments: 2^-38.1).  Eight entries of 16 bytes
// span the 32 banks once: lanes that read different ones never conflict.
// ---------------------------------------------------------------------------
struct alignas(16) ExpEntry {
    u64 fixed;  // 2^(j / 8) with 43 fraction bits
    float hi, lo;  // the same as a pair of floats
};
constexpr int kExpEntries = 8;
constexpr double exp_series(double x) {
    double term = 1, sum = 1;
    for (int i = 1; i < 30; ++i) term *= x / i, sum += term;
    return sum;
}
struct ExpTable {
    ExpEntry e[kExpEntries];
};
constexpr double kLn2 = 0.69314718055994530942;
constexpr ExpTable make_exp_table() {
    ExpTable t{};
    for (int j = 0; j < kExpEntries; ++j) {
        const double v = exp_series(j * (kLn2 / 8));
        t.e[j].fixed = (u64)(v * (double)(2ull << kFrac) + 0.5);
        t.e[j].hi = (float)v;
        t.e[j].lo = (float)(v - (double)t.e[j].hi);
    }
    return t;
}
__constant__ ExpTable kExp = make_exp_table();

// log2(e) / T as a pair of floats
struct Scale {
    float hi, lo;
};

// Two floats in one instruction (rounded each as the scalar operation is).
struct F2 {
    u64 v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 sub(F2 a, F2 b) { return fma(b, f2(-1.f), a); }  // (exact product: rounded once)

// The weights of two logits in a row whose largest is top (l <= top).
__device__ __forceinline__ void sp_weights(float l0, float l1, float top, const Scale &c, const ExpEntry *table, u64 *w) {
    const F2 l = f2(l0, l1), tp = f2(top);
    // d + e = top - l exactly
    const F2 d = sub(tp, l), bb = sub(tp, d);
    const F2 e = add(sub(tp, add(d, bb)), sub(bb, l));
    // t + tl = (d + e) log2(e) / T
    const F2 t2 = mul(d, f2(c.hi));
    float t0, t1;
    split(t2, t0, t1);
    const bool some0 = t0 < 43.5f, some1 = t1 < 43.5f;  // otherwise 2^-t is below half of the last place
    const F2 t = f2(some0 ? t0 : 0.f, some1 ? t1 : 0.f), nt = mul(t, f2(-1.f));
    const F2 tl = add(fma(d, f2(c.hi), nt), fma(d, f2(c.lo), mul(e, f2(c.hi))));
    // (integers are read off the low bits of a float near 1.5 2^23: conversions run at an eighth of the rate)
    constexpr float kRound = 12582912.f;
    const F2 vr = fma(t, f2(8.f), f2(kRound));
    float v0f, v1f;
    split(vr, v0f, v1f);
    const int v0 = __float_as_int(v0f) - __float_as_int(kRound), v1 = __float_as_int(v1f) - __float_as_int(kRound);
    const F2 g = fma(add(vr, f2(-kRound)), f2(0.125f), nt);  // v / 8 - t: exact
    const ExpEntry x0 = table[-v0 & 7], x1 = table[-v1 & 7];
    const F2 xh = f2(x0.hi, x1.hi), xl = f2(x0.lo, x1.lo);
    // 2^(g - tl) - 1 = a + b + a^2 / 2 + .. with a + b = (g - tl) ln 2
    constexpr float kL = (float)kLn2, kLl = (float)(kLn2 - (double)(float)kLn2);
    const F2 a = mul(g, f2(kL)), na = mul(a, f2(-1.f));
    const F2 b = add(fma(g, f2(kL), na), fma(g, f2(kLl), mul(tl, f2(-kL))));
    // a^2 / 2 = h + hl; u = a^3 / 6 + .. + a^6 / 720; b times the whole 2^g
    const F2 ha = mul(a, f2(0.5f)), h = mul(ha, a), hl = fma(ha, a, mul(h, f2(-1.f)));
    F2 q = fma(a, f2(1.f / 360.f), f2(1.f / 60.f));
    q = fma(a, q, f2(1.f / 12.f));
    q = fma(a, q, f2(1.f / 3.f));
    // 2^(j/8) (a + h + rest) = y + yl
    const F2 s1 = add(a, h), u = mul(mul(h, a), q), rest = add(u, add(fma(b, add(s1, u), b), hl));
    const F2 s2 = add(add(sub(a, s1), h), rest);
    const F2 p = mul(xh, s1), pl = add(fma(xh, s1, mul(p, f2(-1.f))), fma(xh, s2, mul(xl, s1)));
    const F2 y = add(p, pl), yl = add(sub(p, y), pl);
    // y's leading part on a grid of 2^-21, the rest below it
    const F2 r1 = fma(y, f2(2097152.f), f2(kRound)), i1 = add(r1, f2(-kRound));
    const F2 r2 = fma(add(fma(i1, f2(-1.f / 2097152.f), y), yl), f2(8796093022208.f), f2(kRound));
    float r10, r11, r20, r21;
    split(r1, r10, r11);
    split(r2, r20, r21);
    auto fixed = [&](u64 base, float hi, float lo, int v, bool some) {
        const long long m = (long long)base + (long long)(__float_as_int(hi) - __float_as_int(kRound)) * (1 << (kFrac - 20)) +
                            (__float_as_int(lo) - __float_as_int(kRound));
        const u64 r = (((u64)m >> ((v + 7) >> 3)) + 1) >> 1;
        return some ? r : 0ull;  // (no branch: several logits are worked on at a time)
    };
    w[0] = fixed(x0.fixed, r10, r20, v0, some0);
    w[1] = fixed(x1.fixed, r11, r21, v1, some1);
}

template <typename V>
__device__ __forceinline__ V warp_add(V v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// f < 1 as a multiple of 2^-64 (exact but for what lies below)
__device__ __forceinline__ u64 frac64(float f) { return __float2ull_rz(f * 18446744073709551616.f); }

// What the CTAs of a row share; a CTA's copy is written by the others through
// distributed shared memory, each word once between two cluster barriers.
struct SampleShare {
    float top[kMaxCluster];
    u64 sum[kMaxCluster];
    uint32_t count[kMaxCluster];  // of gathered logits, or of those equal to the cut
    uint32_t first[kMaxCluster];  // first id of the largest logit; ties of the final pass
    // what a histogram says (every CTA finds it by itself)
    uint32_t bin, found, fewest;
    u64 want, wanted, total;
    // what rank 0 settles, in its copy read by all (before they enter the next barrier; it is written behind one)
    uint32_t key;
    u64 left;
    uint32_t gathered;  // this CTA's
};

struct alignas(16) SampleSmem {
    SampleShare sh;
    ExpEntry exp[kExpEntries];
    union {
        struct {
            alignas(16) uint32_t lo[kBins];  // counts in lo, or masses in (hi, lo); read by the row's other CTAs
            alignas(16) uint32_t hi[kBins];
        };
        struct {                    // rank 0, once nobody reads its histogram
            u64 mass[kList];        // weights of the sorted list
            uint32_t order[kList];  // (id, place) of the kept ones
        };
    };
    alignas(16) u64 list[kList];  // (key, ~id) of gathered tokens, in rank 0 sorted; each warp's queue (each_above)
    u64 wsum[kSpWarps];
    uint32_t wcnt[kSpWarps];
};
// 16-byte accesses: the histograms and the row behind this object
static_assert(offsetof(SampleSmem, lo) % 16 == 0 && offsetof(SampleSmem, hi) % 16 == 0 &&
                  offsetof(SampleSmem, exp) % 16 == 0 && sizeof(SampleSmem) % 16 == 0,
              "alignment");

// Inclusive sums over the block of two values per thread (2t, 2t + 1).
__device__ __forceinline__ void block_scan2(u64 &x0, u64 &x1, u64 *wsum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    u64 c = x0 + x1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += y;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = c;
    __syncthreads();
    for (int w = 0; w < warp; ++w) c += wsum[w];
    x0 = c - x1, x1 = c;
}

// Sort v[0 .. n), distinct but for the padding (`pad`, last in the order), ascending or descending; n <= kList, v has
// room for kList.  Few: every element counts those in front of it.  More: a bitonic network over two elements per
// thread, 2t and 2t + 1: partners up to 32 apart are a shuffle away, others meet in v.
template <bool Up, typename V>
__device__ __forceinline__ void block_sort(V *v, int n, V pad) {
    const int t = threadIdx.x;
    if (n <= 128) {
        V x = pad;
        int place = 0;
        if (t < n) {
            x = v[t];
#pragma unroll 8
            for (int j = 0; j < n; ++j) place += Up ? v[j] < x : v[j] > x;
        }
        __syncthreads();
        if (t < n) v[place] = x;
        __syncthreads();
        return;
    }
    int full = 256;
    while (full < n) full *= 2;
    V x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) x[e] = 2 * t + e < n ? v[2 * t + e] : pad;
    for (int size = 2; size <= full; size <<= 1) {
        const bool up = ((2 * t & size) == 0) == Up;
        int stride = size >> 1;
        for (; stride > 32; stride >>= 1) {
            __syncthreads();
            v[2 * t] = x[0], v[2 * t + 1] = x[1];
            __syncthreads();
            const bool low = ((2 * t & stride) == 0) == up;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const V o = v[(2 * t + e) ^ stride];
                x[e] = (o < x[e]) == low ? o : x[e];
            }
        }
        for (; stride > 1; stride >>= 1) {
            const bool low = ((2 * t & stride) == 0) == up;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const V o = __shfl_xor_sync(0xffffffffu, x[e], stride >> 1);
                x[e] = (o < x[e]) == low ? o : x[e];
            }
        }
        if ((x[0] > x[1]) == up) {
            const V y = x[0];
            x[0] = x[1], x[1] = y;
        }
    }
    __syncthreads();
    v[2 * t] = x[0], v[2 * t + 1] = x[1];
    __syncthreads();
}

// Held: the row is kept in shared memory; otherwise (rows of more ids than a cluster holds) every pass reads the
// logits again.
template <typename T, bool Held>
__global__ void __launch_bounds__(kSpThreads, 2) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t sp_raw[];
    SampleSmem &sm = *reinterpret_cast<SampleSmem *>(sp_raw);
    float *val = reinterpret_cast<float *>(sp_raw + sizeof(SampleSmem));
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int r = blockIdx.x / C;
    constexpr unsigned kAll = 0xffffffffu;
    // the same object in another CTA of the row
    auto peer = [&](int c) -> SampleSmem & { return *cluster.map_shared_rank(&sm, c); };
    auto meet = [&]() {
        if (C > 1) cluster.sync();
        else __syncthreads();
    };
    if (tid < kExpEntries) sm.exp[tid] = kExp.e[tid];
    cg::cluster_group::arrival_token here;  // every CTA of the row runs before another writes to its shared memory
    if (C > 1) here = cluster.barrier_arrive();
    pdl_trigger();
    pdl_wait();

    if (a.by_work) {
        // 0: a top-p over all ids, or a long top-k; 1: no filter; 2: a short top-k; 3: greedy.  A row's position is by
        // (class, index); every CTA finds the one of its cluster's.
        auto work = [&](int i) {
            if (i >= a.n_rows) return 4;
            const int ki = a.top_k ? a.top_k[i] : 0;
            const float pi = a.top_p ? a.top_p[i] : 1.f, ti = a.temperature ? a.temperature[i] : 1.f;
            const bool listed = ki > 0 && ki <= kList;
            return ti == 0.f ? 3 : listed ? 2 : pi < 1.f || (ki > kList && ki < a.V) ? 0 : 1;
        };
        int place = r, cls = -1, before;
        do {  // the class
            ++cls, before = place;
            for (int i = 0; i < a.n_rows; i += kSpThreads) place -= __syncthreads_count(work(i + tid) == cls);
        } while (place >= 0 && cls < 3);
        place = before;
        for (int i = 0; i < a.n_rows; i += kSpThreads) {
            const bool in = work(i + tid) == cls;
            const uint32_t mask = __ballot_sync(kAll, in);
            if (lane == 0) sm.wcnt[warp] = __popc(mask);
            const int count = __syncthreads_count(in);
            if (place < count) {
                int rank_in = __popc(mask & ((1u << lane) - 1u));
                for (int w = 0; w < warp; ++w) rank_in += sm.wcnt[w];
                if (in && rank_in == place) sm.sh.bin = (uint32_t)(i + tid);
                break;
            }
            place -= count;
            __syncthreads();
        }
        __syncthreads();
        r = (int)sm.sh.bin;
        __syncthreads();
    }
    const float temp = a.temperature ? a.temperature[r] : 1.f, p = a.top_p ? a.top_p[r] : 1.f,
                mp = a.min_p ? a.min_p[r] : 0.f, u = a.uniform[r];
    const int k = a.top_k ? a.top_k[r] : 0;
    // this CTA's ids: first .. first + n - 1
    const int first = min(a.V, rank * a.per), n = min(a.V - first, a.per);
    const T *row = (const T *)a.logits + (size_t)r * a.ld + first;
    auto at = [&](int i) -> float {
        if constexpr (Held) return val[i];
        else return sp_logit(Elem<T>::to_f(row[i]));
    };
    // logits i .. i + 3 below `end` (a multiple of four, or n; held rows are padded to a multiple of four with -inf)
    auto load4 = [&](int i, int end, float *l) {
        if (i >= end) return;
        if constexpr (Held) {
            const float4 x = *reinterpret_cast<const float4 *>(val + i);
            l[0] = x.x, l[1] = x.y, l[2] = x.z, l[3] = x.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < end) l[e] = at(i + e);
        }
    };
    // f(i, logit) for every id of this CTA, in any order (held rows are padded to a multiple of four with -inf)
    auto each = [&](auto f) {
        if constexpr (Held) {
            for (int i = 4 * tid; i < n; i += 4 * kSpThreads) {
                const float4 x = *reinterpret_cast<const float4 *>(val + i);
                f(i, x.x), f(i + 1, x.y), f(i + 2, x.z), f(i + 3, x.w);
            }
        } else {
            for (int i = tid; i < n; i += kSpThreads) f(i, at(i));
        }
    };
    // the same by fours (f(first id, four logits); those past the end are -inf)
    auto each4 = [&](auto f) {
        for (int i = 4 * tid; i < n; i += 4 * kSpThreads) {
            float l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) l[e] = -INFINITY;
            load4(i, n, l);
            f(i, l);
        }
    };
    float top = -INFINITY;
    if constexpr (!Held) {
        for (int i = tid; i < n; i += kSpThreads) top = fmaxf(top, at(i));
    } else {
        constexpr int VEC = Elem<T>::kPer16;
        const int head = min(n, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
        const int body = (n - head) / VEC;
        auto put = [&](int i, float l) {
            l = sp_logit(l);
            val[i] = l;
            top = fmaxf(top, l);
        };
        if (tid < head) put(tid, Elem<T>::to_f(row[tid]));
#pragma unroll 4
        for (int i = tid; i < body; i += kSpThreads) {
            float x[VEC];
            load16_stream(row + head + i * VEC, x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) put(head + i * VEC + e, x[e]);
        }
        for (int i = head + body * VEC + tid; i < n; i += kSpThreads) put(i, Elem<T>::to_f(row[i]));
        if (tid < 4 && n + tid < (n + 3) / 4 * 4) val[n + tid] = -INFINITY;
    }
    if (C > 1) cluster.barrier_wait(std::move(here));
    if (!(temp >= 0.f && temp <= 1e6f && p >= 0.f && p <= 1.f && mp >= 0.f && mp <= 1.f && u >= 0.f && u < 1.f)) {
        if (rank == 0 && tid == 0) raise_err(a.err, ERR_BAD_SAMPLE), a.out[r] = -1;
        return;  // (the whole cluster)
    }
    const float own = top;  // the largest of this thread's
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    if (lane == 0) sm.wcnt[warp] = __float_as_uint(top);
    __syncthreads();
    if (warp == 0) {
        top = lane < kSpWarps ? __uint_as_float(sm.wcnt[lane]) : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        if (lane < C) peer(lane).sh.top[rank] = top;
    }
    meet();
    top = -INFINITY;
    for (int c = 0; c < C; ++c) top = fmaxf(top, sm.sh.top[c]);

    if (top == -INFINITY) {  // nothing but -inf and NaN
        if (rank == 0 && tid == 0) a.out[r] = -1;
        return;
    }
    if (temp == 0.f) {  // the lowest id of the largest logit
        uint32_t low = 0xffffffffu;
        each([&](int i, float l) {
            if (l == top) low = min(low, (uint32_t)(first + i));
        });
        low = __reduce_min_sync(kAll, low);
        if (lane == 0) sm.wcnt[warp] = low;
        __syncthreads();
        if (warp == 0) {
            low = __reduce_min_sync(kAll, lane < kSpWarps ? sm.wcnt[lane] : 0xffffffffu);
            if (lane == 0) peer(0).sh.first[rank] = low;
        }
        meet();
        if (rank == 0 && tid == 0) {
            for (int c = 0; c < C; ++c) low = min(low, sm.sh.first[c]);
            a.out[r] = (int32_t)low;
        }
        return;
    }

    Scale cs;
    {
        constexpr float kE = 1.4426950408889634074f, kEl = (float)(1.4426950408889634074 - (double)kE);
        cs.hi = fminf(__fdiv_rn(kE, temp), 3e38f);
        cs.lo = __fdiv_rn(__fmaf_rn(-cs.hi, temp, kE) + kEl, temp);
        if (!(fabsf(cs.lo) < 1e30f)) cs.lo = 0.f;  // (a subnormal T: only the largest logits keep weight)
    }
    auto weights = [&](float l0, float l1, u64 *w) {
        sp_weights(l0, l1, top, cs, sm.exp, w);
        if (l0 == top) w[0] = 1ull << kFrac;  // (top may be +inf)
        if (l1 == top) w[1] = 1ull << kFrac;
    };
    auto weight = [&](float l) {
        u64 w[2];
        weights(l, l, w);
        return w[0];
    };
    // The bin of a logit: octaves below the largest, kBins of them over 43.5 (monotone in the logit;
    // the last bin also takes everything without weight)
    auto bin_of = [&](float l) {
        const float d = __fmul_rn(__fmul_rn(__fsub_rn(top, l), cs.hi), (float)(kBins / 43.5));
        const float near = fminf(d, (float)(kBins - 1)) + 8388608.f;  // (to the nearest: the low bits of 2^23 + bin)
        return l == top ? 0 : __float_as_int(near) & (2 * kBins - 1);
    };
    // a logit that none of bins 0 .. b is below (one bin of slack for the roundings)
    auto low_of = [&](int b) { return top - (float)(b + 2) * (float)(43.5 / kBins) * 1.000001f / cs.hi; };
    // and one that none of bins b .. is above
    auto high_of = [&](int b) { return b < 3 ? INFINITY : top - (float)(b - 2) * (float)(43.5 / kBins) * 0.999999f / cs.hi; };
    SampleSmem &root = peer(0);
    // f(l0, l1, on0, on1) for 64 logits above the cut at a time (all lanes; on: this lane has that one), g(l) for every
    // logit, over a warp's contiguous stretch of ids; the logits above are queued so that few of them cost little.
    const int per_warp = (n + 4 * kSpThreads - 1) / (4 * kSpThreads) * 128;
    const int i0 = min(n, warp * per_warp), i1 = min(n, i0 + per_warp);
    auto each_above = [&](float above, auto f, auto g) {
        constexpr int kQueue = 2 * kList / kSpWarps;  // floats per warp
        static_assert(kQueue >= 63 + 64, "what two ballots add to a rest of 63");
        float *queue = reinterpret_cast<float *>(sm.list) + warp * kQueue;
        int held = 0;
        for (int i = i0 + 4 * lane; i - 4 * lane < i1; i += 128) {
            float l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) l[e] = -INFINITY;
            load4(i, i1, l);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g(l[e]);
                const uint32_t mask = __ballot_sync(kAll, l[e] > above);
                if (l[e] > above) queue[held + __popc(mask & ((1u << lane) - 1u))] = l[e];
                held += __popc(mask);
                if ((e & 1) && held >= 64) {
                    __syncwarp();
                    held -= 64;
                    f(queue[held + lane], queue[held + 32 + lane], true, true);
                    __syncwarp();
                }
            }
        }
        __syncwarp();
        const bool on0 = lane < held, on1 = lane + 32 < held;
        if (held > 0) f(on0 ? queue[lane] : above, on1 ? queue[lane + 32] : above, on0, on1);
    };

    // the mass that a prefix has to reach: p times the whole, rounded up, at least one
    const u64 pf = p < 1.f ? frac64(p) : 0ull;
    auto share = [&](u64 whole) {
        const u64 want = __umul64hi(pf, whole) + (pf * whole != 0);
        return want < 1 ? 1ull : want;
    };
    const u64 least = __float2ull_ru(mp * (float)(1ull << kFrac));
    bool by_count = k > 0 && k < a.V;
    // kept: logits above cut, and the first `ties` of those equal to it
    float cut = -INFINITY;
    uint32_t ties = 0xffffffffu;

    // Histogram over the bins of(l) >= 0 of the logits above the cut, counts or masses, added up over the row's CTAs
    // by each of them.  pick(total) says what is wanted, and sm.sh gets whether that much is there (found), the bin in
    // which it is reached from the largest logits down, what is left of it for that bin (want) and all of it (wanted).
    // `down`: larger logits are in higher bins.  `largest`: of each thread's largest logit alone.  A barrier has to
    // follow before the next histogram.
    auto histogram = [&](bool by_mass, bool down, bool largest, auto of, auto pick) {
        for (int i = tid; i < kBins / 4; i += kSpThreads) {
            reinterpret_cast<uint4 *>(sm.lo)[i] = make_uint4(0, 0, 0, 0);
            if (by_mass) reinterpret_cast<uint4 *>(sm.hi)[i] = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
        auto put = [&](float l, u64 w) {
            const int b = l > cut ? of(l) : -1;
            if (b < 0) return;
            const uint32_t wl = (uint32_t)w, old = atomicAdd(&sm.lo[b], wl);
            const uint32_t wh = (uint32_t)(w >> 32) + (old + wl < old);
            if (wh) atomicAdd(&sm.hi[b], wh);
        };
        if (by_mass && cut != -INFINITY)
            each_above(
                cut,
                [&](float l0, float l1, bool on0, bool on1) {
                    u64 w[2];
                    weights(l0, l1, w);
                    if (on0) put(l0, w[0]);
                    if (on1) put(l1, w[1]);
                },
                [](float) {});
        else if (by_mass)
            each4([&](int, const float *l) {
                u64 w[4];
                weights(l[0], l[1], w), weights(l[2], l[3], w + 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) put(l[e], w[e]);
            });
        else {
            auto count = [&](int, float l) {
                const int b = l > cut ? of(l) : -1;
                if (b >= 0) atomicAdd(&sm.lo[b], 1u);
            };
            if (largest) count(0, own);
            else each(count);
        }
        meet();
        {
            // thread t: four bins, in the order of descending logits
            const int q = down ? kBins / 4 - 1 - tid : tid;
            u64 x[4] = {0, 0, 0, 0}, s = 0;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) {  // (all loads in flight)
                if (c >= C) break;
                const SampleSmem &o = peer(c);
                const uint4 lo = reinterpret_cast<const uint4 *>(o.lo)[q];
                uint4 hi = make_uint4(0, 0, 0, 0);
                if (by_mass) hi = reinterpret_cast<const uint4 *>(o.hi)[q];
                x[0] += (u64)hi.x << 32 | lo.x, x[1] += (u64)hi.y << 32 | lo.y;
                x[2] += (u64)hi.z << 32 | lo.z, x[3] += (u64)hi.w << 32 | lo.w;
            }
            s = x[0] + x[1] + x[2] + x[3];
            u64 incl = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 y = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += y;
            }
            if (lane == 31) sm.wsum[warp] = incl;
            if (tid == 0) sm.sh.found = 0;
            __syncthreads();
            u64 base = incl - s, all = 0;
#pragma unroll
            for (int w = 0; w < kSpWarps; ++w) {
                const u64 y = sm.wsum[w];
                base += w < warp ? y : 0ull;
                all += y;
            }
            const u64 want = pick(all);
            if (tid == 0) sm.sh.total = all, sm.sh.wanted = want, sm.sh.fewest = 0;
            if (base < want && want <= base + s) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const u64 y = down ? x[3 - e] : x[e];
                    if (base < want && want <= base + y) {
                        sm.sh.bin = (uint32_t)(4 * q + (down ? 3 - e : e));
                        sm.sh.want = want - base;
                        sm.sh.found = 1;
                    }
                    base += y;
                }
            }
            if (by_mass && !down) {
                // how many logits the bins down to that one hold at least: a bin's mass over the largest weight in it
                // (its upper edge, half a bin above; a little more for the roundings)
                __syncthreads();
                float few = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int b = 4 * tid + e;
                    if (sm.sh.found && b <= (int)sm.sh.bin)
                        few += (float)x[e] * exp2f(((float)b - 0.51f) * (float)(43.5 / kBins) - (float)kFrac);
                }
                few = warp_add(few * 0.999f);
                if (lane == 0) atomicAdd(&sm.sh.fewest, (uint32_t)fminf(few, 1e9f));
            }
        }
        __syncthreads();
    };

    // Every (key, ~id) of the logits above the cut that take(l) names, in rank 0's list; returns how many there
    // are (more than kList: the list is not to be used).
    // No logit below `low` or above `high` is taken.
    auto collect = [&](float low, float high, auto take) {
        if (tid == 0) sm.sh.gathered = 0;
        __syncthreads();
        each4([&](int i, const float *l) {
            if (!(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= low)) return;
            if (*const_cast<volatile uint32_t *>(&sm.sh.gathered) > kList) return;  // too many: only that counts
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!(l[e] > cut && l[e] >= low && l[e] <= high) || !take(l[e])) continue;
                const uint32_t j = atomicAdd(&sm.sh.gathered, 1u);
                if (j < kList) sm.list[j] = (u64)sp_key(l[e]) << 32 | (uint32_t) ~(first + i + e);
            }
        });
        __syncthreads();
        if (tid < C) peer(tid).sh.count[rank] = sm.sh.gathered;
        meet();
        uint32_t m = 0;
        for (int c = 0; c < C; ++c) m += sm.sh.count[c];
        if (C > 1) {
            if (rank == 0 && m <= kList) {  // two warps per CTA
                const int from = warp / 2 + 1;
                if (from < C) {
                    uint32_t to = 0;
                    for (int c = 0; c < from; ++c) to += sm.sh.count[c];
                    const u64 *theirs = peer(from).list;
                    for (uint32_t j = tid & 63; j < sm.sh.count[from]; j += 64) sm.list[to + j] = theirs[j];
                }
            }
            meet();  // (the other CTAs' lists are free, and they may leave)
        } else {
            __syncthreads();
        }
        return (int)m;
    };

    // Rank 0: the token, from a list of m that holds all that may be kept: of the first `most` by logit descending
    // and id ascending those whose mass in front is below `want` (share_of_most: p times the mass of the `most`).
    auto finish = [&](int m, int most, u64 want, bool share_of_most) {
        block_sort<false>(sm.list, m, 0ull);
        u64 w[2] = {0, 0}, c[2];
        if (2 * tid < most) {
            weights(sp_value((uint32_t)(sm.list[2 * tid] >> 32)), sp_value((uint32_t)(sm.list[2 * tid + 1] >> 32)), w);
            if (2 * tid + 1 >= most) w[1] = 0;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) c[e] = sm.mass[2 * tid + e] = w[e];
        block_scan2(c[0], c[1], sm.wsum);
        if (share_of_most) {
            if (tid == kSpThreads - 1) sm.sh.total = c[1];
            __syncthreads();
            want = share(sm.sh.total);
        }
        bool keep[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) keep[e] = w[e] >= max(least, 1ull) && c[e] - w[e] < want;
        const int kept = __syncthreads_count(keep[0]) + __syncthreads_count(keep[1]);  // a prefix
        if (2 * tid == kept - 1) sm.sh.total = c[0];
        if (2 * tid + 1 == kept - 1) sm.sh.total = c[1];
        if (kept > 128) {
            // the id by its upper, then its lower bits: masses per digit, and the one in which u times the total lies
            // (sorted by id instead, 5 500 to 8 200 cycles: one row of 4486 at top-p 0.9 17.3 us, now 16.1)
            const int shift = max(0, 22 - __clz(a.V - 1));  // (at most 2^10 digits each)
            uint32_t digit = 0;
            u64 target = 0;
            for (int level = 0; level < 2; ++level) {
                __syncthreads();
                if (level == 0) target = __umul64hi(frac64(u), sm.sh.total);
                *reinterpret_cast<uint2 *>(sm.lo + 2 * tid) = *reinterpret_cast<uint2 *>(sm.hi + 2 * tid) = make_uint2(0, 0);
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (!keep[e]) continue;
                    const uint32_t id = ~(uint32_t)sm.list[2 * tid + e];
                    if (level == 1 && id >> shift != digit) continue;
                    const uint32_t b = level == 0 ? id >> shift : id & ((1u << shift) - 1u);
                    const uint32_t wl = (uint32_t)w[e], old = atomicAdd(&sm.lo[b], wl);
                    const uint32_t wh = (uint32_t)(w[e] >> 32) + (old + wl < old);
                    if (wh) atomicAdd(&sm.hi[b], wh);
                }
                __syncthreads();
                u64 x[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) x[e] = c[e] = (u64)sm.hi[2 * tid + e] << 32 | sm.lo[2 * tid + e];
                block_scan2(c[0], c[1], sm.wsum);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (c[e] - x[e] <= target && target < c[e]) {
                        sm.sh.bin = 2 * tid + e, sm.sh.want = target - (c[e] - x[e]);
                        if (level == 1) a.out[r] = (int32_t)(digit << shift | (uint32_t)(2 * tid + e));
                    }
                __syncthreads();
                digit = sm.sh.bin, target = sm.sh.want;
            }
            return;
        }
        // the kept ones in the order of their ids
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int j = 2 * tid + e;
            if (j < kept) sm.order[j] = ~(uint32_t)sm.list[j] << 10 | (uint32_t)j;
        }
        __syncthreads();
        const u64 target = __umul64hi(frac64(u), sm.sh.total);
        block_sort<true>(sm.order, kept, 0xffffffffu);
        uint32_t o[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            o[e] = 2 * tid + e < kept ? sm.order[2 * tid + e] : 0u;
            w[e] = c[e] = 2 * tid + e < kept ? sm.mass[o[e] & (kList - 1)] : 0ull;
        }
        block_scan2(c[0], c[1], sm.wsum);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (c[e] - w[e] <= target && target < c[e]) a.out[r] = (int32_t)(o[e] >> 10);
    };

    // The cut from bin bin0 of the logits' histogram, in which what is left to reach is `want`: while the bin holds
    // more logits than a list takes, it is split by 11, 11 and 10 bits of their keys.
    auto settle = [&](bool by_mass, int bin0, u64 want) {
        uint32_t prefix = 0;
        for (int level = 0;; ++level) {
            auto of = [&](float l) {  // the bin of the keys at this level, or -1
                const uint32_t key = sp_key(l);
                int b = -1;
                if (bin_of(l) == bin0) {
                    if (level == 1) b = (int)(key >> 21);
                    else if (level == 2) b = (key >> 21) == (prefix >> 21) ? (int)((key >> 10) & 2047u) : -1;
                    else b = (key >> 10) == (prefix >> 10) ? (int)(key & 1023u) : -1;
                }
                return b;
            };
            if (level > 0) {
                const u64 goal = want;
                histogram(by_mass, true, false, of, [=](u64) { return goal; });
                want = sm.sh.want;
                prefix |= sm.sh.bin << (level == 1 ? 21 : level == 2 ? 10 : 0);
                if (level == 3) {
                    cut = sp_value(prefix);
                    meet();
                    break;
                }
            }
            const int low = level == 0 ? 31 : level == 1 ? 21 : 10;  // bits of the keys not yet fixed
            const uint32_t high = level == 0 ? 0u : prefix >> low;
            auto in_bin = [&](float l) { return bin_of(l) == bin0 && (level == 0 || sp_key(l) >> low == high); };
            const int m = collect(low_of(bin0), high_of(bin0), in_bin);
            if (m > kList) continue;
            if (rank == 0) {
                block_sort<false>(sm.list, m, 0ull);
                uint32_t key[2];
                u64 x[2], c[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 2 * tid + e;
                    key[e] = j < m ? (uint32_t)(sm.list[j] >> 32) : 0u;
                    x[e] = c[e] = j >= m ? 0ull : by_mass ? weight(sp_value(key[e])) : 1ull;
                }
                block_scan2(c[0], c[1], sm.wsum);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (c[e] - x[e] < want && want <= c[e]) sm.sh.key = key[e];
                __syncthreads();
                const uint32_t hit = sm.sh.key;
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // the first of those equal to it says what is left for them
                    const int j = 2 * tid + e;
                    if (j < m && key[e] == hit && (j == 0 || (uint32_t)(sm.list[j - 1] >> 32) != hit))
                        sm.sh.left = want - (c[e] - x[e]);
                }
            }
            meet();
            cut = sp_value(root.sh.key);
            want = root.sh.left;
            break;
        }
        const u64 w = by_mass ? weight(cut) : 1ull;
        ties = (uint32_t)((want + w - 1) / w);
    };

    if (by_count) {
        // No logit of the k largest is below the k-th largest of the threads' largest: with k well below the number of
        // threads few more than k lie above it (n ln(n / (n - k)) of logits in any order, n threads), and counting
        // one logit a thread is enough.
        if (k <= kList / 2 && k <= kSpThreads / 2 * C) {
            histogram(false, false, true, bin_of, [&](u64) { return (u64)k; });
            const int bin = (int)sm.sh.bin;
            if (sm.sh.found && bin != kBins - 1) {
                const int m = collect(low_of(bin), high_of(0), [&](float l) { return bin_of(l) <= bin; });
                if (m <= kList) {
                    if (rank == 0) finish(m, k, ~0ull, p < 1.f);
                    return;
                }
            } else {
                meet();
            }
        }
        histogram(false, false, false, bin_of, [&](u64) { return (u64)k; });
        const int bin = (int)sm.sh.bin;
        const u64 want = sm.sh.want;
        // fewer than k logits, or the k-th without weight: the same as all kept
        by_count = sm.sh.found && bin != kBins - 1;
        if (!by_count) meet();
        if (by_count) {
            if (k <= kList) {
                const int m = collect(low_of(bin), high_of(0), [&](float l) { return bin_of(l) <= bin; });
                if (m <= kList) {
                    if (rank == 0) finish(m, k, ~0ull, p < 1.f);
                    return;
                }
            }
            settle(false, bin, want);
        }
    }
    if (p < 1.f) {
        const u64 wt = by_count ? weight(cut) : 0ull;
        histogram(true, false, false, bin_of, [&](u64 above) { return share(above + wt * (by_count ? ties : 0u)); });
        const bool found = sm.sh.found;
        const int bin = (int)sm.sh.bin;
        const u64 want = sm.sh.want, wanted = sm.sh.wanted, above = sm.sh.total;
        const bool many = sm.sh.fewest > kList;
        if (found) {
            if (!many) {
                const int m = collect(low_of(bin), high_of(0), [&](float l) { return bin_of(l) <= bin; });
                if (m <= kList) {
                    if (rank == 0) finish(m, m, wanted, false);
                    return;
                }
            }
            settle(true, bin, want);
        } else if (wt) {  // it reaches into those equal to the k-th
            ties = (uint32_t)min((u64)ties, (wanted - above + wt - 1) / wt);
        }
    }
    // the tokens in the order of their ids, by the warps' stretches
    const bool tied = cut != -INFINITY;
    u64 wt = tied ? weight(cut) : 0ull;
    if (wt < least) wt = 0ull;
    u64 s = 0;
    uint32_t c = 0;
    if (tied) {
        each_above(
            cut,
            [&](float l0, float l1, bool on0, bool on1) {
                u64 w[2];
                weights(l0, l1, w);
                s += (on0 && w[0] >= least ? w[0] : 0ull) + (on1 && w[1] >= least ? w[1] : 0ull);
            },
            [&](float l) { c += l == cut; });
    } else {
        for (int i = i0 + 4 * lane; i < i1; i += 128) {
            float l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) l[e] = -INFINITY;
            load4(i, i1, l);
            u64 w[4];
            weights(l[0], l[1], w), weights(l[2], l[3], w + 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) s += w[e] >= least ? w[e] : 0ull;
        }
    }
    s = warp_add(s), c = warp_add(c);
    __syncthreads();
    if (lane == 0) sm.wsum[warp] = s, sm.wcnt[warp] = c;
    __syncthreads();
    if (warp == 0) {
        const u64 sc = warp_add(lane < kSpWarps ? sm.wsum[lane] : 0ull);
        const uint32_t cc = warp_add(lane < kSpWarps ? sm.wcnt[lane] : 0u);
        if (lane < C) peer(lane).sh.sum[rank] = sc, peer(lane).sh.first[rank] = cc;
    }
    meet();
    // mass of a stretch with s above the cut and c equal to it, `seen` of those equal lying in front
    auto stretch = [&](u64 sx, uint32_t cx, uint32_t seen) {
        return sx + wt * (seen < ties ? min(ties - seen, cx) : 0u);
    };
    u64 all = 0, start = 0, mine = 0;
    uint32_t seen = 0, before = 0;
    for (int x = 0; x < C; ++x) {
        const u64 part = stretch(sm.sh.sum[x], sm.sh.first[x], seen);
        if (x == rank) start = all, before = seen, mine = part;
        all += part;
        seen += sm.sh.first[x];
    }
    const u64 target = __umul64hi(frac64(u), all);
    if (target < start || target >= start + mine) return;  // (the whole CTA)
    for (int w = 0; w < warp; ++w) {
        start += stretch(sm.wsum[w], sm.wcnt[w], before);
        before += sm.wcnt[w];
    }
    if (lane == 0 && target >= start && target < start + stretch(s, c, before))
        sm.sh.bin = (uint32_t)warp, sm.sh.want = start, sm.sh.found = before;
    __syncthreads();
    // all warps look through the stretch in which it lies, four ids a thread (the warp alone, 32 ids at a time: one row
    // of 102018 in bf16 without a filter 18.6 us, now 13.7)
    const int j0 = min(n, (int)sm.sh.bin * per_warp), j1 = min(n, j0 + per_warp);
    u64 sum = sm.sh.want;
    seen = sm.sh.found;
    auto scan = [&](u64 v, u64 &total) {  // inclusive, over the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += y;
        }
        __syncthreads();
        if (lane == 31) sm.wsum[warp] = v;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < kSpWarps; ++w) {
            const u64 y = sm.wsum[w];
            v += w < warp ? y : 0ull;
            total += y;
        }
        return v;
    };
    for (int b = j0; b < j1; b += 4 * kSpThreads) {
        const int i = b + 4 * tid;
        float l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) l[e] = -INFINITY;
        load4(i, j1, l);
        u64 w[4] = {0, 0, 0, 0}, x = 0, total;
        if (i < j1) weights(l[0], l[1], w), weights(l[2], l[3], w + 2);
        if (tied) {
            uint32_t equal = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) equal += l[e] == cut;
            uint32_t place = seen + (uint32_t)scan(equal, total) - equal;
            seen += (uint32_t)total;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (l[e] < cut) w[e] = 0;
                if (l[e] == cut) w[e] = place++ < ties ? wt : 0ull;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (w[e] < least) w[e] = 0;
            x += w[e];
        }
        u64 to = sum + scan(x, total) - x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (to <= target && target < to + w[e]) a.out[r] = first + i + e;
            to += w[e];
        }
        sum += total;
        if (target < sum) break;
    }
}

}  // namespace

cudaError_t sample_rows(int dtype_bf16, const void *logits, int64_t ld, int n_rows, int V, const float *temperature,
                        const int32_t *top_k, const float *top_p, const float *min_p, const float *uniform,
                        int32_t *out, unsigned *err, int num_sms, cudaStream_t st) {
    if (n_rows <= 0) return cudaSuccess;
    constexpr int kMaxPer = (227 * 1024 - (int)sizeof(SampleSmem)) / 4 / kSpThreads * kSpThreads;
    // CTAs per row: as few as let two of them share an SM (192 mixed rows of 50257: three per row 61 us, four 67.5, two,
    // which leave an SM to one CTA, 101); more, by the ids, while all run at once (one row: one 19.1, two 14.7, four 12.2,
    // eight 12.7 us; one of 70000 at top-p 0.9: four 30.8, six 27.4).  Larger clusters do not fill every SM: 40 rows of
    // 102018 at top-p 0.9, five per row 57 us, seven 71, eight 77.
    constexpr int kPairPer = (113 * 1024 - (int)sizeof(SampleSmem)) / 4;
    int C = std::min(kMaxCluster, (V + kPairPer - 1) / kPairPer);
    const int goal = V <= 8192 ? 1 : V <= 16384 ? 2 : std::min(kMaxCluster, std::max(4, (V + 12999) / 13000));
    while (C < goal && (int64_t)n_rows * (C + 1) <= (C < 4 ? 2 * num_sms : num_sms + num_sms / 2)) ++C;
    const int per = ((V + C - 1) / C + 3) / 4 * 4;
    const bool held = per <= kMaxPer;
    // more rows than run at once: the ones with the most work first, so that none of them starts last (with thousands
    // the last ones matter little, and every CTA looks through all of them)
    const bool by_work = (int64_t)n_rows * C > 2 * num_sms && n_rows <= 1024 && (temperature || top_k || top_p);
    SampleArgs a{logits, ld, V, per, n_rows, by_work, temperature, top_p, min_p, uniform, top_k, out, err};
    const void *f = dtype_bf16 ? (held ? (const void *)sample_kernel<bf16, true> : (const void *)sample_kernel<bf16, false>)
                               : (held ? (const void *)sample_kernel<float, true> : (const void *)sample_kernel<float, false>);
    const size_t smem = sizeof(SampleSmem) + (held ? (size_t)per * 4 : 0);
    cudaError_t e = max_smem_once(f, (int)(sizeof(SampleSmem) + kMaxPer * 4));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_rows * C);
    cfg.blockDim = dim3(kSpThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, f, args);
}

}  // namespace orca
