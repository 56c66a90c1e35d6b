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
#include <cfloat>

#include "common.cuh"
#include "kernels.cuh"

namespace orca {

namespace {

constexpr int kSpThreads = 1024, kSpWarps = kSpThreads / 32;
constexpr int kFrac = 42;  // fraction bits of a weight
using u64 = unsigned long long;

struct SampleArgs {
    const void *logits;
    int64_t ld;
    int V;
    const float *temperature, *top_p, *min_p, *uniform;
    const int32_t *top_k;
    int32_t *out;
    unsigned *err;
};

// Keys ordered as the logits are (a row's NaN below everything; -0 = +0).
__device__ __forceinline__ uint32_t sp_key(float l) {
    if (l != l) return 0u;
    const uint32_t u = __float_as_uint(l + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float sp_value(uint32_t key) {
    return key == 0u ? -INFINITY : __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// The weight of a key in fixed point; inv_t = 1 / T.
__device__ __forceinline__ u64 sp_weight(uint32_t key, uint32_t top, double inv_t) {
    if (key == top) return 1ull << kFrac;
    const double x = ((double)sp_value(key) - (double)sp_value(top)) * inv_t;
    if (!(x > -30.5)) return 0ull;  // below half of the last place
    return (u64)llrint(exp(x) * (double)(1ull << kFrac));
}

template <typename V>
__device__ __forceinline__ V warp_add(V v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// x * f for a fraction f given as f * 2^64
__device__ __forceinline__ u64 frac64(float f) { return (u64)((double)f * 18446744073709551616.0); }

struct SampleSmem {
    u64 mass[256];
    uint32_t count[256];
    u64 wsum[kSpWarps];
    uint32_t wcnt[kSpWarps], wkey[kSpWarps];
    uint32_t bin;
    uint32_t above_n;
    u64 above_m;
    int found;
};

template <typename T>
__global__ void __launch_bounds__(kSpThreads) sample_kernel(const SampleArgs a) {
    __shared__ SampleSmem sm;
    pdl_trigger();
    pdl_wait();
    const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T *row = (const T *)a.logits + (size_t)r * a.ld;
    const int V = a.V;
    const float temp = a.temperature ? a.temperature[r] : 1.f, p = a.top_p ? a.top_p[r] : 1.f,
                mp = a.min_p ? a.min_p[r] : 0.f, u = a.uniform[r];
    const int k = a.top_k ? a.top_k[r] : 0;
    if (!(temp >= 0.f && temp <= 1e6f && p >= 0.f && p <= 1.f && mp >= 0.f && mp <= 1.f && u >= 0.f && u < 1.f)) {
        if (tid == 0) raise_err(a.err, ERR_BAD_SAMPLE), a.out[r] = -1;
        return;
    }
    auto key_at = [&](int i) { return sp_key(Elem<T>::to_f(row[i])); };
    // the largest key
    uint32_t top = 0;
    for (int i = tid; i < V; i += kSpThreads) top = max(top, key_at(i));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) sm.wkey[warp] = top;
    if (tid == 0) sm.found = -1;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, sm.wkey[lane]);
    if (top <= sp_key(-INFINITY)) {  // nothing but -inf and NaN
        if (tid == 0) a.out[r] = -1;
        return;
    }
    const double inv_t = temp > 0.f ? 1.0 / (double)temp : 0.0;
    uint32_t cut = 0;             // kept: keys above cut, and the first `ties` of those equal to it
    uint32_t ties = 0xffffffffu;
    if (temp == 0.f) {
        cut = top, ties = 1;
    } else {
        // one round of a radix selection: the histogram of 8 key bits of the
        // keys above `floor_key` with the prefix chosen so far, from the top
        // bin down to where the count (or mass) reaches what is wanted
        auto select = [&](bool by_mass, u64 want, uint32_t floor_key, uint32_t *got, u64 *left) {
            uint32_t prefix = 0;
            for (int shift = 24; shift >= 0; shift -= 8) {
                if (tid < 256) sm.mass[tid] = 0, sm.count[tid] = 0;
                __syncthreads();
                for (int i = tid; i < V; i += kSpThreads) {
                    const uint32_t key = key_at(i);
                    if (key <= floor_key || (shift < 24 && (key >> (shift + 8)) != (prefix >> (shift + 8)))) continue;
                    const uint32_t b = (key >> shift) & 255u;
                    if (by_mass) {
                        const u64 w = sp_weight(key, top, inv_t);
                        if (w) atomicAdd(&sm.mass[b], w);
                    } else {
                        atomicAdd(&sm.count[b], 1u);
                    }
                }
                __syncthreads();
                if (tid == 0) {
                    int b = 255;
                    for (; b > 0; --b) {
                        const u64 x = by_mass ? sm.mass[b] : (u64)sm.count[b];
                        if (x >= want) break;
                        want -= x;
                    }
                    sm.bin = b;
                    sm.above_m = want;
                }
                __syncthreads();
                prefix |= sm.bin << shift;
                want = sm.above_m;
                __syncthreads();
            }
            *got = prefix;
            *left = want;  // of the keys equal to *got
        };
        if (k > 0 && k < V) {
            u64 left;
            select(false, (u64)k, 0u, &cut, &left);
            ties = (uint32_t)left;
        }
        if (p < 1.f) {
            // masses of the keys above the cut, and of the kept ones equal to it
            u64 s = 0;
            uint32_t c = 0;
            for (int i = tid; i < V; i += kSpThreads) {
                const uint32_t key = key_at(i);
                if (key > cut) s += sp_weight(key, top, inv_t);
                c += key == cut;
            }
            s = warp_add(s), c = warp_add(c);
            if (lane == 0) sm.wsum[warp] = s, sm.wcnt[warp] = c;
            __syncthreads();
            s = warp_add(sm.wsum[lane]), c = warp_add(sm.wcnt[lane]);
            const u64 wt = cut ? sp_weight(cut, top, inv_t) : 0ull;
            const u64 all = s + wt * min(c, ties);
            const u64 f = frac64(p);
            u64 want = __umul64hi(f, all) + (f * all != 0);
            if (want < 1) want = 1;
            if (want <= s) {
                u64 left;
                uint32_t got;
                select(true, want, cut, &got, &left);
                const u64 w = sp_weight(got, top, inv_t);
                cut = got;
                ties = (uint32_t)((left + w - 1) / w);
            } else if (wt) {
                ties = min(ties, (uint32_t)min((want - s + wt - 1) / wt, (u64)0xffffffffu));
            }
        }
    }
    // the tokens in the order of their ids: a warp takes a contiguous stretch
    const u64 least = temp > 0.f ? (u64)ceil((double)mp * (double)(1ull << kFrac)) : 0ull;
    const int per = ((V + kSpThreads - 1) / kSpThreads) * 32, i0 = warp * per, i1 = min(V, i0 + per);
    uint32_t before = 0;  // keys equal to the cut in front of this stretch
    {
        uint32_t c = 0;
        for (int i = i0 + lane; i < i1; i += 32) c += key_at(i) == cut;
        c = warp_add(c);
        __syncthreads();
        if (lane == 0) sm.wcnt[warp] = c;
        __syncthreads();
        const uint32_t x = lane < warp ? sm.wcnt[lane] : 0u;
        before = warp_add(x);
    }
    // weight of token i (0 if it is not kept); advances the count of ties by the warp's
    auto kept = [&](int i, uint32_t &seen) -> u64 {
        const uint32_t key = i < i1 ? key_at(i) : 0u;
        const bool tie = i < i1 && key == cut;
        const uint32_t mask = __ballot_sync(0xffffffffu, tie);
        const uint32_t rank = seen + __popc(mask & ((1u << lane) - 1u));
        seen += __popc(mask);
        if (i >= i1 || key < cut || (tie && rank >= ties)) return 0ull;
        const u64 w = key == top ? 1ull << kFrac : temp > 0.f ? sp_weight(key, top, inv_t) : 0ull;
        return w >= least ? w : 0ull;
    };
    u64 s = 0;
    uint32_t seen = before;
    for (int b = i0; b < i1; b += 32) s += kept(b + lane, seen);
    s = warp_add(s);
    if (lane == 0) sm.wsum[warp] = s;
    __syncthreads();
    const u64 mine = sm.wsum[lane];
    const u64 all = warp_add(mine), first = warp_add(lane < warp ? mine : 0ull);
    const u64 target = __umul64hi(frac64(u), all);
    if (target >= first && target < first + s) {
        u64 sum = first;
        seen = before;
        for (int b = i0; b < i1; b += 32) {
            const u64 w = kept(b + lane, seen);
            u64 c = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 x = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) c += x;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, sum + c > target);
            if (hit) {
                if (lane == 0) a.out[r] = b + __ffs(hit) - 1;
                break;
            }
            sum += __shfl_sync(0xffffffffu, c, 31);
        }
    }
}

}  // namespace

cudaError_t sample_rows(int dtype_bf16, const void *logits, int64_t ld, int n_rows, int V, const float *temperature,
                        const int32_t *top_k, const float *top_p, const float *min_p, const float *uniform,
                        int32_t *out, unsigned *err, cudaStream_t st) {
    if (n_rows <= 0) return cudaSuccess;
    SampleArgs a{logits, ld, V, temperature, top_p, min_p, uniform, top_k, out, err};
    if (dtype_bf16) return launch_pdl(sample_kernel<bf16>, dim3(n_rows), dim3(kSpThreads), 0, st, a);
    return launch_pdl(sample_kernel<float>, dim3(n_rows), dim3(kSpThreads), 0, st, a);
}

}  // namespace orca
