// Paged K/V cache: append with the rotation of positions, and attention over
// the pages.
//
// A layer is [K|V][kv_head][slot][head_dim], the layout of the engine's pool,
// its slots cut into pages of page_size (a multiple of 16) slots.  Position t of
// request i lies in slot table[i][t / page_size] * page_size + t % page_size.  The
// plan turns the page table into one index for every 16 positions (the slot of
// the first divided by 16), so that no kernel divides by the page size and a
// tile of 16 keys never crosses a page.
#include <algorithm>
#include <cstring>
#include <vector>

#include "common.cuh"
#include "kernels.cuh"

namespace orca {

namespace {

constexpr int32_t kPagedMagic = 0x50474B56;
constexpr int kPagedHdr = 64;
enum {  // header words of a plan
    G_MAGIC,
    G_DTYPE,
    G_HEADS,
    G_KV_HEADS,
    G_DIM,
    G_SLOTS,
    G_ROWS,
    G_MAXPOS,  // positions of the batch: the largest ctx + n
    G_TWICE,
    G_TOTAL,
    G_O_ROWS,   // per row: slot, position, request, 0
    G_O_REQS,   // per request with rows: its first tile
    G_O_TILES,  // slot / 16 of every 16 positions
};

int64_t up4(int64_t x) { return (x + 3) & ~int64_t(3); }

struct PagedSizes {
    int64_t rows, tiles, keys, maxpos, off_rows, off_reqs, off_tiles, total;
};

bool paged_sizes(const PagedBatch &b, PagedSizes *z) {
    *z = {};
    const int64_t slots = b.n_pages * b.page_size;
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t n = b.n_input[i], c = b.ctx_len[i];
        if (n < 0) return false;
        if (n == 0) continue;  // takes no part
        if (c < 0 || c + n > slots || (c + n + b.page_size - 1) / b.page_size > b.table_ld) return false;
        const int32_t *t = b.page_table + (int64_t)i * b.table_ld;
        for (int64_t p = 0; p * b.page_size < c + n; ++p)
            if (t[p] < 0 || t[p] >= b.n_pages) return false;
        z->rows += n;
        z->keys += c + n;
        z->tiles += (c + n + 15) / 16;
        z->maxpos = std::max(z->maxpos, c + n);
    }
    int64_t w = kPagedHdr;
    z->off_rows = w, w = up4(w + 4 * z->rows);
    z->off_reqs = w, w = up4(w + b.n_req);
    z->off_tiles = w, w = up4(w + z->tiles);
    z->total = w;
    return w <= INT32_MAX && z->rows * b.n_heads <= INT32_MAX;  // 32-bit table entries and grid sizes
}

// Whether two rows of the batch are written to one slot.
bool writes_twice(const PagedBatch &b) {
    struct Range {
        int64_t first, end;
    };
    std::vector<Range> w;
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t c = b.ctx_len[i], end = c + b.n_input[i];
        if (b.n_input[i] == 0) continue;
        const int32_t *t = b.page_table + (int64_t)i * b.table_ld;
        for (int64_t at = c; at < end;) {
            const int64_t p = at / b.page_size, stop = std::min(end, (p + 1) * b.page_size);
            const int64_t base = ((int64_t)t[p] - p) * b.page_size;
            w.push_back({base + at, base + stop});
            at = stop;
        }
    }
    std::sort(w.begin(), w.end(), [](const Range &x, const Range &y) { return x.first < y.first; });
    for (size_t i = 1; i < w.size(); ++i)
        if (w[i].first < w[i - 1].end) return true;
    return false;
}

}  // namespace

int64_t paged_plan_words(const PagedBatch &b, int num_sms) {
    (void)num_sms;
    PagedSizes z;
    return paged_sizes(b, &z) ? z.total : -1;
}

bool paged_plan_build(const PagedBatch &b, int num_sms, int32_t *buf, int64_t cap) {
    (void)num_sms;
    PagedSizes z;
    if (!paged_sizes(b, &z) || cap < z.total) return false;
    const bool twice = writes_twice(b);
    std::memset(buf, 0, sizeof(int32_t) * (size_t)z.total);
    int32_t *row = buf + z.off_rows, *req = buf + z.off_reqs, *tile = buf + z.off_tiles;
    const int32_t per_page = b.page_size / 16;
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t n = b.n_input[i], c = b.ctx_len[i];
        if (n == 0) continue;
        const int32_t *t = b.page_table + (int64_t)i * b.table_ld;
        req[i] = (int32_t)(tile - buf);
        for (int64_t at = 0; at < c + n; at += 16)
            *tile++ = t[at / b.page_size] * per_page + (int32_t)(at % b.page_size) / 16;
        const int32_t *mine = buf + req[i];
        for (int64_t j = 0; j < n; ++j, row += 4) {
            const int64_t pos = c + j;
            row[0] = mine[pos / 16] * 16 + (int32_t)(pos % 16);
            row[1] = (int32_t)pos;
            row[2] = i;
        }
    }
    buf[G_MAGIC] = kPagedMagic;
    buf[G_DTYPE] = b.dtype;
    buf[G_HEADS] = b.n_heads;
    buf[G_KV_HEADS] = b.n_kv_heads;
    buf[G_DIM] = b.head_dim;
    buf[G_SLOTS] = (int32_t)(b.n_pages * b.page_size);
    buf[G_ROWS] = (int32_t)z.rows;
    buf[G_MAXPOS] = (int32_t)z.maxpos;
    buf[G_TWICE] = twice;
    buf[G_TOTAL] = (int32_t)z.total;
    buf[G_O_ROWS] = (int32_t)z.off_rows;
    buf[G_O_REQS] = (int32_t)z.off_reqs;
    buf[G_O_TILES] = (int32_t)z.off_tiles;
    return true;
}

bool paged_plan_ok(const int32_t *hp) { return hp && hp[0] == kPagedMagic; }
PagedInfo paged_plan_info(const int32_t *hp) {
    return {hp[G_DTYPE], hp[G_HEADS], hp[G_KV_HEADS], hp[G_DIM], hp[G_SLOTS], hp[G_ROWS], hp[G_MAXPOS], hp[G_TWICE] != 0};
}

int64_t paged_workspace_bytes(const int32_t *hp) {
    (void)hp;
    return 0;
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
namespace {

struct AppendArgs {
    const void *qkv;
    void *layer, *q_out;  // q_out null: queries are left alone
    const float *rope;    // [position][rot]: rot / 2 cosines, rot / 2 sines
    const int4 *rows;     // slot, position
    int64_t ld_qkv, ld_q, slots;
    int n_rows, heads, kv_heads, rot, first_head;  // (first_head: heads are worked on from there)
};

// One thread per two 16-byte chunks of a head's row.
// NEIGH: components 2i and 2i + 1 are a pair; else i and i + rot / 2.
// A thread reads all that it and its pairs need before it writes, so q_out may
// be the queries' own place.
template <typename T, int D, bool NEIGH>
__global__ void __launch_bounds__(256) paged_append_kernel(const AppendArgs a) {
    constexpr int VEC = Elem<T>::kPer16;
    constexpr int U = D / VEC / 2;  // units of a head
    pdl_trigger();
    pdl_wait();
    const int per_row = (a.heads + 2 * a.kv_heads - a.first_head) * U;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int row = (int)(at / per_row);
    if (row >= a.n_rows) return;
    const int rest = (int)(at - (int64_t)row * per_row);
    const int h = a.first_head + rest / U, u = rest % U;
    const int4 rec = a.rows[row];
    const T *src = reinterpret_cast<const T *>(a.qkv) + (int64_t)row * a.ld_qkv + h * D;
    const bool turns = a.rot > 0 && h < a.heads + a.kv_heads;
    const int half = a.rot / 2;
    int c0 = 2 * u * VEC, c1 = c0 + VEC;  // the unit's components
    if (!NEIGH && turns && u * VEC < half) c0 = u * VEC, c1 = c0 + half;
    float x[VEC], y[VEC];
    load16(src + c0, x);
    load16(src + c1, y);
    if (turns) {
        const float *cs = a.rope + (int64_t)rec.y * a.rot;
        if (NEIGH) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                if (c0 + e < a.rot) {
                    const float c = cs[(c0 + e) / 2], s = cs[half + (c0 + e) / 2], p = x[e], q = x[e + 1];
                    x[e] = p * c - q * s, x[e + 1] = q * c + p * s;
                }
                if (c1 + e < a.rot) {
                    const float c = cs[(c1 + e) / 2], s = cs[half + (c1 + e) / 2], p = y[e], q = y[e + 1];
                    y[e] = p * c - q * s, y[e + 1] = q * c + p * s;
                }
            }
        } else if (u * VEC < half) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float c = cs[c0 + e], s = cs[half + c0 + e], p = x[e], q = y[e];
                x[e] = p * c - q * s, y[e] = q * c + p * s;
            }
        }
    }
    T *dst;
    if (h < a.heads)
        dst = reinterpret_cast<T *>(a.q_out) + (int64_t)row * a.ld_q + h * D;
    else  // key heads, then value heads: the layer's planes in this order
        dst = reinterpret_cast<T *>(a.layer) + ((int64_t)(h - a.heads) * a.slots + rec.x) * D;
    store16(dst + c0, x);
    store16(dst + c1, y);
}

// Halves whose middle is inside a 16-byte chunk: a warp per head's row, a
// component's partner loaded on its own.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_append_odd_kernel(const AppendArgs a) {
    constexpr int N = (D + 31) / 32;
    pdl_trigger();
    pdl_wait();
    const int per_row = a.heads + 2 * a.kv_heads - a.first_head;
    const int64_t at = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    const int row = (int)(at / per_row), lane = threadIdx.x & 31;
    if (row >= a.n_rows) return;
    const int h = a.first_head + (int)(at - (int64_t)row * per_row);
    const int4 rec = a.rows[row];
    const T *src = reinterpret_cast<const T *>(a.qkv) + (int64_t)row * a.ld_qkv + h * D;
    const float *cs = a.rope + (int64_t)rec.y * a.rot;
    const int half = a.rot / 2;
    T *dst;
    if (h < a.heads)
        dst = reinterpret_cast<T *>(a.q_out) + (int64_t)row * a.ld_q + h * D;
    else
        dst = reinterpret_cast<T *>(a.layer) + ((int64_t)(h - a.heads) * a.slots + rec.x) * D;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        if (e >= D) continue;
        x[i] = Elem<T>::to_f(src[e]);
        if (h < a.heads + a.kv_heads && e < a.rot) {
            const float c = cs[e % half], s = cs[half + e % half];
            const float o = Elem<T>::to_f(src[e < half ? e + half : e - half]);
            x[i] = e < half ? x[i] * c - o * s : x[i] * c + o * s;
        }
    }
    __syncwarp();  // the whole head is read before any of it is written
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane + 32 * i < D) dst[lane + 32 * i] = Elem<T>::from_f(x[i]);
}

template <typename T, int D>
cudaError_t launch_append(const AppendArgs &a, bool neighbours, cudaStream_t st) {
    constexpr int VEC = Elem<T>::kPer16;
    const int64_t heads = (int64_t)a.n_rows * (a.heads + 2 * a.kv_heads - a.first_head);
    const dim3 grid((unsigned)((heads * (D / VEC / 2) + 255) / 256));
    if (neighbours) return launch_pdl(paged_append_kernel<T, D, true>, grid, dim3(256), 0, st, a);
    if ((a.rot / 2) % VEC == 0) return launch_pdl(paged_append_kernel<T, D, false>, grid, dim3(256), 0, st, a);
    return launch_pdl(paged_append_odd_kernel<T, D>, dim3((unsigned)((heads + 7) / 8)), dim3(256), 0, st, a);
}

}  // namespace

cudaError_t paged_append(const PagedAppend &p, const int32_t *hp, const int32_t *dp, cudaStream_t st) {
    AppendArgs a;
    a.qkv = p.qkv, a.layer = p.layer, a.q_out = p.q_out, a.rope = p.rope;
    a.rows = reinterpret_cast<const int4 *>(dp + hp[G_O_ROWS]);
    a.ld_qkv = p.ld_qkv, a.ld_q = p.ld_q, a.slots = hp[G_SLOTS];
    a.n_rows = hp[G_ROWS], a.heads = hp[G_HEADS], a.kv_heads = hp[G_KV_HEADS], a.rot = p.rot;
    a.first_head = p.q_out ? 0 : a.heads;
    const auto go = [&](auto t) -> cudaError_t {
        using T = decltype(t);
        switch (hp[G_DIM]) {
            case 16: return launch_append<T, 16>(a, p.neighbours, st);
            case 32: return launch_append<T, 32>(a, p.neighbours, st);
            case 64: return launch_append<T, 64>(a, p.neighbours, st);
            default: return launch_append<T, 128>(a, p.neighbours, st);
        }
    };
    return hp[G_DTYPE] ? go(bf16()) : go(float());
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
namespace {

struct PagedArgs {
    const void *q, *layer;
    void *out;
    int64_t ld_q, ld_out, slots;
    const int32_t *plan;
    const int4 *rows;
    const int32_t *reqs;
    int n_rows, heads, kv_heads;
    float scale_log2;
};

// One warp per row and head: LPT lanes hold a key's components, 32 / LPT keys at
// a time, the running maximum m and sum l of the softmax in each lane group.
template <typename T, int D>
__global__ void __launch_bounds__(128) paged_attn_kernel(const PagedArgs a) {
    constexpr int VEC = Elem<T>::kPer16;
    constexpr int LPT = D / VEC, TPW = 32 / LPT;
    pdl_trigger();
    pdl_wait();
    const int at = blockIdx.x * 4 + threadIdx.x / 32, lane = threadIdx.x & 31;
    const int row = at / a.heads, h = at % a.heads;
    if (row >= a.n_rows) return;
    const int4 rec = a.rows[row];
    const int32_t *tiles = a.plan + a.reqs[rec.z];
    const int keys = rec.y + 1, g = lane / LPT, sub = lane % LPT;
    const int64_t kvh = h / (a.heads / a.kv_heads);
    const T *kb = reinterpret_cast<const T *>(a.layer) + kvh * a.slots * D + sub * VEC;
    const T *vb = kb + a.kv_heads * a.slots * D;
    float q[VEC], o[VEC], m = -INFINITY, l = 0.f;
    load16(reinterpret_cast<const T *>(a.q) + row * a.ld_q + h * D + sub * VEC, q);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = 0.f;
    for (int t0 = 0; t0 < keys; t0 += TPW) {  // (uniform across the warp)
        const int t = t0 + g;
        const bool valid = t < keys;
        float k[VEC], v[VEC], s = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) k[e] = v[e] = 0.f;
        if (valid) {
            const int64_t slot = (int64_t)tiles[t / 16] * 16 + t % 16;
            load16(kb + slot * D, k);
            load16(vb + slot * D, v);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
        for (int x = LPT / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s = valid ? s * a.scale_log2 : -INFINITY;
        const float mx = fmaxf(m, s), base = mx == -INFINITY ? 0.f : mx;
        const float corr = exp2f(m - base), p = exp2f(s - base);
        l = l * corr + p;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = fmaf(p, v[e], o[e] * corr);
        m = mx;
    }
#pragma unroll
    for (int x = LPT; x < 32; x <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, x), l2 = __shfl_xor_sync(0xffffffffu, l, x);
        const float mx = fmaxf(m, m2), base = mx == -INFINITY ? 0.f : mx;
        const float c1 = exp2f(m - base), c2 = exp2f(m2 - base);
        l = l * c1 + l2 * c2;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = o[e] * c1 + __shfl_xor_sync(0xffffffffu, o[e], x) * c2;
        m = mx;
    }
    if (g == 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] /= l;
        store16(reinterpret_cast<T *>(a.out) + row * a.ld_out + h * D + sub * VEC, o);
    }
}

}  // namespace

cudaError_t paged_attention(const PagedAttn &p, const int32_t *hp, const int32_t *dp, unsigned *err, int *launches,
                            cudaStream_t st) {
    (void)err;
    PagedArgs a;
    a.q = p.q, a.layer = p.layer, a.out = p.out, a.ld_q = p.ld_q, a.ld_out = p.ld_out;
    a.plan = dp, a.rows = reinterpret_cast<const int4 *>(dp + hp[G_O_ROWS]), a.reqs = dp + hp[G_O_REQS];
    a.slots = hp[G_SLOTS], a.n_rows = hp[G_ROWS], a.heads = hp[G_HEADS], a.kv_heads = hp[G_KV_HEADS];
    a.scale_log2 = p.scale * 1.4426950408889634f;
    *launches = 1;
    const auto go = [&](auto t) -> cudaError_t {
        using T = decltype(t);
        const dim3 grid((unsigned)(((int64_t)a.n_rows * a.heads + 3) / 4));
        switch (hp[G_DIM]) {
            case 16: return launch_pdl(paged_attn_kernel<T, 16>, grid, dim3(128), 0, st, a);
            case 32: return launch_pdl(paged_attn_kernel<T, 32>, grid, dim3(128), 0, st, a);
            case 64: return launch_pdl(paged_attn_kernel<T, 64>, grid, dim3(128), 0, st, a);
            default: return launch_pdl(paged_attn_kernel<T, 128>, grid, dim3(128), 0, st, a);
        }
    };
    return hp[G_DTYPE] ? go(bf16()) : go(float());
}

}  // namespace orca
