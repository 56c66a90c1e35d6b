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
constexpr int kClasses = 3;  // column tiles of 8, 16 and 32
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
    G_SMS,
    G_ITEMS,                       // work items by class (8, 16, 32 columns)
    G_PARTS = G_ITEMS + kClasses,  // partial columns of split items (per key/value head)
    G_JOINS,                       // columns whose keys are split
    G_O_ITEMS,                     // 8 words each, class by class, most keys first
    G_O_JOINS,                     // 8 words each
};
constexpr int kCwCtasPerSm = 2;
constexpr int kSplitAt = 256;  // fewest keys of a part

int64_t up4(int64_t x) { return (x + 3) & ~int64_t(3); }

struct PagedSizes {
    int64_t rows, tiles, maxpos, chunk, items[kClasses], parts, joins;
    int64_t off_rows, off_reqs, off_tiles, off_items, off_joins, total;
};

// Columns of a request: the smallest class that holds them all, else tiles of the widest (fp32: 16, by registers).
int class_of(int64_t cols, int dtype) { return cols <= 8 ? 0 : cols <= 16 || !dtype ? 1 : 2; }

// The column tiles of request i: fn(class, first column, columns, keys that the last of them sees).
template <typename F>
void column_tiles(const PagedBatch &b, int i, F fn) {
    const int64_t group = b.n_heads / b.n_kv_heads, cols = b.n_input[i] * group;
    const int cl = class_of(cols, b.dtype);
    for (int64_t c = 0; c < cols; c += 8 << cl) {
        const int64_t n = std::min<int64_t>(8 << cl, cols - c);
        fn(cl, c, n, b.ctx_len[i] + (c + n - 1) / group + 1);
    }
}
// Parts that a tile's keys are cut into.
int64_t parts_of(int64_t keys, int64_t chunk) { return keys * 2 <= chunk * 3 ? 1 : (keys + chunk - 1) / chunk; }

bool paged_sizes(const PagedBatch &b, int num_sms, PagedSizes *z) {
    *z = {};
    int64_t work = 0;
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
        column_tiles(b, i, [&](int, int64_t, int64_t, int64_t keys) { work += keys * b.n_kv_heads; });
        z->tiles += (c + n + 15) / 16;
        z->maxpos = std::max(z->maxpos, c + n);
    }
    // a third of a block's share, so that uneven items even out over the blocks
    const int64_t share = work / ((int64_t)kCwCtasPerSm * num_sms * 3);
    z->chunk = std::max<int64_t>(kSplitAt, (share + 63) / 64 * 64);
    for (int i = 0; i < b.n_req; ++i) {
        if (b.n_input[i] == 0) continue;
        column_tiles(b, i, [&](int cl, int64_t, int64_t n, int64_t keys) {
            const int64_t parts = parts_of(keys, z->chunk);
            z->items[cl] += parts;
            if (parts > 1) z->parts += parts * (8 << cl), z->joins += n;
        });
    }
    int64_t w = kPagedHdr;
    z->off_rows = w, w = up4(w + 4 * z->rows);
    z->off_reqs = w, w = up4(w + b.n_req);
    z->off_tiles = w, w = up4(w + z->tiles);
    const int64_t items = z->items[0] + z->items[1] + z->items[2];
    z->off_items = w, w = up4(w + 8 * items);
    z->off_joins = w, w = up4(w + 8 * z->joins);
    z->total = w;
    // 32-bit table entries and grid sizes
    return w <= INT32_MAX && z->rows * b.n_heads <= INT32_MAX && items * b.n_kv_heads <= INT32_MAX / 2 &&
           z->parts <= INT32_MAX && z->joins * b.n_kv_heads <= INT32_MAX;
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
    PagedSizes z;
    return paged_sizes(b, num_sms, &z) ? z.total : -1;
}

bool paged_plan_build(const PagedBatch &b, int num_sms, int32_t *buf, int64_t cap) {
    PagedSizes z;
    if (!paged_sizes(b, num_sms, &z) || cap < z.total) return false;
    const bool twice = writes_twice(b);
    std::memset(buf, 0, sizeof(int32_t) * (size_t)z.total);
    int32_t *row = buf + z.off_rows, *req = buf + z.off_reqs, *tile = buf + z.off_tiles;
    const int32_t per_page = b.page_size / 16;
    int32_t *item[kClasses], *join = buf + z.off_joins;
    item[0] = buf + z.off_items;
    for (int c = 1; c < kClasses; ++c) item[c] = item[c - 1] + 8 * z.items[c - 1];
    int64_t part = 0, first_row = 0;
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
        column_tiles(b, i, [&](int cl, int64_t col, int64_t cols, int64_t keys) {
            const int64_t parts = parts_of(keys, z.chunk), per = parts == 1 ? keys : z.chunk;
            for (int64_t p = 0; p < parts; ++p, item[cl] += 8) {
                int32_t *r = item[cl];
                r[0] = req[i] + (int32_t)(p * per / 16);
                r[1] = (int32_t)std::min<int64_t>(per, keys - p * per);
                r[2] = (int32_t)first_row;
                r[3] = (int32_t)col;
                r[4] = (int32_t)cols;
                r[5] = (int32_t)(c - p * per);
                r[6] = parts == 1 ? -1 : (int32_t)(part + p * (8 << cl));
            }
            for (int64_t x = 0; parts > 1 && x < cols; ++x, join += 8) {
                join[0] = (int32_t)first_row;
                join[1] = (int32_t)(col + x);
                join[2] = (int32_t)parts;
                join[3] = (int32_t)part;
                join[4] = 8 << cl;
                join[5] = (int32_t)x;
            }
            if (parts > 1) part += parts * (8 << cl);
        });
        first_row += n;
    }
    struct Rec {
        int32_t w[8];
    };
    Rec *rec = reinterpret_cast<Rec *>(buf + z.off_items);
    for (int c = 0; c < kClasses; rec += z.items[c], ++c)
        std::stable_sort(rec, rec + z.items[c], [](const Rec &x, const Rec &y) { return x.w[1] > y.w[1]; });
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
    buf[G_SMS] = num_sms;
    for (int c = 0; c < kClasses; ++c) buf[G_ITEMS + c] = (int32_t)z.items[c];
    buf[G_PARTS] = (int32_t)z.parts;
    buf[G_JOINS] = (int32_t)z.joins;
    buf[G_O_ITEMS] = (int32_t)z.off_items;
    buf[G_O_JOINS] = (int32_t)z.off_joins;
    return true;
}

bool paged_plan_ok(const int32_t *hp) { return hp && hp[0] == kPagedMagic; }
PagedInfo paged_plan_info(const int32_t *hp) {
    return {hp[G_DTYPE], hp[G_HEADS], hp[G_KV_HEADS], hp[G_DIM], hp[G_SLOTS], hp[G_ROWS], hp[G_MAXPOS], hp[G_TWICE] != 0};
}

int64_t paged_workspace_bytes(const int32_t *hp) {
    return (int64_t)hp[G_PARTS] * hp[G_KV_HEADS] * (hp[G_DIM] + 2) * 4;
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
// One product serves all query rows that read the same keys: the heads that
// share a key/value head, and the rows of a request.  A column is such a (row j,
// head g) pair, number j * group + g of its request and key/value head; a work
// item is up to 8 NT columns over a range of keys, times the key/value heads.
// With keys as the first operand's rows the tensor-core products are
//   S^T = K q^T    16 keys x head_dim times head_dim x 8 columns
//   O^T += V^T P   16 components x 16 keys times 16 keys x 8 columns
// so that one query costs a product of 8 columns and 32 queries four, each key
// read from shared memory once for all of them.  The kernel streams keys: one
// query per key/value head is 0.5 flop per byte, 32 are 16, where mma.sync's rate
// is still several times what HBM delivers.
//
// Each warp is a pipeline of its own: it takes every fourth tile of 16 keys of
// the item, loads it by TMA (K and V of a 64-dim block in one box) into its
// own ring of stages several tiles ahead, across items, and keeps its own
// running maximum m, sum l and outputs per column.  At the end of an item the
// block's four warps meet and add up.  No warp waits for another while it
// streams, and nothing is shared between blocks.
namespace {

constexpr int kCwWarps = 4;
constexpr int kCwThreads = 32 * kCwWarps;

struct PagedArgs {
    const void *q;
    void *out;
    float *part, *part_ml;  // partial outputs [column][head_dim], their maxima and sums [column][2]
    const int32_t *plan;
    const int4 *items;  // {tiles at, keys, first row, first column}, {columns, last key of row 0, part or -1, 0}
    int64_t ld_q, ld_out;
    int n_items, kv_heads, group;
    float scale_log2;
    unsigned *err;
};

template <typename T, int D, int NT>
struct CwShape {
    static constexpr int kEs = sizeof(T);
    static constexpr int kRow = D * kEs < 128 ? D * kEs : 128;  // bytes of a box's rows
    static constexpr int kBlocks = D * kEs / kRow;              // boxes across head_dim
    static constexpr uint32_t kBox = 2 * 16 * kRow;             // K and V of 16 keys
    static constexpr uint32_t kStage = kBlocks * kBox;
    static constexpr int kWant = (NT == 1 ? 24576 : 16384) / (int)kStage;
    static constexpr int kStages = kWant < 2 ? 2 : kWant > 8 ? 8 : kWant;
    static constexpr int kMerge = NT < 2 ? 8 : 16;  // columns that meet at a time
    static constexpr int kLd = D + 4;               // floats from column to column (no bank conflicts)
    static constexpr uint32_t kRing = kCwWarps * kStages * kStage;
    static constexpr uint32_t kO = kRing;
    static constexpr uint32_t kMl = kO + kCwWarps * kMerge * kLd * 4;
    static constexpr uint32_t kBars = kMl + kCwWarps * kMerge * 8;
    static constexpr uint32_t kBytes = kBars + kCwWarps * kStages * 8;
};

__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(bf16 *p, float a, float b, float c, float d) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}
__device__ __forceinline__ void cw_tma_load(uint32_t dst, const void *tmap, uint64_t *bar, int c0, int slot, int h,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
        "{%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
        "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(slot), "r"(h), "r"(0), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void cw_ldsm(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void cw_ldsm_t(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void cw_mma_bf16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 16-bit elements over the warp, transposed.
__device__ __forceinline__ uint32_t cw_transpose(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float cw_exp2(float x) {  // (2^-22 relative; 2^-inf = 0)
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t cw_pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// fp32 operands as two tf32 parts of 11 bits each, x = hi + lo up to 2^-22 |x|:
// products hi hi + hi lo + lo hi.  An infinity has no lower part and takes no part
// in the mixed products (0 * inf, inf - inf): they use `fin`.
__device__ __forceinline__ void cw_split(uint32_t x, uint32_t &hi, uint32_t &lo, uint32_t &fin) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "r"(x));
    const float rest = hi == x ? 0.f : __uint_as_float(x) - __uint_as_float(hi);
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
    fin = (hi & 0x7fffffffu) == 0x7f800000u ? 0u : hi;
}
__device__ __forceinline__ void cw_mma_tf32(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t cw_lds(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// exp2(m - new) of a running maximum, and what to subtract from scores: no key seen yet is m = -inf.
__device__ __forceinline__ float cw_base(float m) { return m == -INFINITY ? 0.f : m; }

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kCwThreads, 2)
    paged_cols_kernel(const __grid_constant__ CUtensorMap tm, const PagedArgs a) {
    using S = CwShape<T, D, NT>;
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int KS = D / (F32 ? 8 : 16), MT = D / 16;
    constexpr bool kKeepQ = NT <= 2 && !F32;  // the queries' fragments stay in registers (else they come from L1 every tile)
    constexpr unsigned kFull = 0xffffffffu;
    extern __shared__ __align__(1024) uint8_t cw_smem[];
    pdl_trigger();
    if (smem_u32(cw_smem) & 1023u) {  // uniform: every thread leaves
        if (threadIdx.x == 0) raise_err(a.err, 8u);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
    const uint32_t ring = smem_u32(cw_smem) + (uint32_t)(warp * S::kStages) * S::kStage;
    uint64_t *full = reinterpret_cast<uint64_t *>(cw_smem + S::kBars) + warp * S::kStages;
    float *const mo = reinterpret_cast<float *>(cw_smem + S::kO);
    float2 *const ml = reinterpret_cast<float2 *>(cw_smem + S::kMl);
    if (lane == 0) {
        for (int s = 0; s < S::kStages; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
        if (warp == 0) prefetch_tmap(&tm);
    }
    __syncwarp();
    pdl_wait();

    const int total = a.n_items * a.kv_heads, G = gridDim.x;
    // The block's k-th (item, key/value head): items come longest first, dealt forwards and backwards in turn.
    const auto nth = [&](int k) { return k * G + ((k & 1) ? G - 1 - (int)blockIdx.x : (int)blockIdx.x); };

    // ---- the warp's loads: tile pt of entry nth(pk), lane x holding the slot index of tile pb + 4 x ----
    const uint64_t pol = l2_policy_evict_first();
    int pk = -1, pt = 0, p_tiles = 0, p_at = 0, p_h = 0, pb = 0, p_idx = 0;
    uint32_t issued = 0, used = 0;
    bool more = true, ok = true;
    const auto issue = [&]() {  // the next tile, if there is one, into its stage
        if (!more) return;
        while (pt >= p_tiles) {
            const int e = nth(++pk);
            if (e >= total) {
                more = false;
                return;
            }
            const int4 r = a.items[2 * (e / a.kv_heads)];
            p_h = e % a.kv_heads, p_at = r.x, p_tiles = (r.y + 15) / 16, pt = warp, pb = pt - 128;
        }
        if (pt >= pb + 128) {
            pb = pt;
            const int x = pb + kCwWarps * lane;
            p_idx = x < p_tiles ? a.plan[p_at + x] : 0;
        }
        const int slot = 16 * __shfl_sync(kFull, p_idx, (pt - pb) / kCwWarps);
        const uint32_t s = issued % S::kStages;
        if (lane == 0) {
            mbar_arrive_expect_tx(&full[s], S::kStage);
#pragma unroll
            for (int b = 0; b < S::kBlocks; ++b)
                cw_tma_load(ring + s * S::kStage + b * S::kBox, &tm, &full[s], b * (S::kRow / S::kEs), slot, p_h, pol);
        }
        ++issued;
        pt += kCwWarps;
    };
    for (int s = 0; s < S::kStages; ++s) issue();

    for (int k = 0;; ++k) {
        const int e = nth(k);
        if (e >= total) break;
        const int h = e % a.kv_heads;
        const int4 r0 = a.items[2 * (e / a.kv_heads)], r1 = a.items[2 * (e / a.kv_heads) + 1];
        const int keys = r0.y, n_tiles = (keys + 15) / 16, c0 = r0.w, n_cols = r1.x, last0 = r1.y;
        // keys that the first column sees (the others see more), and this lane's columns 8 nt + 2 t4 + i
        const int first_sees = last0 + c0 / a.group + 1;
        const bool one_row = c0 / a.group == (c0 + n_cols - 1) / a.group;
        int sees[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) sees[nt][i] = last0 + (c0 + 8 * nt + 2 * t4 + i) / a.group + 1;
        // q as the second operand: column g8, components 2 t4 + {0, 1} and + 8 of every 16
        const uint32_t *qp[NT];
        uint32_t qb[NT][kKeepQ ? KS : 1][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int c = c0 + min(8 * nt + g8, n_cols - 1);  // (columns behind the last repeat it and are not written)
            qp[nt] = reinterpret_cast<const uint32_t *>(reinterpret_cast<const T *>(a.q) +
                                                        (int64_t)(r0.z + c / a.group) * a.ld_q +
                                                        (h * a.group + c % a.group) * D) + t4;
            if constexpr (kKeepQ)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) qb[nt][ks][0] = qp[nt][8 * ks], qb[nt][ks][1] = qp[nt][8 * ks + 4];
        }
        float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
        }
        for (int t = warp; t < n_tiles && ok; t += kCwWarps) {
            const uint32_t s = used % S::kStages;
            ok = __all_sync(kFull, mbar_wait_bounded(&full[s], (used / S::kStages) & 1u, a.err));
            if (!ok) break;
            const uint32_t kb = ring + s * S::kStage, vb = kb + 16 * S::kRow;
            // address of 16-byte chunk ch of row r of the box at `base` (swizzled by address bits 7 and up)
            const auto at = [&](uint32_t base, int r, int ch) {
                const uint32_t x = (uint32_t)(ch / (S::kRow / 16)) * S::kBox + (uint32_t)(r * S::kRow);
                const uint32_t swz = S::kRow == 128 ? r & 7 : S::kRow == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
                return base + x + (((uint32_t)(ch % (S::kRow / 16)) ^ swz) << 4);
            };
            float c[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
            if constexpr (F32) {
                // chains of at most four products, added up in fp32: the tensor core cuts its sums off
                constexpr int NC = KS < 4 ? KS : 4;
                float hh[NC][NT][4];
#pragma unroll
                for (int x = 0; x < NC * NT * 4; ++x) (&hh[0][0][0])[x] = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t f[4], fh[4], fl[4], ff[4], qh[2], ql[2], qf[2];
                    cw_ldsm(at(kb, lane & 15, 2 * ks + (lane >> 4)), f);
#pragma unroll
                    for (int x = 0; x < 4; ++x) cw_split(f[x], fh[x], fl[x], ff[x]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        cw_split(qp[nt][8 * ks], qh[0], ql[0], qf[0]);
                        cw_split(qp[nt][8 * ks + 4], qh[1], ql[1], qf[1]);
                        cw_mma_tf32(hh[ks % NC][nt], fh, qh[0], qh[1]);
                        cw_mma_tf32(c[nt], ff, ql[0], ql[1]);
                        cw_mma_tf32(c[nt], fl, qf[0], qf[1]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int n = 0; n < NC; ++n) c[nt][x] += hh[n][nt][x];
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t f[4];
                    cw_ldsm(at(kb, lane & 15, 2 * ks + (lane >> 4)), f);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (kKeepQ)
                            cw_mma_bf16(c[nt], f, qb[nt][ks][0], qb[nt][ks][1]);
                        else
                            cw_mma_bf16(c[nt], f, qp[nt][8 * ks], qp[nt][8 * ks + 4]);
                    }
                }
            }
            // scores of keys 16 t + g8 and + 8, columns 2 t4 and + 1 of every 8; those not seen are -inf
            const bool masked = 16 * t + 16 > first_sees;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    c[nt][x] *= a.scale_log2;
                    if (masked && 16 * t + g8 + 8 * (x >> 1) >= sees[nt][x & 1]) c[nt][x] = -INFINITY;
                }
            float mx[NT][2];
            bool grew = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v = fmaxf(c[nt][i], c[nt][2 + i]);
                    v = fmaxf(v, __shfl_xor_sync(kFull, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(kFull, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(kFull, v, 16));
                    mx[nt][i] = fmaxf(m[nt][i], v);
                    grew |= mx[nt][i] > m[nt][i];
                }
            if (__any_sync(kFull, grew)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float corr = cw_exp2(m[nt][i] - cw_base(mx[nt][i]));
                        m[nt][i] = mx[nt][i];
                        l[nt][i] *= corr;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) o[nt][mt][i] *= corr, o[nt][mt][2 + i] *= corr;
                    }
            }
            // weights; bf16: rounded for the second product, and l sums what is used
            uint32_t pw[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float b0 = cw_base(m[nt][0]), b1 = cw_base(m[nt][1]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    c[nt][2 * x] = cw_exp2(c[nt][2 * x] - b0), c[nt][2 * x + 1] = cw_exp2(c[nt][2 * x + 1] - b1);
                    if constexpr (!F32) {
                        pw[nt][x] = cw_pack(c[nt][2 * x], c[nt][2 * x + 1]);
                        c[nt][2 * x] = __uint_as_float(pw[nt][x] << 16);
                        c[nt][2 * x + 1] = __uint_as_float(pw[nt][x] & 0xffff0000u);
                    }
                    l[nt][0] += c[nt][2 * x], l[nt][1] += c[nt][2 * x + 1];
                }
            }
            bool by_key = false;  // a value that is not finite behind a key that some column does not see
            if (masked) {
                const int rest = keys - 16 * t;  // rows behind the item's last key may hold anything: zero in V
                if (rest < 16) {
                    for (int x = lane; x < (16 - rest) * (D * S::kEs / 16); x += 32) {
                        const uint32_t p = at(vb, rest + x / (D * S::kEs / 16), x % (D * S::kEs / 16));
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(p), "r"(0u) : "memory");
                    }
                    fence_proxy_async_smem();  // before the stage's next load
                    __syncwarp();
                }
                if (!one_row) {
                    for (int x = lane; x < 16 * (D * S::kEs / 4); x += 32) {
                        const int r = x / (D * S::kEs / 4), w = x % (D * S::kEs / 4);
                        const uint32_t v = cw_lds(at(vb, r, w / 4) + 4 * (w % 4));
                        by_key |= (!F32 && (v & 0x7f80u) == 0x7f80u) || (v & 0x7f800000u) == 0x7f800000u;
                    }
                    by_key = __any_sync(kFull, by_key);
                }
            }
            if (by_key) {  // key by key, so that 0 * inf reaches no column that does not see it
                for (int r = 0; r < 16; ++r)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int src = (r & 7) * 4 + t4;
                        const float p[2] = {__shfl_sync(kFull, r < 8 ? c[nt][0] : c[nt][2], src),
                                            __shfl_sync(kFull, r < 8 ? c[nt][1] : c[nt][3], src)};
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int d = (16 * mt + g8 + 8 * x) * S::kEs;  // (byte)
                                const uint32_t v = cw_lds(at(vb, r, d / 16) + d % 16 / 4 * 4);
                                const float vf = __uint_as_float(F32 ? v : d % 4 ? v & 0xffff0000u : v << 16);
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    if (16 * t + r < sees[nt][i]) o[nt][mt][2 * x + i] = fmaf(p[i], vf, o[nt][mt][2 * x + i]);
                            }
                    }
            } else if constexpr (F32) {
                // the keys of a product in the order 0 2 4 6 1 3 5 7, which spreads V's rows over the banks
                uint32_t ph[NT][2][2], pl[NT][2][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int src = (2 * t4 + i) * 4 + (g8 >> 1);
                            const float p0 = __shfl_sync(kFull, c[nt][2 * x], src);
                            const float p1 = __shfl_sync(kFull, c[nt][2 * x + 1], src);
                            uint32_t unused;  // (weights are finite, or their column is NaN)
                            cw_split(__float_as_uint(g8 & 1 ? p1 : p0), ph[nt][x][i], pl[nt][x][i], unused);
                        }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float y[NT][4];  // this tile's sum on its own: o is added to in fp32
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) y[nt][0] = y[nt][1] = y[nt][2] = y[nt][3] = 0.f;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t fh[4], fl[4], ff[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int d = 16 * mt + g8 + 8 * (z & 1);
                            cw_split(cw_lds(at(vb, 8 * x + 2 * t4 + (z >> 1), d / 4) + d % 4 * 4), fh[z], fl[z], ff[z]);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            cw_mma_tf32(y[nt], fl, ph[nt][x][0], ph[nt][x][1]);
                            cw_mma_tf32(y[nt], ff, pl[nt][x][0], pl[nt][x][1]);
                            cw_mma_tf32(y[nt], fh, ph[nt][x][0], ph[nt][x][1]);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[nt][mt][x] += y[nt][x];
                }
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) pw[nt][0] = cw_transpose(pw[nt][0]), pw[nt][1] = cw_transpose(pw[nt][1]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t f[4];
                    cw_ldsm_t(at(vb, (lane >> 4) * 8 + (lane & 7), 2 * mt + ((lane >> 3) & 1)), f);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) cw_mma_bf16(o[nt][mt], f, pw[nt][0], pw[nt][1]);
                }
            }
            __syncwarp();  // every lane has read the stage
            ++used;
            issue();
        }
        // ---- the four warps of the block meet: kMerge columns at a time ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[nt][i] += __shfl_xor_sync(kFull, l[nt][i], 4);
                l[nt][i] += __shfl_xor_sync(kFull, l[nt][i], 8);
                l[nt][i] += __shfl_xor_sync(kFull, l[nt][i], 16);
            }
        constexpr int kPer = S::kMerge / 8;
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += kPer) {
            if (8 * n0 >= n_cols) break;
#pragma unroll
            for (int nt = n0; nt < n0 + kPer; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int x = warp * S::kMerge + 8 * (nt - n0) + 2 * t4 + i;
                    if (g8 == 0) ml[x] = make_float2(m[nt][i], l[nt][i]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        mo[x * S::kLd + 16 * mt + g8] = o[nt][mt][i], mo[x * S::kLd + 16 * mt + g8 + 8] = o[nt][mt][2 + i];
                }
            __syncthreads();
            for (int x = threadIdx.x; x < S::kMerge * (D / 4); x += kCwThreads) {
                const int col = x / (D / 4), d = x % (D / 4) * 4;
                if (8 * n0 + col >= n_cols) break;
                float M = -INFINITY, L = 0.f;
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kCwWarps; ++w) M = fmaxf(M, ml[w * S::kMerge + col].x);
                const float base = cw_base(M);
#pragma unroll
                for (int w = 0; w < kCwWarps; ++w) {
                    const float2 v = ml[w * S::kMerge + col];
                    const float4 p = *reinterpret_cast<const float4 *>(&mo[(w * S::kMerge + col) * S::kLd + d]);
                    const float f = cw_exp2(v.x - base);
                    L += v.y * f;
                    O.x += p.x * f, O.y += p.y * f, O.z += p.z * f, O.w += p.w * f;
                }
                if (r1.z < 0) {
                    const int c = c0 + 8 * n0 + col;
                    T *dst = reinterpret_cast<T *>(a.out) + (int64_t)(r0.z + c / a.group) * a.ld_out +
                             (h * a.group + c % a.group) * D + d;
                    const float f = 1.f / L;
                    store4(dst, O.x * f, O.y * f, O.z * f, O.w * f);
                } else {
                    const int64_t at = (int64_t)r1.z * a.kv_heads + h * (8 * NT) + 8 * n0 + col;
                    *reinterpret_cast<float4 *>(a.part + at * D + d) = O;
                    if (d == 0) *reinterpret_cast<float2 *>(a.part_ml + at * 2) = make_float2(M, L);
                }
            }
            __syncthreads();  // the buffers are free again
        }
    }
    // a wait that gave up: the copies in flight land before the block ends
    for (; used < issued; ++used) mbar_wait_bounded(&full[used % S::kStages], (used / S::kStages) & 1u, a.err);
}

// Split keys: the parts of a column, in their order.  One block per (column,
// key/value head); 4 components per thread, the parts dealt to the thread groups.
struct JoinArgs {
    const float *part, *part_ml;
    const int4 *joins;  // {first row, column of the request, parts, first part}, {columns from part to part, column there, 0, 0}
    void *out;
    int64_t ld_out;
    int kv_heads, group;
};
template <typename T, int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const JoinArgs a) {
    constexpr int L4 = D / 4, N = 128 / L4;  // thread groups
    __shared__ float4 so[N][L4];
    __shared__ float2 sml[N];
    pdl_trigger();
    pdl_wait();
    const int j = blockIdx.x / a.kv_heads, h = blockIdx.x % a.kv_heads;
    const int4 r0 = a.joins[2 * j], r1 = a.joins[2 * j + 1];
    const int grp = threadIdx.x / L4, d = threadIdx.x % L4;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add = [&](float m2, float l2, const float4 &o2) {
        const float mx = fmaxf(m, m2), base = cw_base(mx), f = cw_exp2(m - base), f2 = cw_exp2(m2 - base);
        l = l * f + l2 * f2, m = mx;
        o.x = o.x * f + o2.x * f2, o.y = o.y * f + o2.y * f2, o.z = o.z * f + o2.z * f2, o.w = o.w * f + o2.w * f2;
    };
#pragma unroll 4
    for (int p = grp; p < r0.z; p += N) {
        const int64_t at = (int64_t)(r0.w + p * r1.x) * a.kv_heads + h * r1.x + r1.y;
        const float2 v = *reinterpret_cast<const float2 *>(a.part_ml + 2 * at);
        add(v.x, v.y, *reinterpret_cast<const float4 *>(a.part + at * D + 4 * d));
    }
    so[grp][d] = o;
    if (d == 0) sml[grp] = make_float2(m, l);
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int x = 1; x < N; ++x) add(sml[x].x, sml[x].y, so[x][d]);
    T *dst = reinterpret_cast<T *>(a.out) + (int64_t)(r0.x + r0.y / a.group) * a.ld_out +
             (h * a.group + r0.y % a.group) * D + 4 * d;
    const float f = 1.f / l;
    store4(dst, o.x * f, o.y * f, o.z * f, o.w * f);
}

template <typename T, int D, int NT>
cudaError_t launch_cols(const PagedArgs &a, const void *layer, int64_t slots, int sms, cudaStream_t st) {
    using S = CwShape<T, D, NT>;
    const cudaError_t e = max_smem_once((const void *)paged_cols_kernel<T, D, NT>, (int)S::kBytes);
    if (e != cudaSuccess) return e;
    CUtensorMap tm;  // the layer as [K|V][head][slot][component]
    const uint64_t row = D * sizeof(T);
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)slots, (uint64_t)a.kv_heads, 2};
    const uint64_t strides[3] = {row, row * (uint64_t)slots, row * (uint64_t)slots * (uint64_t)a.kv_heads};
    const uint32_t box[4] = {(uint32_t)(S::kRow / S::kEs), 16, 1, 2};
    if (!encode_tensor_map(&tm, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
                           layer, dims, strides, box,
                           S::kRow == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                           : S::kRow == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_32B))
        return cudaErrorInvalidValue;
    const int64_t total = (int64_t)a.n_items * a.kv_heads;
    const int grid = (int)std::min<int64_t>(total, (int64_t)kCwCtasPerSm * sms);
    return launch_pdl(paged_cols_kernel<T, D, NT>, dim3((unsigned)grid), dim3(kCwThreads), S::kBytes, st, tm, a);
}

template <typename T, int D>
cudaError_t launch_attention(const PagedAttn &p, const int32_t *hp, const int32_t *dp, unsigned *err, int *launches,
                             cudaStream_t st) {
    const float scale_log2 = p.scale * 1.4426950408889634f;
    PagedArgs a;
    a.q = p.q, a.out = p.out, a.ld_q = p.ld_q, a.ld_out = p.ld_out, a.plan = dp, a.err = err;
    a.kv_heads = hp[G_KV_HEADS], a.group = hp[G_HEADS] / hp[G_KV_HEADS], a.scale_log2 = p.scale * 1.4426950408889634f;
    a.part = reinterpret_cast<float *>(p.workspace);
    a.part_ml = a.part + (int64_t)hp[G_PARTS] * a.kv_heads * D;
    *launches = 0;
    cudaError_t e = cudaSuccess;
    const int32_t *at = dp + hp[G_O_ITEMS];
    for (int c = 0; c < kClasses && e == cudaSuccess; ++c) {
        a.items = reinterpret_cast<const int4 *>(at), a.n_items = hp[G_ITEMS + c];
        at += 8 * (int64_t)a.n_items;
        if (!a.n_items) continue;
        ++*launches;
        if (c == 0)
            e = launch_cols<T, D, 1>(a, p.layer, hp[G_SLOTS], hp[G_SMS], st);
        else if (c == 1)
            e = launch_cols<T, D, 2>(a, p.layer, hp[G_SLOTS], hp[G_SMS], st);
        else if constexpr (sizeof(T) == 2)  // (an fp32 plan has no tiles of 32)
            e = launch_cols<T, D, 4>(a, p.layer, hp[G_SLOTS], hp[G_SMS], st);
    }
    if (e != cudaSuccess || !hp[G_JOINS]) return e;
    ++*launches;
    const JoinArgs j = {a.part, a.part_ml, reinterpret_cast<const int4 *>(dp + hp[G_O_JOINS]), p.out, p.ld_out,
                        a.kv_heads, a.group};
    return launch_pdl(paged_join_kernel<T, D>, dim3((unsigned)hp[G_JOINS] * a.kv_heads), dim3(128), 0, st, j);
}

}  // namespace

cudaError_t paged_attention(const PagedAttn &p, const int32_t *hp, const int32_t *dp, unsigned *err, int *launches,
                            cudaStream_t st) {
    const auto go = [&](auto t) -> cudaError_t {
        using T = decltype(t);
        switch (hp[G_DIM]) {
            case 16: return launch_attention<T, 16>(p, hp, dp, err, launches, st);
            case 32: return launch_attention<T, 32>(p, hp, dp, err, launches, st);
            case 64: return launch_attention<T, 64>(p, hp, dp, err, launches, st);
            default: return launch_attention<T, 128>(p, hp, dp, err, launches, st);
        }
    };
    return hp[G_DTYPE] ? go(bf16()) : go(float());
}

}  // namespace orca
