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
#include <cmath>
#include <cstring>
#include <functional>
#include <numeric>
#include <type_traits>
#include <utility>
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
    G_O_ROWS,   // per row: slot, position, 0, 0
    G_O_REQS,   // per request with rows: its first tile (for who reads a plan; the items have their own)
    G_O_TILES,  // slot / 16 of every 16 positions (each request at a multiple of four)
    G_SMS,
    G_ITEMS,                       // work items by class (8, 16, 32 columns)
    G_PARTS = G_ITEMS + kClasses,  // partial columns of split items (per key/value head)
    G_JOINS,                       // column tiles whose keys are split
    G_JOINROWS,                    // blocks that one takes per key/value head, at most
    G_O_ITEMS,                     // 8 words each, class by class, most keys first
    G_O_JOINS,                     // 8 words each
    G_PITEMS,                      // the same for prompts: pairs of row tiles
    G_PPARTS,
    G_PJOINS,
    G_PJOINROWS,
    G_O_PITEMS,
    G_O_PJOINS,
    G_PACK,  // heads of a prompt's row tile
    G_BOX,   // slots that one load of a prompt's keys may take
    G_O_DEAL,  // per block its first entry, then the entries: item * tile heads + tile head
};
constexpr int kCwCtasPerSm = 2;
constexpr int kManyParts = 16;  // parts of a column from which on a block joins it alone

int64_t up4(int64_t x) { return (x + 3) & ~int64_t(3); }

struct PagedSizes {
    int64_t rows, tiles, maxpos, chunk, items[kClasses], parts, joins, join_rows;
    int64_t pchunk, pitems, pparts, pjoins, pjoin_rows;
    int64_t off_rows, off_reqs, off_tiles, off_items, off_joins, off_pitems, off_pjoins, off_deal, total;
    int64_t blocks;  // of paged_prompt_kernel
};

// Prompts: rows x heads of one key/value head as the 128 rows of a tensor-core tile; two tiles share their keys, 64 at
// a time.
constexpr int kPpRows = 128, kPpKeys = 64;
constexpr int kPromptExtra = 3;  // what an item takes beside its keys, in key tiles
// Heads in a tile: all that share a key/value head, or one where they are too many to fill 128 rows well.
int pack_of(int group) { return group <= 64 ? group : 1; }

// How requests are attended: classes 0 to 2 as column tiles of 8, 16 and 32, kClasses as prompts.  A request is in the
// narrowest class that holds all its columns (rows x heads of a key/value head; fp32: 16 at most, by registers).
// Prompts (bf16, head_dim 64 and 128): above 16 columns (4 requests of <= 7 rows over <= 500 keys, 32 heads over 8: 9.7
// us, from 65 columns on 11.3; 64 single rows over <= 8000, 40 heads over one: 43 and 70), unless the batch has none
// above 64 columns and more than twice their keys below (9 of <= 5 over <= 1500: 17.5 us, with a launch of prompts 22.7).
// Where heads are tiles of their own, above 32 rows (8 of 1 / 8 rows over <= 1000 keys, 71 heads over one: 11.8 / 18.4
// us, as prompts 40 / 40; <= 110 rows 43, as tiles 78).
// A class goes along with the next wider one of the batch if that has at least as many keys, which saves a launch
// beside another: 9 of <= 7 over <= 1500 17.4 us, each class in its own 22.9; 4 over <= 500 9.7 and 12.6.  Where the
// narrow ones have many keys it is a loss: 64 of <= 7 over <= 3000 94 and 92; 64 single rows over <= 1000 keys beside
// 2000 over 1000, 40 heads over 8, 95 and 89, 32 over 8 86 and 74.  fp32 pays for empty columns in products, so there
// none does: 9 of <= 3 rows 27.9 us, along with one another 32.1.  (Calls among others.)
struct Classes {
    int to[kClasses + 1] = {0, 1, 2, kClasses};
    bool fp32, prompts = false;
    int64_t group;

    int base(int64_t n) const {
        const int64_t cols = n * group;
        if (cols <= 8) return 0;
        if (fp32 || cols <= 16) return 1;
        return prompts && (group <= 64 || n > 32) ? kClasses : 2;
    }
    int of(int64_t n) const { return to[base(n)]; }
    // Up to 16 columns weights have 16 bits, whatever the request goes along with.
    bool narrow(int64_t n) const { return n * group <= 16; }

    explicit Classes(const PagedBatch &b) : fp32(!b.dtype), group(b.n_heads / b.n_kv_heads) {
        if (fp32) return;
        double keys[kClasses + 1];
        bool sure = false;
        const auto count = [&]() {  // (of a batch whose sizes are not checked yet)
            std::fill(keys, keys + kClasses + 1, 0.);
            for (int i = 0; i < b.n_req; ++i) {
                const double n = b.n_input[i], cols = n * (double)group;
                if (n <= 0) continue;
                keys[base(b.n_input[i])] += std::ceil(cols / (prompts ? 256 : 32)) * (b.ctx_len[i] + n);
                sure |= cols > 64;
            }
        };
        prompts = b.head_dim >= 64;
        count();
        if (prompts && !sure && 2 * keys[kClasses] < keys[0] + keys[1] + keys[2]) prompts = false, count();
        for (int x = kClasses - 1; x >= 0; --x) {
            int next = x + 1;
            while (next <= kClasses && keys[next] == 0) ++next;
            if (next > kClasses || keys[x] > keys[to[next]]) continue;
            to[x] = to[next], keys[to[x]] += keys[x];
        }
    }
};

// The column tiles of request i: fn(class, first column, columns, keys that the last of them sees).
template <typename F>
void column_tiles(const PagedBatch &b, int i, const Classes &classes, F fn) {
    const int64_t group = classes.group, cols = b.n_input[i] * group;
    const int cl = classes.of(b.n_input[i]);
    for (int64_t c = 0; c < cols; c += 8 << cl) {
        const int64_t n = std::min<int64_t>(8 << cl, cols - c);
        fn(cl, c, n, b.ctx_len[i] + (c + n - 1) / group + 1);
    }
}
// The pairs of row tiles of a prompt: fn(first row, rows, keys that the last of them sees).
template <typename F>
void row_pairs(const PagedBatch &b, int i, F fn) {
    const int64_t per = 2 * (kPpRows / pack_of(b.n_heads / b.n_kv_heads));
    for (int64_t r = 0; r < b.n_input[i]; r += per) {
        const int64_t n = std::min<int64_t>(per, b.n_input[i] - r);
        fn(r, n, b.ctx_len[i] + r + n);
    }
}
// Parts that a tile's keys are cut into.
int64_t parts_of(int64_t keys, int64_t chunk) { return keys * 4 <= chunk * 5 ? 1 : (keys + chunk - 1) / chunk; }

// Keys of a part, in units of 64, by a model of the time: an item takes its units and `extra` more, a block its items
// one after another (the longest first, so that the last start evens out to half of the longest), and parts have to
// be joined.  `units`: the items' keys, each for `heads` heads; a part has `least_units` or more.
int64_t choose_chunk(const std::vector<int32_t> &units, int64_t heads, int64_t blocks, int64_t least_units, double extra,
                     double join, double per_part) {
    int64_t total = 0, most = 1;
    for (const int32_t u : units) total += u * heads, most = std::max<int64_t>(most, u);
    int64_t best = most;
    double least = 0;
    const int64_t cand[] = {most, total / blocks + 1, total / (2 * blocks) + 1, total / (3 * blocks) + 1,
                            total / (6 * blocks) + 1, 48, 40, 32, 28, 24, 20, 16, 14, 12, 10, 8, 6, 4, 3, 2};
    for (const int64_t c : cand) {
        if (c > most || c < least_units) continue;
        int64_t items = 0, parts = 0;
        double cost = 0, longest = 0;
        for (const int32_t u : units) {
            const int64_t p = parts_of(u, c);
            items += p * heads, cost += (double)heads * ((double)u + extra * (double)p);
            longest = std::max(longest, (p == 1 ? u : c) + extra);
            if (p > 1) parts += p * heads;
        }
        double t = items <= blocks ? longest : std::max(longest, cost / (double)blocks + longest / 2);
        if (parts) t += join + per_part * (double)parts;
        if (c == most || t < least) best = c, least = t;
    }
    return best;
}

bool paged_sizes(const PagedBatch &b, int num_sms, PagedSizes *z) {
    *z = {};
    std::vector<int32_t> work, pwork;  // 64 keys each
    const int64_t pack = pack_of(b.n_heads / b.n_kv_heads), vheads = b.n_heads / pack;
    const Classes classes(b);
    // blocks of paged_join_kernel for the columns of a tile
    const auto join_rows = [&](int64_t cols, int64_t parts) {
        const int64_t per = 512 / b.head_dim;
        return parts >= kManyParts ? cols : (cols + per - 1) / per;
    };
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
        if (classes.of(b.n_input[i]) == kClasses)
            row_pairs(b, i, [&](int64_t, int64_t, int64_t keys) { pwork.push_back((int32_t)((keys + 63) / 64)); });
        else
            column_tiles(b, i, classes,
                         [&](int, int64_t, int64_t, int64_t keys) { work.push_back((int32_t)((keys + 63) / 64)); });
        z->tiles += up4((c + n + 15) / 16);
        z->maxpos = std::max(z->maxpos, c + n);
    }
    // a unit's time goes with its bytes (one request over 500 / 2000 keys, 32 heads over 8 of 128: 6.8 / 8.0 us with
    // parts of 256 keys or more, 5.7 / 6.0 of 128; 300 keys, 20 heads of 64: 5.0 whole, 5.8 in parts of 128; replayed)
    const double small = std::min(2.0, 256.0 / (b.head_dim * (b.dtype ? 2 : 4)));
    z->chunk = 64 * choose_chunk(work, b.n_kv_heads, (int64_t)kCwCtasPerSm * num_sms, 2, 4 * small, 2 * small, 0.0);
    z->pchunk = 64 * choose_chunk(pwork, vheads, num_sms, 4, kPromptExtra, 3.0, 0.03);
    for (int i = 0; i < b.n_req; ++i) {
        if (b.n_input[i] == 0) continue;
        if (classes.of(b.n_input[i]) == kClasses) {
            row_pairs(b, i, [&](int64_t, int64_t rows, int64_t keys) {
                const int64_t parts = parts_of(keys, z->pchunk);
                z->pitems += parts;
                if (parts == 1) return;
                z->pparts += parts * 2 * kPpRows, z->pjoins++;
                z->pjoin_rows = std::max(z->pjoin_rows, join_rows(rows * pack, parts));
            });
            continue;
        }
        column_tiles(b, i, classes, [&](int cl, int64_t, int64_t n, int64_t keys) {
            const int64_t parts = parts_of(keys, z->chunk);
            z->items[cl] += parts;
            if (parts == 1) return;
            z->parts += parts * (8 << cl), z->joins++;
            z->join_rows = std::max(z->join_rows, join_rows(n, parts));
        });
    }
    int64_t w = kPagedHdr;
    z->off_rows = w, w = up4(w + 4 * z->rows);
    z->off_reqs = w, w = up4(w + b.n_req);
    z->off_tiles = w, w = up4(w + z->tiles);
    const int64_t items = z->items[0] + z->items[1] + z->items[2];
    z->off_items = w, w = up4(w + 8 * items);
    z->off_joins = w, w = up4(w + 8 * z->joins);
    z->off_pitems = w, w = up4(w + 8 * z->pitems);
    z->off_pjoins = w, w = up4(w + 8 * z->pjoins);
    z->blocks = std::min<int64_t>(z->pitems * vheads, num_sms);
    z->off_deal = w, w = up4(w + z->blocks + 1 + z->pitems * vheads);
    z->total = w;
    // 32-bit table entries and grid sizes
    return w <= INT32_MAX && z->rows * b.n_heads <= INT32_MAX && items * b.n_kv_heads <= INT32_MAX / 2 &&
           z->parts <= INT32_MAX && z->joins * b.n_kv_heads <= INT32_MAX && z->pitems * vheads <= INT32_MAX / 2 &&
           z->pparts <= INT32_MAX && z->pjoins * vheads <= INT32_MAX;
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
    const Classes classes(b);
    std::memset(buf, 0, sizeof(int32_t) * (size_t)z.total);
    int32_t *row = buf + z.off_rows, *req = buf + z.off_reqs, *tile = buf + z.off_tiles;
    const int32_t per_page = b.page_size / 16;
    int32_t *item[kClasses], *join = buf + z.off_joins;
    item[0] = buf + z.off_items;
    for (int c = 1; c < kClasses; ++c) item[c] = item[c - 1] + 8 * z.items[c - 1];
    int32_t *pitem = buf + z.off_pitems, *pjoin = buf + z.off_pjoins;
    const int32_t pack = pack_of(b.n_heads / b.n_kv_heads), tile_rows = kPpRows / pack;
    int64_t part = 0, ppart = 0, first_row = 0;
    for (int i = 0; i < b.n_req; ++i) {
        const int64_t n = b.n_input[i], c = b.ctx_len[i];
        if (n == 0) continue;
        const int32_t *t = b.page_table + (int64_t)i * b.table_ld;
        req[i] = (int32_t)(tile - buf);
        for (int64_t left = (c + n + 15) / 16; left > 0; ++t)
            for (int32_t k = 0; k < per_page && left > 0; ++k, --left) *tile++ = *t * per_page + k;
        const int32_t *mine = buf + req[i];
        tile = buf + up4(tile - buf);
        for (int32_t pos = (int32_t)c; pos < c + n; ++pos, row += 4)
            row[0] = mine[pos / 16] * 16 + pos % 16, row[1] = pos;
        const auto tile_items = [&](int cl, int64_t col, int64_t cols, int64_t keys) {
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
                r[7] = classes.narrow(n);
            }
            if (parts == 1) return;
            join[0] = (int32_t)first_row, join[1] = (int32_t)col, join[2] = (int32_t)cols, join[3] = (int32_t)parts;
            join[4] = (int32_t)part, join[5] = 8 << cl, join[6] = kPpRows;
            join += 8, part += parts * (8 << cl);
        };
        const auto pair = [&](int64_t r0, int64_t rows, int64_t keys) {
            const int64_t parts = parts_of(keys, z.pchunk), per = parts == 1 ? keys : z.pchunk;
            for (int64_t p = 0; p < parts; ++p, pitem += 8) {
                pitem[0] = req[i] + (int32_t)(p * per / 16);
                pitem[1] = (int32_t)std::min<int64_t>(per, keys - p * per);
                pitem[2] = (int32_t)(first_row + r0);
                pitem[3] = (int32_t)rows;
                pitem[4] = (int32_t)(c + r0 + 1 - p * per);
                pitem[5] = parts == 1 ? -1 : (int32_t)(ppart + p * 2 * kPpRows);
                pitem[6] = classes.narrow(n);
            }
            if (parts == 1) return;
            pjoin[0] = (int32_t)(first_row + r0), pjoin[1] = 0, pjoin[2] = (int32_t)rows * pack;
            pjoin[3] = (int32_t)parts;
            pjoin[4] = (int32_t)ppart, pjoin[5] = 2 * kPpRows, pjoin[6] = tile_rows * pack;
            pjoin += 8, ppart += parts * 2 * kPpRows;
        };
        if (classes.of(b.n_input[i]) == kClasses)
            row_pairs(b, i, pair);
        else
            column_tiles(b, i, classes, tile_items);
        first_row += n;
    }
    struct Rec {
        int32_t w[8];
    };
    Rec *rec = reinterpret_cast<Rec *>(buf + z.off_items);
    for (int c = 0; c < kClasses; rec += z.items[c], ++c)
        std::stable_sort(rec, rec + z.items[c], [](const Rec &x, const Rec &y) { return x.w[1] > y.w[1]; });
    rec = reinterpret_cast<Rec *>(buf + z.off_pitems);
    std::stable_sort(rec, rec + z.pitems, [](const Rec &x, const Rec &y) { return x.w[1] > y.w[1]; });
    // Longest first to the block with the least work so far (forwards and backwards in turn: four prompts of 1024 rows
    // over 1000 keys, 40 heads over 8, left the busiest block 13 % above the mean, this way 2 %).
    if (z.pitems) {
        const int64_t vheads = b.n_heads / pack;
        std::vector<std::pair<int64_t, int32_t>> load((size_t)z.blocks);  // a heap, the least first
        std::vector<int32_t> to((size_t)(z.pitems * vheads));
        int32_t *first = buf + z.off_deal, *entry = first + z.blocks + 1;
        for (int32_t c = 0; c < (int32_t)z.blocks; ++c) load[c] = {0, c};
        for (size_t e = 0; e < to.size(); ++e) {
            std::pop_heap(load.begin(), load.end(), std::greater<>());
            to[e] = load.back().second, ++first[to[e] + 1];
            load.back().first += (rec[e / vheads].w[1] + kPpKeys - 1) / kPpKeys + kPromptExtra;
            std::push_heap(load.begin(), load.end(), std::greater<>());
        }
        for (int64_t c = 0; c < z.blocks; ++c) first[c + 1] += first[c];
        std::vector<int32_t> at(first, first + z.blocks);
        for (size_t e = 0; e < to.size(); ++e) entry[at[to[e]]++] = (int32_t)e;
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
    buf[G_SMS] = num_sms;
    for (int c = 0; c < kClasses; ++c) buf[G_ITEMS + c] = (int32_t)z.items[c];
    buf[G_PARTS] = (int32_t)z.parts;
    buf[G_JOINS] = (int32_t)z.joins;
    buf[G_O_ITEMS] = (int32_t)z.off_items;
    buf[G_O_JOINS] = (int32_t)z.off_joins;
    buf[G_JOINROWS] = (int32_t)z.join_rows;
    buf[G_PJOINROWS] = (int32_t)z.pjoin_rows;
    buf[G_PITEMS] = (int32_t)z.pitems;
    buf[G_PPARTS] = (int32_t)z.pparts;
    buf[G_PJOINS] = (int32_t)z.pjoins;
    buf[G_O_PITEMS] = (int32_t)z.off_pitems;
    buf[G_O_PJOINS] = (int32_t)z.off_pjoins;
    buf[G_O_DEAL] = (int32_t)z.off_deal;
    buf[G_PACK] = pack;
    buf[G_BOX] = std::gcd(b.page_size, kPpKeys);
    return true;
}

bool paged_plan_ok(const int32_t *hp) { return hp && hp[0] == kPagedMagic; }
PagedInfo paged_plan_info(const int32_t *hp) {
    return {hp[G_DTYPE], hp[G_HEADS],  hp[G_KV_HEADS], hp[G_DIM],          hp[G_SLOTS],
            hp[G_ROWS],  hp[G_MAXPOS], hp[G_TOTAL],    hp[G_TWICE] != 0};
}

int64_t paged_workspace_bytes(const int32_t *hp) {
    return ((int64_t)hp[G_PARTS] * hp[G_KV_HEADS] + (int64_t)hp[G_PPARTS] * (hp[G_HEADS] / hp[G_PACK])) *
           (hp[G_DIM] + 2) * 4;
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

// One thread per two 16-byte chunks of a head's row, which hold whole pairs: the
// chunks i and rot / 2 + i, or two neighbouring ones.  In between it reads its
// cosines and sines, which all heads of a row share in L1.  Bound by HBM: 8
// prompts of <= 2047 rows, 40 + 16 heads of 128, 303 MB in 48.9 us, 91 % of the copy rate
// (neighbours 51.4; with the table read 16 bytes at a time 51.3).
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

// Halves whose middle is inside a 16-byte chunk: a thread per chunk, the
// components' partners loaded one by one.  A head's row is within a warp, which
// reads all of it before it writes.  Bound by issue (three quarters of the slots, 2.7
// times the instructions of the kernel above): the same prompts with 20 or 126
// rotated components 84 us, floor 44.6; in fp32 121 us, floor 89.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_append_odd_kernel(const AppendArgs a) {
    constexpr int VEC = Elem<T>::kPer16, CH = D / VEC;
    static_assert(32 % CH == 0, "a head's row in one warp");
    pdl_trigger();
    pdl_wait();
    const int per_row = (a.heads + 2 * a.kv_heads - a.first_head) * CH;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int row = (int)min(at / per_row, (int64_t)a.n_rows - 1);  // (threads behind the last stay for the barrier)
    const int rest = (int)(at % per_row), h = a.first_head + rest / CH, c0 = rest % CH * VEC;
    const int4 rec = a.rows[row];
    const T *src = reinterpret_cast<const T *>(a.qkv) + (int64_t)row * a.ld_qkv + h * D;
    const float *cs = a.rope + (int64_t)rec.y * a.rot;
    const int half = a.rot / 2;
    float x[VEC];
    load16(src + c0, x);
    if (h < a.heads + a.kv_heads) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (c0 + e < a.rot) {
                const bool low = c0 + e < half;
                const int i = low ? c0 + e : c0 + e - half;
                const float o = Elem<T>::to_f(src[low ? i + half : i]), c = cs[i], s = cs[half + i];
                x[e] = low ? x[e] * c - o * s : x[e] * c + o * s;
            }
    }
    T *dst;
    if (h < a.heads)
        dst = reinterpret_cast<T *>(a.q_out) + (int64_t)row * a.ld_q + h * D;
    else
        dst = reinterpret_cast<T *>(a.layer) + ((int64_t)(h - a.heads) * a.slots + rec.x) * D;
    __syncwarp();  // the whole head is read before any of it is written
    if (at / per_row < a.n_rows) store16(dst + c0, x);
}

template <typename T, int D>
cudaError_t launch_append(const AppendArgs &a, bool neighbours, cudaStream_t st) {
    constexpr int VEC = Elem<T>::kPer16;
    const int64_t heads = (int64_t)a.n_rows * (a.heads + 2 * a.kv_heads - a.first_head);
    const dim3 grid((unsigned)((heads * (D / VEC / 2) + 255) / 256));
    if (neighbours) return launch_pdl(paged_append_kernel<T, D, true>, grid, dim3(256), 0, st, a);
    if ((a.rot / 2) % VEC == 0) return launch_pdl(paged_append_kernel<T, D, false>, grid, dim3(256), 0, st, a);
    const dim3 chunks((unsigned)((heads * (D / VEC) + 255) / 256));
    return launch_pdl(paged_append_odd_kernel<T, D>, chunks, dim3(256), 0, st, a);
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
// the item, loads it by TMA (K and V of a 64-dim block in one box; 16 slots
// never cross a page) into its own ring of stages, across items, and keeps its own
// running maximum m, sum l and outputs per column.  (Stages, tiles of 8 columns / of
// more: bf16 of head_dim 128 3 / 2, 64 6 / 4, below 8; fp32 of 64 3 / 2, and of 128 one, so
// that nothing is loaded ahead there but what the block's other warps have under
// way.)  At the end of an item the block's four warps meet and add up.  No warp waits for another
// while it streams, and nothing is shared between blocks: keys are split by the
// plan where there are few items (choose_chunk), the parts joined by
// paged_join_kernel, without atomics, in their order.
//
// Numerics: scores, m, l and outputs in fp32.  bf16: products of 16-bit operands
// are exact; weights go into the second product in two bf16 parts (16 bits) for
// requests of up to 16 columns, whatever they go along with, in one (2^-8) for
// others.  fp32: cw_split.  No score at all is m = -inf, from which cw_base subtracts
// 0.  Keys past a column's last are masked by index.  0 times a value that is not
// finite is NaN, so a tile with such a value behind a key that only some columns see is
// added up key by key.
//
// Bound by HBM for long contexts (64 requests of <= 4000 keys, 40 heads over 8 of
// 128: 663 MB in 105 us, 93 % of the copy rate; 40 heads of their own, 64 x <= 1000 keys:
// 97 %), by latency below some 20 MB: one request over 300 keys, 20 heads of 64, 5.1 us.
// fp32 single rows by latency too, over a tile's chain of loads, splits and products
// (some 800 instructions per 16 keys, issued in 24 to 31 % of the slots by 6 warps per SM,
// DRAM 22 to 47 %): 17 x <= 900 keys, 12 heads over 4 of 64, 10.4 us, floor 3.1; 64 x <=
// 1000 keys, 8 heads of 128, 66, floor 49.  Several rows there by issue and tensor pipe
// (48 and 31 %; a prompt's keys are read once for every 16 columns): 4 x <= 200 rows over
// <= 1000 keys, 12 over 4 of 64, 51 us, floor 1.7.  Rows of head_dim 32 / 16 as tiles of 32,
// by issue (40 %) and the chain: 4 x <= 1024 over <= 1000 keys, 12 heads over 4, 74 / 78
// us, floor 3.2 / 1.6.
namespace {

constexpr int kCwWarps = 4;
constexpr int kCwThreads = 32 * kCwWarps;

struct PagedArgs {
    const void *q;
    void *out;
    float *part, *part_ml;  // partial outputs [column][head_dim], their maxima and sums [column][2]
    const int32_t *plan;
    const int4 *items;  // {tiles at, keys, first row, first column}, {columns, last key of row 0, part or -1, narrow}
    int64_t ld_q, ld_out;
    int n_items, kv_heads, group;
    int beside;  // another kernel of the same call was launched before this one
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
    static constexpr int kStages = kWant < 1 ? 1 : kWant > 8 ? 8 : kWant;
    static constexpr bool kQInSmem = kEs == 4 || NT == 4;  // (else the queries' fragments fit into registers)
    static constexpr int kMerge = 8;                       // columns that meet at a time
    static constexpr int kQRow = D * kEs + 16;             // bytes from column to column (no bank conflicts)
    static constexpr int kLd = D + 4;               // floats from column to column (no bank conflicts)
    static constexpr uint32_t kRing = kCwWarps * kStages * kStage;
    static constexpr uint32_t kO = kRing;
    static constexpr uint32_t kMl = kO + kCwWarps * kMerge * kLd * 4;
    static constexpr uint32_t kBars = kMl + kCwWarps * kMerge * 8;
    static constexpr uint32_t kQ = (kBars + kCwWarps * kStages * 8 + 15) / 16 * 16;  // two items' queries
    static constexpr uint32_t kBytes = kQ + (kQInSmem ? 2 * 8 * NT * kQRow : 0);
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
// The two numbers of such a pair.
__device__ __forceinline__ float cw_lower(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float cw_upper(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// fp32 operands as two tf32 parts, x = hi + lo: hi cut off, lo rounded to 11
// bits, which leaves 2^-21 |x| (both rounded: 2^-22, and 10 % more time); products
// hi hi + hi lo + lo hi.  An infinity has no lower part (inf - inf): what it touches
// becomes NaN.
__device__ __forceinline__ void cw_split(uint32_t x, uint32_t &hi, uint32_t &lo) {
    hi = x & 0xffffe000u;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(__uint_as_float(x) - __uint_as_float(hi)));
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
    constexpr bool kKeepQ = !S::kQInSmem;
    constexpr unsigned kFull = 0xffffffffu;
    extern __shared__ __align__(1024) uint8_t cw_smem[];
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
    // The first kernel of a call triggers behind its wait, so that all in front of the call has ended when the next
    // one starts: that one need not wait for the first, which it does not depend on, but before it ends.
    if (!a.beside) pdl_wait();
    pdl_trigger();

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

    // Queries of entry e to shared memory, buffer `buf` (columns behind the last repeat it and are not written).
    const auto fetch_q = [&](int e, int buf) {
        if (e < total) {
            const int4 r = a.items[2 * (e / a.kv_heads)];
            const int cols = a.items[2 * (e / a.kv_heads) + 1].x, h = e % a.kv_heads;
            constexpr int CH = D * S::kEs / 16;
            for (int x = threadIdx.x; x < 8 * NT * CH; x += kCwThreads) {
                const int c = r.w + min(x / CH, cols - 1);
                const T *src = reinterpret_cast<const T *>(a.q) + (int64_t)(r.z + c / a.group) * a.ld_q +
                               (h * a.group + c % a.group) * D + x % CH * (16 / S::kEs);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 smem_u32(cw_smem) + S::kQ + (buf * 8 * NT + x / CH) * S::kQRow + x % CH * 16),
                             "l"(src)
                             : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (!kKeepQ) fetch_q(nth(0), 0);

    for (int k = 0;; ++k) {
        const int e = nth(k);
        if (e >= total) break;
        if constexpr (!kKeepQ) {
            fetch_q(nth(k + 1), (k + 1) & 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
        }
        const uint32_t qs = smem_u32(cw_smem) + S::kQ + (k & 1) * 8 * NT * S::kQRow;
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
        uint32_t qb[NT][kKeepQ ? KS : 1][2];
        if constexpr (kKeepQ) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int c = c0 + min(8 * nt + g8, n_cols - 1);
                const uint32_t *qp = reinterpret_cast<const uint32_t *>(reinterpret_cast<const T *>(a.q) +
                                                                        (int64_t)(r0.z + c / a.group) * a.ld_q +
                                                                        (h * a.group + c % a.group) * D) + t4;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) qb[nt][ks][0] = qp[8 * ks], qb[nt][ks][1] = qp[8 * ks + 4];
            }
        }
        float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
        }
        // The item's keys.  Weights in two bf16 parts are 1 % of the time of single rows and 8 % of that of 32 columns,
        // where only requests that have up to 16 by themselves take them.
        const auto stream = [&](auto two) __attribute__((always_inline)) {
            constexpr bool kTwo = decltype(two)::value;
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
                        uint32_t f[4], fh[4], fl[4], qh[2], ql[2];
                        cw_ldsm(at(kb, lane & 15, 2 * ks + (lane >> 4)), f);
#pragma unroll
                        for (int x = 0; x < 4; ++x) cw_split(f[x], fh[x], fl[x]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t q = qs + (8 * nt + g8) * S::kQRow + (8 * ks + t4) * 4;
                            cw_split(cw_lds(q), qh[0], ql[0]);
                            cw_split(cw_lds(q + 16), qh[1], ql[1]);
                            cw_mma_tf32(hh[ks % NC][nt], fh, qh[0], qh[1]);
                            cw_mma_tf32(c[nt], fh, ql[0], ql[1]);
                            cw_mma_tf32(c[nt], fl, qh[0], qh[1]);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int n = 0; n < NC; ++n) c[nt][x] += hh[n][nt][x];
                    // an infinity, or a NaN: these scores once more, component by component
                    bool odd = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) odd |= c[nt][x] != c[nt][x] && 16 * t + g8 + 8 * (x >> 1) < keys;
                    if (__any_sync(kFull, odd))
#pragma unroll 1
                        for (int nt = 0; nt < NT; ++nt) {
                            float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                            for (int d = 0; d < D; ++d)
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const uint32_t kv = cw_lds(at(kb, g8 + 8 * (x >> 1), d / 4) + d % 4 * 4);
                                    const uint32_t qv = cw_lds(qs + (8 * nt + 2 * t4 + (x & 1)) * S::kQRow + 4 * d);
                                    z[x] = fmaf(__uint_as_float(kv), __uint_as_float(qv), z[x]);
                                }
#pragma unroll
                            for (int y = 0; y < NT; ++y)
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    if (y == nt) c[y][x] = z[x];
                        }
                } else if constexpr (!kKeepQ) {
#pragma unroll
                    for (int k2 = 0; k2 < KS; k2 += 2) {  // (head_dim 16: the second half of a load is not used)
                        uint32_t f[2][4], q[4];
#pragma unroll
                        for (int z = 0; z < 2 && k2 + z < KS; ++z)
                            cw_ldsm(at(kb, lane & 15, 2 * (k2 + z) + (lane >> 4)), f[z]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int ch = KS == 1 ? (lane >> 3 & 1) : 2 * k2 + (lane >> 3);
                            cw_ldsm(qs + (8 * nt + (lane & 7)) * S::kQRow + ch * 16, q);
#pragma unroll
                            for (int z = 0; z < 2 && k2 + z < KS; ++z) cw_mma_bf16(c[nt], f[z], q[2 * z], q[2 * z + 1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        uint32_t f[4];
                        cw_ldsm(at(kb, lane & 15, 2 * ks + (lane >> 4)), f);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) cw_mma_bf16(c[nt], f, qb[nt][ks][0], qb[nt][ks][1]);
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
                // weights; bf16: in two parts, 16 bits kept, in two products, or in one, and l sums what is used
                uint32_t pw[NT][2], pl[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float b0 = cw_base(m[nt][0]), b1 = cw_base(m[nt][1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        c[nt][2 * x] = cw_exp2(c[nt][2 * x] - b0), c[nt][2 * x + 1] = cw_exp2(c[nt][2 * x + 1] - b1);
                        if constexpr (!F32) {
                            pw[nt][x] = cw_pack(c[nt][2 * x], c[nt][2 * x + 1]);
                            const float w0 = cw_lower(pw[nt][x]), w1 = cw_upper(pw[nt][x]);
                            if constexpr (kTwo)
                                pl[nt][x] = cw_pack(c[nt][2 * x] - w0, c[nt][2 * x + 1] - w1);
                            else
                                c[nt][2 * x] = w0, c[nt][2 * x + 1] = w1;
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
                                        if (16 * t + r < sees[nt][i])
                                            o[nt][mt][2 * x + i] = fmaf(p[i], vf, o[nt][mt][2 * x + i]);
                                }
                        }
                } else if constexpr (F32) {
                    // the keys of a product in the order 0 2 4 6 1 3 5 7, which spreads V's rows over the banks
                    uint32_t qh[NT][2][2], ql[NT][2][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int src = (2 * t4 + i) * 4 + (g8 >> 1);
                                const float p0 = __shfl_sync(kFull, c[nt][2 * x], src);
                                const float p1 = __shfl_sync(kFull, c[nt][2 * x + 1], src);
                                cw_split(__float_as_uint(g8 & 1 ? p1 : p0), qh[nt][x][i], ql[nt][x][i]);
                            }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        float y[NT][4];  // this tile's sum on its own: o is added to in fp32
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) y[nt][0] = y[nt][1] = y[nt][2] = y[nt][3] = 0.f;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t fh[4], fl[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const int d = 16 * mt + g8 + 8 * (z & 1);
                                cw_split(cw_lds(at(vb, 8 * x + 2 * t4 + (z >> 1), d / 4) + d % 4 * 4), fh[z], fl[z]);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                cw_mma_tf32(y[nt], fl, qh[nt][x][0], qh[nt][x][1]);
                                cw_mma_tf32(y[nt], fh, ql[nt][x][0], ql[nt][x][1]);
                                cw_mma_tf32(y[nt], fh, qh[nt][x][0], qh[nt][x][1]);
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int x = 0; x < 4; ++x) o[nt][mt][x] += y[nt][x];
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            pw[nt][x] = cw_transpose(pw[nt][x]);
                            if constexpr (kTwo) pl[nt][x] = cw_transpose(pl[nt][x]);
                        }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t f[4];
                        cw_ldsm_t(at(vb, (lane >> 4) * 8 + (lane & 7), 2 * mt + ((lane >> 3) & 1)), f);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            cw_mma_bf16(o[nt][mt], f, pw[nt][0], pw[nt][1]);
                            if constexpr (kTwo) cw_mma_bf16(o[nt][mt], f, pl[nt][0], pl[nt][1]);
                        }
                    }
                }
                __syncwarp();  // every lane has read the stage
                ++used;
                issue();
            }
        };
        if (NT < 4 || r1.w)
            stream(std::true_type());
        else
            stream(std::false_type());
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
                        mo[x * S::kLd + 16 * mt + g8] = o[nt][mt][i],
                        mo[x * S::kLd + 16 * mt + g8 + 8] = o[nt][mt][2 + i];
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
    if (a.beside) pdl_wait();
}

// Split keys: the parts of a column, in their order.  One block per (column tile,
// head) and column, or column per thread group; 4 components per thread.
// `heads` and `group`: key/value heads and the query heads of each; for prompts
// the tiles' heads and the heads packed into each.
struct JoinArgs {
    const float *part, *part_ml;
    const int4 *joins;  // {first row, first column, columns, parts}, {first part, from part to part, columns of 128, 0}
    void *out;
    int64_t ld_out;
    int heads, group;
};
template <typename T, int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const JoinArgs a) {
    constexpr int L4 = D / 4, N = 128 / L4;  // thread groups
    __shared__ float4 so[N][L4];
    __shared__ float2 sml[N];
    pdl_trigger();
    pdl_wait();
    const int j = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
    const int4 r0 = a.joins[2 * j], r1 = a.joins[2 * j + 1];
    const int grp = threadIdx.x / L4, d = threadIdx.x % L4;
    const bool many = r0.w >= kManyParts;  // the groups share a column's parts, else each has a column
    const int col = many ? blockIdx.y : blockIdx.y * N + grp;
    if ((many ? col : (int)blockIdx.y * N) >= r0.z) return;
    const int x = col / r1.z * kPpRows + col % r1.z;  // (a tile of 128 may hold fewer columns than that)
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // (A prompt's sums may be 2^127 over an m that lags as far behind: factors in two halves, exp2 ends at 2^-126.)
    constexpr bool kHalves = sizeof(T) == 2;
    const auto add = [&](float m2, float l2, const float4 &o2) {
        const float mx = fmaxf(m, m2), base = cw_base(mx), power = kHalves ? 0.5f : 1.f;
        const float f = cw_exp2(power * (m - base)), f2 = cw_exp2(power * (m2 - base));
        const auto sum = [&](float x, float y) { return kHalves ? x * f * f + y * f2 * f2 : x * f + y * f2; };
        l = sum(l, l2), m = mx;
        o = make_float4(sum(o.x, o2.x), sum(o.y, o2.y), sum(o.z, o2.z), sum(o.w, o2.w));
    };
    if (col < r0.z) {
#pragma unroll 4
        for (int p = many ? grp : 0; p < r0.w; p += many ? N : 1) {
            const int64_t at = ((int64_t)r1.x + (int64_t)p * r1.y) * a.heads + (int64_t)h * r1.y + x;
            const float2 v = *reinterpret_cast<const float2 *>(a.part_ml + 2 * at);
            add(v.x, v.y, *reinterpret_cast<const float4 *>(a.part + at * D + 4 * d));
        }
    }
    if (many) {
        so[grp][d] = o;
        if (d == 0) sml[grp] = make_float2(m, l);
        __syncthreads();
        if (grp) return;
#pragma unroll
        for (int z = 1; z < N; ++z) add(sml[z].x, sml[z].y, so[z][d]);
    }
    if (col >= r0.z) return;
    const int c = r0.y + col;
    T *dst = reinterpret_cast<T *>(a.out) + (int64_t)(r0.x + c / a.group) * a.ld_out +
             (h * a.group + c % a.group) * D + 4 * d;
    const float f = 1.f / l;
    store4(dst, o.x * f, o.y * f, o.z * f, o.w * f);
}

}  // namespace

// ---------------------------------------------------------------------------
// Prompts on the fifth-generation tensor cores (bf16, head_dim 64 or 128)
// ---------------------------------------------------------------------------
// The rows of a tile are (row, head) pairs of one key/value head, heads
// innermost, 128 / pack rows of a request: every key tile is loaded once for all
// heads that share it, and short chunks of prompts still fill tiles.  An item is
// two such tiles, t = 0 and 1, over one range of keys, 64 at a time; each has a
// warpgroup of its own, a thread per tile row.
//   S_t = Q_t K^T   128 x 64, both operands from shared memory
//   O_t += P_t V    P (bf16) from tensor memory, V as it lies in its pages
// Tensor memory: two buffers of S per tile (64 columns each; P takes the first
// half of its S, the second part of a narrow request's weights the other), O_0, O_1
// (128 each).  The chain from S over the softmax to P V and back has some 2400 cycles
// of latency beside its work (products, commits, waits, tensor-memory accesses;
// measured with that work left out), so the next S is always under way: a softmax
// finds it when it is done with the last.
// (With one buffer of 128 keys the same work took 4400 cycles per 128 keys of both
// tiles, now 2400.)  Shared memory: Q, a ring of K and one of V; the loads are
// boxes of a page (or of the part of it that divides 64 slots).
// Bound: a step of both tiles takes some 1200 cycles.  head_dim 128: tensor core and
// shared memory, which feeds Q again for every 64 keys, have 1024 of them each, but not
// the same ones: a product of S is 32 cycles of the one and 48 of the other, one of P V
// 64 and 32, which is 1280 if no product overlaps the next.  head_dim 64: nothing is
// full (tensor core 512, exponentials 512, issue 42 %); the softmax of two warps per
// scheduler takes 830, then 350 of waits and tensor-memory accesses: the chain.  Beside
// that 1.5 to 2.4 us at an item's end, where the tensor core idles.
// 4 prompts of <= 1024 rows over <= 1000 keys, 40 heads over 8 of 128: 70 us, 0.55 of
// the tensor peak; 8 of <= 2047 rows, 16 over 2 of 64: 51 us, 0.33.  (K and V released
// together: 72.5 us, and 200 rows over 30000 keys, 32 heads over 8, 138 us for 105;
// the two tiles half a step apart: 75 and 46.6 us, dropped.)
// Weights of two bf16 parts for all requests, not only for narrow ones, would be 87
// and 56 us.  Those of one part are summed up as they are used (4 % of the time at
// head_dim 64, 0.3 % at 128), so that a row of which one weight is above all others does
// not have that one's rounding in its output.
// Every P is formed against the m that O and l carry, which is near a row's
// maximum and need not be it: O is rescaled only where it lags by more than 2^8.
// Keys past the item's last are masked by index and their V rows zeroed.  A
// masked weight of 0 times a value that is not finite is NaN, and a tile's weights
// overflow where its scores are 2^127 above all in front of them: a row whose output is
// not finite, and of which one of these may be so, is computed once more, key by key,
// over what it sees, 1.2 us for two keys (head_dim 64: four): four prompts of <= 1024
// rows over <= 1000 keys, the largest with scores that grow by more than 2^127 from
// tile to tile, 42 ms for 61 us.  (Weights formed anew against the maximum within
// the tile took 120 us there, but 5 to 12 % of everyone else's time.)
namespace {

constexpr int kPpThreads = 384;  // two softmax warpgroups, one with the TMA and the MMA warps
constexpr int kPpTma = 8, kPpMma = 9, kPpTmaV = 11;  // warps: Q and K, products of either row tile, V
constexpr uint32_t kPpAtom = 16384;    // 128 rows of 128 bytes (Q)
constexpr uint32_t kPpKv = 8192;       // 64 rows of 128 bytes (K, V)
constexpr float kPpGrown = 256.f;       // sum of a tile's weights from which on m follows
constexpr float kPpOver = 0x1p20f;      // and from which on O may overflow (values of 2^100)

template <int D>
struct PpLayout {
    static constexpr int kAtoms = D / 64;
    static constexpr int kStages = D == 64 ? 8 : 4;
    static constexpr uint32_t kTile = kAtoms * kPpKv;  // a key tile's K or V
    static constexpr uint32_t kQ = 0;                  // [tile][atom]
    static constexpr uint32_t kK = 2 * kAtoms * kPpAtom;
    static constexpr uint32_t kV = kK + kStages * kTile;
    static constexpr uint32_t kBars = kV + kStages * kTile;
    static constexpr uint32_t kOut = kBars + 512;  // per softmax warp: 32 rows of 32 components, 80 bytes apart
    static constexpr uint32_t kBytes = kOut + 8 * 32 * 80;
};
struct PpBars {
    uint64_t q_full, q_empty, full[2][8], empty[2][8];  // (K, V)
    uint64_t s_full[2][2], p_full[2][2];  // [tile][buffer]
    uint64_t o_done[2][2];                // [tile]: the products of an item's last key tile but one, and of its last
    uint64_t drain[2];
    uint32_t tmem;
    int abort, alive;  // alive: changes while a softmax warp works on rows key by key
};
struct PpArgs {
    const bf16 *q, *layer;
    bf16 *out;
    float *part, *part_ml;
    const int32_t *plan;
    const int4 *items;  // {tiles at, keys, first row, rows}, {keys that the first row sees, part or -1, narrow, 0}
    const int32_t *deal;
    int64_t ld_q, ld_out, slots;
    int vheads, pack, per_kv, kv_heads, box;  // (per_kv: tile heads of a key/value head)
    float scale_log2;
    unsigned *err;
};

__device__ __forceinline__ void pp_tma_q(uint32_t dst, const void *tmap, uint64_t *bar, int c0, int head, int row) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(dst),
        "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(head), "r"(row)
        : "memory");
}
__device__ __forceinline__ void pp_tma_kv(uint32_t dst, const void *tmap, uint64_t *bar, int c0, int slot, int h, int kv,
                                          uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
        "{%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
        "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(slot), "r"(h), "r"(kv), "l"(policy)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem] (a row of A per lane, two elements per column) and A[smem] * B[smem]; the
// descriptors of shared memory by their lower halves, in which the address is.
__device__ __forceinline__ void pp_mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void pp_mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Lower and upper halves of the descriptors (smem_desc_k128): an operand's leading stride goes into the lower one,
// 1 where it is K-major (not used), the blocks' distance where V is read MN-major.
constexpr uint32_t kPpDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t pp_desc_k(uint32_t saddr) { return (saddr >> 4 & 0x3FFFu) | 1u << 16; }
__device__ __forceinline__ uint32_t pp_desc_mn(uint32_t saddr) { return (saddr >> 4 & 0x3FFFu) | (kPpKv >> 4) << 16; }
__device__ __forceinline__ void pp_ld32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Waits for this thread's loads; the registers are operands, so that no use of them is placed before the wait.
__device__ __forceinline__ void pp_wait_ld32(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void pp_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};"
        :
        : "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void pp_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Two fp32 operations at once.
__device__ __forceinline__ uint64_t pp_pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void pp_unpair(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t pp_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t pp_mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Adds the two numbers of a bf16 pair to two fp32 sums.
__device__ __forceinline__ void pp_add_bf16(float &lo, float &hi, uint32_t w) {
    asm("{\n\t.reg .b16 x, y;\n\t"
        "mov.b32 {x, y}, %2;\n\t"
        "add.rn.f32.bf16 %0, x, %0;\n\t"
        "add.rn.f32.bf16 %1, y, %1;\n\t}"
        : "+f"(lo), "+f"(hi)
        : "r"(w));
}

// A bounded wait; when it gives up, or another warp has, the abort flag is set and every later wait ends at once.  A
// warp that computes rows once more, key by key, takes seconds over long contexts: its time does not count.
__device__ __noinline__ bool pp_wait_on(uint32_t bar, uint32_t parity, unsigned *err, volatile int *abort);
__device__ __forceinline__ bool pp_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ bool pp_wait_on(uint32_t bar, uint32_t parity, unsigned *err, volatile int *abort) {
    unsigned long long t0 = 0;
    int alive = abort[1];
    for (uint32_t it = 1;; ++it) {
        if (pp_try(bar, parity)) return true;
        if (*abort) return false;
        if ((it & 63u) == 0) {
            const unsigned long long now = global_timer_ns();
            if (t0 == 0 || alive != abort[1]) t0 = now, alive = abort[1];
            if (now - t0 > kWaitLimitNs) {
                raise_err(err, ERR_WAIT_TIMEOUT);
                *abort = 1;
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool pp_wait(uint32_t bar, uint32_t parity, unsigned *err, volatile int *abort) {
    return pp_try(bar, parity) || pp_wait_on(bar, parity, err, abort);
}
__device__ __forceinline__ void pp_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float pp_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// One row over keys 0 .. n - 1 of its item by the whole warp: afterwards every
// lane holds m, l and 8 components of o, lane % (D / 8) * 8 on.
template <int D>
__device__ __noinline__ void pp_row(const PpArgs &a, const bf16 *q, const int32_t *tiles, int n, int kvh, float &m,
                                    float &l, float *o, volatile int *alive) {
    constexpr int LPT = D / 8, TPW = 32 / LPT;
    const int lane = threadIdx.x & 31, g = lane / LPT, sub = lane % LPT;
    const bf16 *kb = a.layer + (int64_t)kvh * a.slots * D + sub * 8, *vb = kb + (int64_t)a.kv_heads * a.slots * D;
    float qf[8];
    load16(q + sub * 8, qf);
    m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
    for (int t0 = 0; t0 < n; t0 += TPW) {
        const int t = t0 + g;
        if (t0 % 4096 == 0) *alive = *alive + 1;  // (which of the warps' counts stays does not matter)
        if (t0 % 64 == 0 && __any_sync(0xffffffffu, l != l)) break;  // a score of +inf or NaN: so is every component
        float k[8], v[8], s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) k[e] = v[e] = 0.f;
        if (t < n) {
            const int64_t slot = (int64_t)tiles[t / 16] * 16 + t % 16;
            load16(kb + slot * D, k);
            load16(vb + slot * D, v);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(qf[e], k[e], s);
#pragma unroll
        for (int x = LPT / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s = t < n ? s * a.scale_log2 : -INFINITY;
        const float mx = fmaxf(m, s), base = cw_base(mx), corr = cw_exp2(m - base), p = cw_exp2(s - base);
        l = l * corr + p, m = mx;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(p, v[e], o[e] * corr);
    }
#pragma unroll
    for (int x = LPT; x < 32; x <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, x), l2 = __shfl_xor_sync(0xffffffffu, l, x);
        const float mx = fmaxf(m, m2), base = cw_base(mx), f = cw_exp2(m - base), f2 = cw_exp2(m2 - base);
        l = l * f + l2 * f2, m = mx;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] * f + __shfl_xor_sync(0xffffffffu, o[e], x) * f2;
    }
}

// The last of keys first .. end - 1 of an item whose value is not finite in some component, or -1; by the whole warp.
template <int D>
__device__ __noinline__ int pp_last_odd(const PpArgs &a, const int32_t *tiles, int first, int end, int kvh) {
    constexpr int LPT = D / 8, TPW = 32 / LPT;
    const int lane = threadIdx.x & 31;
    const bf16 *vb = a.layer + ((int64_t)a.kv_heads + kvh) * a.slots * D + lane % LPT * 8;
    int last = -1;
    for (int t = first + lane / LPT; t < end; t += TPW) {
        float v[8], z = 0.f;
        load16(vb + ((int64_t)tiles[t / 16] * 16 + t % 16) * D, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) z = fmaf(v[e], 0.f, z);
        if (z != 0.f) last = t;
    }
    return __reduce_max_sync(0xffffffffu, last);
}

template <int D>
__global__ void __launch_bounds__(kPpThreads, 1)
    paged_prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmkv,
                        const PpArgs a) {
    using L = PpLayout<D>;
    constexpr unsigned kFull = 0xffffffffu;
    extern __shared__ __align__(1024) uint8_t pp_smem[];
    if (smem_u32(pp_smem) & 1023u) {  // uniform: every thread leaves before any barrier
        if (threadIdx.x == 0) raise_err(a.err, 8u);
        return;
    }
    uint8_t *const sm = pp_smem;
    PpBars &bar = *reinterpret_cast<PpBars *>(sm + L::kBars);
    volatile int *const abort = &bar.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        // (the empty ones: both MMA threads, also for what their row tile does not see)
        for (int kv = 0; kv < 2; ++kv)
            for (int s = 0; s < L::kStages; ++s) mbar_init(&bar.full[kv][s], 1), mbar_init(&bar.empty[kv][s], 2);
        mbar_init(&bar.q_full, 1);
        mbar_init(&bar.q_empty, 2);
        for (int x = 0; x < 4; ++x) {
            mbar_init(&bar.s_full[x >> 1][x & 1], 1);
            mbar_init(&bar.p_full[x >> 1][x & 1], 4);  // an arrival per warp
            mbar_init(&bar.o_done[x >> 1][x & 1], 1);
        }
        mbar_init(&bar.drain[0], 1);
        mbar_init(&bar.drain[1], 1);
        *abort = 0, abort[1] = 0;
        fence_mbar_init();
        prefetch_tmap(&tmq);
        prefetch_tmap(&tmkv);
    }
    // Tensor memory only once the kernel in front has ended: one that triggers ahead of its own allocation could wait
    // for these columns, and this one for its end.
    pdl_wait();
    if (warp == kPpMma) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    pdl_trigger();  // (behind the wait: paged_cols_kernel may run beside this one)

    const int tile_rows = kPpRows / a.pack;
    const int32_t *const entry = a.deal + gridDim.x + 1 + a.deal[blockIdx.x];
    const int entries = a.deal[blockIdx.x + 1] - a.deal[blockIdx.x];
    struct Item {
        int next;  // the entry after this one
        int vh, at, keys, row, rows, sees, part;
        bool narrow;
        int n_rows[2], nk[2], n_kt;  // rows and key tiles of either row tile, key tiles of the item
    };
    // The block's k-th item, asked for in order; false behind the last.
    const auto item_at = [&](int k, Item &it) {
        if (k && k >= entries) return false;
        const int e = k ? it.next : (int)blockIdx.x;  // (which is entry[0], without waiting for it)
        if (k + 1 < entries) it.next = entry[k + 1];
        const int4 r0 = a.items[2 * (e / a.vheads)], r1 = a.items[2 * (e / a.vheads) + 1];
        it.vh = e % a.vheads;
        it.at = r0.x, it.keys = r0.y, it.row = r0.z, it.rows = r0.w, it.sees = r1.x, it.part = r1.y;
        it.narrow = r1.z;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            it.n_rows[t] = min(max(it.rows - t * tile_rows, 0), tile_rows);
            const int last = min(it.sees + t * tile_rows + it.n_rows[t] - 1, it.keys);  // keys that its last row sees
            it.nk[t] = it.n_rows[t] > 0 && last > 0 ? (last + kPpKeys - 1) / kPpKeys : 0;
        }
        it.n_kt = max(it.nk[0], it.nk[1]);
        return true;
    };
    const auto wait = [&](uint64_t *b, uint32_t phase) { return pp_wait(smem_u32(b), phase & 1u, a.err, abort); };
    // Key tiles are numbered g = 0, 1, .. across this block's items (stage g % kStages, its use g / kStages).

    if (warp == kPpTma || warp == kPpTmaV) {
        // ------------------------------ TMA ------------------------------
        // One thread for Q and K, one for V (a box per lane is issued lane after lane, at some 140 cycles each).  K and V
        // have a ring each: a stage of K is free once its S is done, two steps ahead of its P V.
        if (elect_one()) {
            const int kv = warp == kPpTmaV;
            uint64_t *const full = bar.full[kv], *const empty = bar.empty[kv];
            const uint32_t ring = smem_u32(sm + (kv ? L::kV : L::kK));
            const uint64_t pol = l2_policy_evict_normal();  // every row tile of the request reads them
            const int per = a.box / 16;
            uint32_t g = 0, q_used = 0, used = 0;
            bool ok = true;
            Item it;
            for (int k = 0; ok && item_at(k, it); ++k) {
                if (!kv) {
                    if (k >= 1 && !(ok = wait(&bar.q_empty, (uint32_t)(k - 1)))) break;
                    const int tiles = it.n_rows[1] > 0 ? 2 : 1;
                    mbar_arrive_expect_tx(&bar.q_full, (uint32_t)(tiles * L::kAtoms * tile_rows * a.pack * 128));
                    for (int t = 0; t < tiles; ++t)
#pragma unroll
                        for (int c = 0; c < L::kAtoms; ++c)
                            pp_tma_q(smem_u32(sm + L::kQ) + (uint32_t)(t * L::kAtoms + c) * kPpAtom, &tmq, &bar.q_full,
                                     64 * c, it.vh * a.pack, it.row + t * tile_rows);
                    ++q_used;
                }
                const int kvh = it.vh / a.per_kv, n_tiles = (it.keys + 15) / 16;
                // slots / 16 of a key tile's four 16 keys (the plan's tables of a request start 16-byte aligned, a part
                // of its keys at a multiple of 64)
                const int4 *index = reinterpret_cast<const int4 *>(a.plan + it.at);
                int4 next = index[0];
                for (int j = 0; j < it.n_kt; ++j, ++g) {
                    const uint32_t s = g % L::kStages;
                    const int slot[4] = {next.x, next.y, next.z, next.w}, here = min(n_tiles - 4 * j, 4);
                    if (j + 1 < it.n_kt) next = index[j + 1];
                    if (g >= L::kStages && !(ok = wait(&empty[s], g / L::kStages - 1))) break;
                    mbar_arrive_expect_tx(&full[s], (uint32_t)((here + per - 1) / per * a.box * (128 * L::kAtoms)));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < here && (e & (per - 1)) == 0)
#pragma unroll
                            for (int c = 0; c < L::kAtoms; ++c)
                                pp_tma_kv(ring + s * L::kTile + c * kPpKv + e * 2048u, &tmkv, &full[s], 64 * c,
                                          slot[e] * 16, kvh, kv, pol);
                    ++used;
                }
            }
            if (!ok) {  // the copies in flight land before the block ends
                *abort = 1;
                if (q_used > 0) mbar_wait_bounded(&bar.q_full, (q_used - 1) & 1u, a.err);
                for (uint32_t x = used > L::kStages ? used - L::kStages : 0; x < used; ++x)
                    mbar_wait_bounded(&full[x % L::kStages], (x / L::kStages) & 1u, a.err);
            }
        }
        __syncwarp();
    } else if (warp == kPpMma || warp == kPpMma + 1) {
        // ------------------------------ MMA ------------------------------
        // A thread for each row tile: a product with its waits and commits takes it some 500 cycles, so that one thread
        // for both tiles held up everything else.  It walks all key tiles of the block, the P V of key tile g in
        // step; S runs ahead by up to two products, and less than the ring in key tiles (both may block for a load,
        // which has to be one that no release of its own stands in front of).
        if (elect_one()) {
            const uint32_t t = (uint32_t)(warp - kPpMma);
            const uint32_t idesc_s = idesc_bf16_f32(kPpRows, kPpKeys);
            const uint32_t idesc_pv = idesc_bf16_f32(kPpRows, D) | (1u << 16);  // B (V) MN-major
            Item is, iv;  // the items of S and of P V
            int ks = 0, js = 0;
            uint32_t gs = 0, ns = 0, np = 0;
            bool more = item_at(0, is), ok = true, ready = false;
            const auto next_s = [&]() {  // behind the last use of key tile gs
                ++gs;
                if (++js == is.n_kt) {
                    tc_commit(&bar.q_empty);  // (a commit covers all of this thread's products so far)
                    js = 0, more = item_at(++ks, is);
                }
            };
            // Comes to the next key tile that the row tile sees, below key tile `end`, and waits for its keys.
            const auto prepare_s = [&](uint32_t end) {
                while (ok && !ready && more && gs < end) {
                    const uint32_t st = gs % L::kStages;
                    ok = wait(&bar.full[0][st], gs / L::kStages) && (js > 0 || wait(&bar.q_full, (uint32_t)ks));
                    if (!ok) break;
                    ready = js < (t ? is.nk[1] : is.nk[0]);
                    if (!ready) mbar_arrive(&bar.empty[0][st]), next_s();
                }
            };
            // S of one key tile, P V of one key tile: the products, and the commit that says so.
            const uint32_t s_t = tmem + 128u * t, qd = pp_desc_k(smem_u32(sm + L::kQ) + t * (L::kAtoms * kPpAtom));
            const auto mma_s = [&](uint32_t b, uint32_t kd) {
                // S takes the place of P two products before it, whose P V this thread has issued: the tensor core runs
                // the products of one thread in their order.
#pragma unroll
                for (uint32_t x = 0; x < D / 16; ++x)  // 16 components: 32 bytes of a 64-component block
                    pp_mma_ss(s_t + 64u * b, qd + (((x >> 2) * kPpAtom + (x & 3u) * 32u) >> 4),
                              kd + (((x >> 2) * kPpKv + (x & 3u) * 32u) >> 4), kPpDescHi, idesc_s, x);
                pp_commit(smem_u32(&bar.s_full[t][0]) + 8u * b);
            };
            const auto mma_pv = [&](uint32_t b, uint32_t vd, uint32_t accumulate) {
#pragma unroll
                for (uint32_t x = 0; x < kPpKeys / 16; ++x)  // 16 keys: 16 rows of V, 8 columns of P
                    pp_mma_ts(s_t + 256u, s_t + 64u * b + 8u * x, vd + x * (2048 >> 4), kPpDescHi, idesc_pv,
                              accumulate | x);
                if (iv.narrow)  // the weights' second part
#pragma unroll
                    for (uint32_t x = 0; x < kPpKeys / 16; ++x)
                        pp_mma_ts(s_t + 256u, s_t + 64u * b + 32u + 8u * x, vd + x * (2048 >> 4), kPpDescHi, idesc_pv,
                                  1u);
            };
            const uint32_t kd0 = pp_desc_k(smem_u32(sm + L::kK)), vd0 = pp_desc_mn(smem_u32(sm + L::kV));
            const auto issue_s = [&]() {
                tc_fence_after();
                mma_s(ns & 1u, kd0 + gs % L::kStages * (L::kTile >> 4));
                tc_commit(&bar.empty[0][gs % L::kStages]);
                ++ns, ready = false;
                next_s();
            };
            uint32_t g = 0;
            for (int k = 0; ok && item_at(k, iv); ++k) {
                const int nk = t ? iv.nk[1] : iv.nk[0];
                // (not into the next item: its queries come once the last S of this one is done, and its P V wait behind)
                const uint32_t item_end = g + iv.n_kt;
                for (int j = 0; ok && j < iv.n_kt; ++j, ++g) {
                    const uint32_t st = g % L::kStages, b = np & 1u;
                    for (;;) {  // (the next S is ready to go when P arrives)
                        prepare_s(min(g + L::kStages, item_end));
                        if (!ready || ns >= np + 2) break;
                        issue_s();
                    }
                    if (!ok) break;
                    if (j >= nk) {  // (its own arrivals are in the order of the loads)
                        if (!(ok = wait(&bar.full[1][st], g / L::kStages))) break;
                        mbar_arrive(&bar.empty[1][st]);
                        continue;
                    }
                    // (an item's first P is written after the last item's O has been read out)
                    if (ready && ks == k && js == j + 2) {
                        // The steps in the middle of an item, with as few instructions as they can do with: this
                        // thread is alone, each of them takes its whole latency.
                        const uint32_t k_full = smem_u32(bar.full[0]), k_empty = smem_u32(bar.empty[0]);
                        const uint32_t v_full = smem_u32(bar.full[1]), v_empty = smem_u32(bar.empty[1]);
                        const uint32_t p0 = smem_u32(&bar.p_full[t][0]);
                        uint32_t s_st = gs % L::kStages, s_ph = gs / L::kStages & 1u, n = np;
                        uint32_t v_st = st, v_ph = g / L::kStages & 1u;
                        const int steps = nk - js;  // S of the item's key tiles js .. nk - 1
                        for (int i = 0; i < steps; ++i) {
                            const uint32_t b = n & 1u;
                            ok = pp_wait(k_full + 8u * s_st, s_ph, a.err, abort) &&
                                 pp_wait(v_full + 8u * v_st, v_ph, a.err, abort) &&
                                 pp_wait(p0 + 8u * b, n >> 1 & 1u, a.err, abort);
                            if (!ok) break;
                            tc_fence_after();
                            mma_pv(b, vd0 + v_st * (L::kTile >> 4), (uint32_t)(j + i));
                            pp_commit(v_empty + 8u * v_st);
                            mma_s(b, kd0 + s_st * (L::kTile >> 4));
                            pp_commit(k_empty + 8u * s_st);
                            ++n;
                            if (++v_st == L::kStages) v_st = 0, v_ph ^= 1u;
                            if (++s_st == L::kStages) s_st = 0, s_ph ^= 1u;
                        }
                        if (!ok) break;
                        np += steps, ns += steps, ready = false;
                        g += steps - 1, j += steps - 1;  // (this step among them)
                        gs += steps - 1, js = nk - 1;
                        next_s();
                        continue;
                    }
                    if (!(ok = wait(&bar.full[1][st], g / L::kStages) && wait(&bar.p_full[t][b], np >> 1))) break;
                    tc_fence_after();
                    mma_pv(b, vd0 + st * (L::kTile >> 4), (uint32_t)j);
                    tc_commit(&bar.empty[1][st]);
                    if (j >= nk - 2) tc_commit(&bar.o_done[t][j == nk - 1]);
                    if (ready) issue_s();
                    ++np;
                }
            }
            if (!ok) *abort = 1;
            // every product issued has completed before stages and tensor memory are given up
            tc_commit(&bar.drain[t]);
            mbar_wait_bounded(&bar.drain[t], 0u, a.err);
        }
        __syncwarp();
    } else if (warp < kPpTma) {
        // ------------------------------ softmax ------------------------------
        // A thread per row.  What bounds it is the number of instructions between one S and the next: a tile's weights
        // are formed against the m that is there, without a look at its maximum, and m follows with the next tile where
        // their sum shows that it lags by more than 2^8 (O and l with it).  What overflows meanwhile is not finite in O
        // and is computed once more below.
        // (A wait that gave up sets the abort flag, with which all others give up too: the item's key tiles run through on
        // what is there, then the role ends at the wait for their products.)
        const int t = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_t = tmem + ((uint32_t)(quarter * 32) << 16), o_t = lane_t + 256u + 128u * t;
        const uint32_t s_full = smem_u32(&bar.s_full[t][0]);
        // the item's first key tile, this row tile's key tiles so far, the uses of o_done
        uint32_t g0 = 0, n = 0, n_before = 0, n_last = 0;
        uint32_t s[64];
        const auto load = [&](uint32_t n) {  // starts the load of this row tile's n-th S
            pp_wait(s_full + 8u * (n & 1u), n >> 1 & 1u, a.err, abort);
            tc_fence_after();
            const uint32_t s_t = lane_t + 128u * t + 64u * (n & 1u);
            pp_ld32(s_t, s);
            pp_ld32(s_t + 32, s + 32);
        };
        Item it;
        for (int k = 0; item_at(k, it); g0 += it.n_kt, ++k) {
            const int n_rows = t ? it.n_rows[1] : it.n_rows[0], nk = t ? it.nk[1] : it.nk[0];
            if (n_rows == 0) continue;
            // keys 0 .. sees - 1 of the item are this row's
            const int jr = r / a.pack, sees = it.sees + t * tile_rows + jr;
            const int clean = min(it.sees + t * tile_rows, it.keys) / kPpKeys;  // key tiles that all rows see in full
            // Lanes without a row of the item (the next request's rows, or what lay in shared memory where the heads of a
            // tile do not divide 128) take no part in the warp's votes: m stays 0, their sums are not looked at.
            const bool mine = r < n_rows * a.pack;
            // m in the units of S, neg = -m scale, the last tile's sum and the largest from which m followed
            float m = mine ? -INFINITY : 0.f, l = 0.f, neg = 0.f, last = 0.f, most = 0.f;
            bool big = false;                                     // s scale - m in one step would keep what m lost
            // (The key tiles' loop twice: with narrow requests' part as a branch of one loop, the others took 4 to 7 % more.)
            const auto key_tiles = [&](auto narrow) __attribute__((always_inline)) {
                constexpr bool kNarrow = decltype(narrow)::value;
                for (int j = 0; j < nk; ++j, ++n) {
                    const uint32_t b = n & 1u, s_t = lane_t + 128u * t + 64u * b;
                    load(n);
                    const bool slow = __any_sync(kFull, last > kPpGrown || m == -INFINITY);
                    pp_wait_ld32(s);
                    pp_wait_ld32(s + 32);
                    if (j >= clean) {
                        const int valid = min(sees, it.keys) - j * kPpKeys;
#pragma unroll
                        for (int x = 0; x < 64; ++x)
                            if (x >= valid) s[x] = 0xff800000u;
                    }
                    if (slow) {
                        float top = -INFINITY;
#pragma unroll
                        for (int x = 0; x < 64; x += 2)
                            top = pp_max3(top, __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
                        // The factor in two halves: sums of up to 2^128 have to come down to 1, and exp2 ends at 2^-126.
                        float alpha = 1.f;
                        if (m == -INFINITY) {  // no key seen so far: O and l are 0
                            m = top;
                        } else if (last > kPpGrown) {
                            const float to = fmaxf(top, m + __log2f(last) / a.scale_log2);
                            alpha = cw_exp2(0.5f * ((m - to) * a.scale_log2));
                            m = to;
                            l = l * alpha * alpha;
                            most = fmaxf(most, last);
                        }
                        if (__any_sync(kFull, alpha != 1.f)) {  // (not in an item's first tile)
                            // O: once the P V so far are done (the next S was issued behind them)
                            if (j + 1 < nk)
                                pp_wait(s_full + 8u * (b ^ 1u), (n + 1) >> 1 & 1u, a.err, abort);
                            else
                                wait(&bar.o_done[t][0], n_before);
                            tc_fence_after();
#pragma unroll 1
                            for (int x = 0; x < D; x += 16) {
                                float o[16];
                                tmem_ld16(o_t + x, o);
                                uint32_t w[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha * alpha);
                                pp_st16(o_t + x, w);
                            }
                        }
                        neg = -cw_base(m) * a.scale_log2;
                        big = __any_sync(kFull, fabsf(neg) > 16384.f);
                        if (big) neg = 0.f;
                    }
                    if (big) {
#pragma unroll
                        for (int x = 0; x < 64; ++x) s[x] = __float_as_uint(__uint_as_float(s[x]) - cw_base(m));
                    }
                    const uint64_t scale2 = pp_pair(a.scale_log2, a.scale_log2), neg2 = pp_pair(neg, neg);
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int x = 0; x < 64; x += 32) {
                        uint32_t w[16], low[16];  // (low: of a narrow request's weights, what bf16 leaves of them)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float p0, p1;
                            const uint64_t sp =
                                pp_pair(__uint_as_float(s[x + 2 * e]), __uint_as_float(s[x + 2 * e + 1]));
                            pp_unpair(pp_fma2(sp, scale2, neg2), p0, p1);
                            p0 = cw_exp2(p0), p1 = cw_exp2(p1);
                            w[e] = cw_pack(p0, p1);
                            float *const of = sum + 2 * (e & 1);
                            if constexpr (kNarrow) {
                                low[e] = cw_pack(p0 - cw_lower(w[e]), p1 - cw_upper(w[e]));
                                of[0] += p0, of[1] += p1;
                            } else {  // l sums what is used: one weight above all others leaves its value as it is
                                pp_add_bf16(of[0], of[1], w[e]);
                            }
                        }
                        pp_st16(s_t + x / 2, w);
                        if constexpr (kNarrow) pp_st16(s_t + 32 + x / 2, low);
                    }
                    last = mine ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
                    l += last;
                    if (j >= clean) {
                        // V rows past the item's last key: zero, once they have landed
                        const int here = it.keys - j * kPpKeys;
                        if (here < kPpKeys) {
                            const uint32_t v = g0 + j, st = v % L::kStages;
                            const bool landed = wait(&bar.full[1][st], v / L::kStages);
                            const int c = r / kPpKeys, vr = r % kPpKeys;  // (64 rows of up to two blocks)
                            if (landed && vr >= here && c < L::kAtoms)
#pragma unroll
                                for (int x = 0; x < 8; ++x)
                                    *reinterpret_cast<uint4 *>(sm + L::kV + st * L::kTile + c * kPpKv + vr * 128 +
                                                               x * 16) = make_uint4(0, 0, 0, 0);
                            fence_proxy_async_smem();
                        }
                    }
                    pp_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_full[t][b]);
                }
            };
            if (it.narrow)
                key_tiles(std::true_type());
            else
                key_tiles(std::false_type());
            // ---- the item's output ----
            const int row = it.row + t * tile_rows + jr, head = it.vh * a.pack + r % a.pack;
            const int64_t out_at = mine ? (int64_t)row * a.ld_out + (int64_t)head * D : -1;
            uint8_t *const stage = sm + L::kOut + warp * (32 * 80);
            const int64_t at = (int64_t)it.part * a.vheads + (int64_t)it.vh * (2 * kPpRows) + t * kPpRows + r;
            float *const part = a.part + at * D;
            bool bad = false;
            if (nk > 0) {
                if (nk >= 2) wait(&bar.o_done[t][0], n_before++);
                if (!__all_sync(kFull, wait(&bar.o_done[t][1], n_last++))) break;  // (gave up)
                tc_fence_after();
                const float inv = 1.f / l;
                const uint64_t inv2 = pp_pair(inv, inv);
                uint64_t zero = 0;  // 0 times every component: NaN if one is not finite
                bf16 *to[4];        // where this lane writes, of rows 8 z + lane / 4
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int64_t at = __shfl_sync(kFull, out_at, 8 * z + (lane >> 2));
                    to[z] = at >= 0 ? a.out + at + (lane & 3) * 8 : nullptr;
                }
#pragma unroll
                for (int x = 0; x < D; x += 32) {
                    uint32_t o[32];
                    pp_ld32(o_t + x, o);
                    pp_wait_ld32(o);
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        zero = pp_fma2(pp_pair(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), 0ull, zero);
                    if (it.part < 0) {  // by way of shared memory: four lanes write 64 bytes of a row
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float f0, f1;
                            pp_unpair(pp_mul2(pp_pair(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), inv2),
                                      f0, f1);
                            w[e] = cw_pack(f0, f1);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4 *>(stage + lane * 80)[e] =
                                make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                        __syncwarp();
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const uint4 v =
                                *reinterpret_cast<const uint4 *>(stage + (8 * z + (lane >> 2)) * 80 + (lane & 3) * 16);
                            if (to[z]) *reinterpret_cast<uint4 *>(to[z] + x) = v;
                        }
                        __syncwarp();
                    } else if (mine) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4 *>(part + x + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                float z0, z1;
                pp_unpair(zero, z0, z1);
                bad = z0 != 0.f || z1 != 0.f;
                tc_fence_before();
            } else if (mine) {  // a part of the keys of which this tile sees none
                for (int x = 0; x < D; x += 4) *reinterpret_cast<uint4 *>(part + x) = make_uint4(0, 0, 0, 0);
            }
            if (mine && it.part >= 0)
                *reinterpret_cast<float2 *>(a.part_ml + 2 * at) = make_float2(m * a.scale_log2, l);
            unsigned todo = __ballot_sync(kFull, mine && (bad || (l - l) != 0.f));
            if (todo) {
                // Rows that are not finite and might not have to be: where a tile's weights outgrew m, and where (no score but)
                // a value is not finite that the tiles held and that is not the row's to see.
                const bool jumped = fmaxf(most, last) > kPpOver;
                const int odd = pp_last_odd<D>(a, a.plan + it.at, max(it.sees + t * tile_rows, 0),
                                               min(nk * kPpKeys, it.keys), it.vh / a.per_kv);
                todo &= __ballot_sync(kFull, jumped || ((l - l) == 0.f && sees <= odd));
            }
            // (key by key over what they see)
            for (; todo && !__any_sync(kFull, *abort != 0); todo &= todo - 1) {
                const int rr = quarter * 32 + __ffs(todo) - 1;
                const int row2 = it.row + t * tile_rows + rr / a.pack, head2 = it.vh * a.pack + rr % a.pack;
                const int seen = min(it.sees + t * tile_rows + rr / a.pack, it.keys);
                float m2, l2, o2[8];
                pp_row<D>(a, a.q + (int64_t)row2 * a.ld_q + (int64_t)head2 * D, a.plan + it.at, seen, it.vh / a.per_kv,
                          m2, l2, o2, abort + 1);
                const int64_t at2 = at - r + rr;
                if (lane < D / 8) {
                    if (it.part < 0) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) o2[e] /= l2;
                        store16(a.out + (int64_t)row2 * a.ld_out + (int64_t)head2 * D + lane * 8, o2);
                    } else {
                        store16(a.part + at2 * D + lane * 8, o2);
                        store16(a.part + at2 * D + lane * 8 + 4, o2 + 4);
                        if (lane == 0) *reinterpret_cast<float2 *>(a.part_ml + 2 * at2) = make_float2(m2, l2);
                    }
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kPpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch_prompts(const PagedAttn &p, const int32_t *hp, const int32_t *dp, float *part, float scale_log2,
                           unsigned *err, int *launches, cudaStream_t st) {
    using L = PpLayout<D>;
    cudaError_t e = max_smem_once((const void *)paged_prompt_kernel<D>, (int)L::kBytes);
    if (e != cudaSuccess) return e;
    PpArgs a;
    a.q = reinterpret_cast<const bf16 *>(p.q), a.layer = reinterpret_cast<const bf16 *>(p.layer);
    a.out = reinterpret_cast<bf16 *>(p.out), a.ld_q = p.ld_q, a.ld_out = p.ld_out, a.slots = hp[G_SLOTS];
    a.plan = dp, a.items = reinterpret_cast<const int4 *>(dp + hp[G_O_PITEMS]), a.deal = dp + hp[G_O_DEAL];
    a.pack = hp[G_PACK], a.vheads = hp[G_HEADS] / a.pack, a.kv_heads = hp[G_KV_HEADS];
    a.per_kv = a.vheads / a.kv_heads, a.box = hp[G_BOX], a.scale_log2 = scale_log2, a.err = err;
    a.part = part, a.part_ml = part + (int64_t)hp[G_PPARTS] * a.vheads * D;
    CUtensorMap tmq, tmkv;  // q as [row][head][component], the layer as [K|V][head][slot][component]
    const uint64_t qdims[3] = {(uint64_t)D, (uint64_t)hp[G_HEADS], (uint64_t)hp[G_ROWS]};
    const uint64_t qstrides[2] = {(uint64_t)D * 2, (uint64_t)p.ld_q * 2};
    const uint32_t qbox[3] = {64, (uint32_t)a.pack, (uint32_t)(kPpRows / a.pack)};
    const uint64_t row = D * 2, dims[4] = {(uint64_t)D, (uint64_t)a.slots, (uint64_t)a.kv_heads, 2};
    const uint64_t strides[3] = {row, row * (uint64_t)a.slots, row * (uint64_t)a.slots * (uint64_t)a.kv_heads};
    const uint32_t box[4] = {64, (uint32_t)a.box, 1, 1};
    if (!encode_tensor_map(&tmq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.q, qdims, qstrides, qbox,
                           CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tensor_map(&tmkv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p.layer, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    const int grid = (int)std::min<int64_t>((int64_t)hp[G_PITEMS] * a.vheads, hp[G_SMS]);
    ++*launches;
    e = launch_pdl(paged_prompt_kernel<D>, dim3((unsigned)grid), dim3(kPpThreads), L::kBytes, st, tmq, tmkv, a);
    if (e != cudaSuccess || !hp[G_PJOINS]) return e;
    ++*launches;
    const int4 *joins = reinterpret_cast<const int4 *>(dp + hp[G_O_PJOINS]);
    const JoinArgs j = {a.part, a.part_ml, joins, p.out, p.ld_out, a.vheads, a.pack};
    return launch_pdl(paged_join_kernel<bf16, D>, dim3((unsigned)hp[G_PJOINS] * a.vheads, (unsigned)hp[G_PJOINROWS]),
                      dim3(128), 0, st, j);
}

}  // namespace

namespace {

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
    float *const ppart = a.part_ml + (int64_t)hp[G_PARTS] * a.kv_heads * 2;
    *launches = 0;
    cudaError_t e = cudaSuccess;
    if constexpr (sizeof(T) == 2 && D >= 64)
        if (hp[G_PITEMS]) {
            e = launch_prompts<D>(p, hp, dp, ppart, a.scale_log2, err, launches, st);
            if (e != cudaSuccess) return e;
        }
    const int32_t *at = dp + hp[G_O_ITEMS];
    for (int c = 0; c < kClasses && e == cudaSuccess; ++c) {
        a.items = reinterpret_cast<const int4 *>(at), a.n_items = hp[G_ITEMS + c];
        at += 8 * (int64_t)a.n_items;
        if (!a.n_items) continue;
        a.beside = (*launches)++ > 0;
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
    return launch_pdl(paged_join_kernel<T, D>, dim3((unsigned)hp[G_JOINS] * a.kv_heads, (unsigned)hp[G_JOINROWS]),
                      dim3(128), 0, st, j);
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
