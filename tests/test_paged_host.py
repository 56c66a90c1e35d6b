"""Host side of the paged K/V cache: plans, sizes and refusals.  No GPU."""

import ctypes as C

import numpy as np
import pytest

from iteration_level_scheduling_gb300 import build
from oracle import paged


@pytest.fixture(scope="module")
def native():
    build.build()
    from iteration_level_scheduling_gb300 import native as n
    return n


def batch(native, dtype=1, heads=8, kv_heads=2, d=64, page=16, n_pages=10, n=(3,), c=(40,), table=((7, 2, 5),), **over):
    n, c, t = np.array(n, np.int32), np.array(c, np.int32), np.array(table, np.int32)
    b = native.PagedBatch(dtype, heads, kv_heads, d, page, len(n), n_pages, t.shape[1], n.ctypes.data, c.ctypes.data,
                          t.ctypes.data)
    b._keep = (n, c, t)
    for k, v in over.items():
        setattr(b, k, v)
    return b


def words(native, **kw):
    return native.lib.orca_paged_plan_words(None, C.byref(batch(native, **kw)))


def plan(native, **kw):
    b = batch(native, **kw)
    w = native.lib.orca_paged_plan_words(None, C.byref(b))
    assert w > 0
    buf = np.zeros(w, np.int32)
    assert native.lib.orca_paged_plan_build(None, C.byref(b), buf.ctypes.data, w) == 0
    return buf


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dtype=-1), dict(heads=0), dict(heads=7), dict(heads=1026), dict(kv_heads=0), dict(kv_heads=16),
    dict(kv_heads=3), dict(d=48), dict(d=256), dict(page=0), dict(page=8), dict(page=24), dict(page=-16),
    dict(n_pages=0), dict(n_pages=2 ** 27), dict(n_pages=2 ** 40), dict(n=(-1,)), dict(c=(-1,)),
    dict(n=(9,)), dict(c=(46,)),                # a fourth page is needed, the table has three
    dict(table=((7, 2, 10),)), dict(table=((7, -1, 5),)),
    dict(n=(2 ** 31 - 1,), c=(2 ** 31 - 1,)), dict(n_req=0), dict(n_req=-1), dict(table_ld=0), dict(table_ld=2),
    dict(n_input=None), dict(ctx_len=None), dict(page_table=None),
    dict(n=(150,), c=(20,), table=(tuple(range(10)) + (0,),)),  # more positions than the layer has slots
])
def test_plan_refusals(native, kw):
    assert words(native, **kw) == native.ERR_INVALID
    buf = np.zeros(4096, np.int32)
    assert native.lib.orca_paged_plan_build(None, C.byref(batch(native, **kw)), buf.ctypes.data, 4096) == \
        native.ERR_INVALID
    assert not buf.any()


def test_plan_accepts_what_is_not_used(native):
    """Pages behind the last position and all of a request without rows are not looked at."""
    assert words(native, table=((7, 2, 5, -9),)) > 0
    assert words(native, n=(3, 0), c=(40, -5), table=((7, 2, 5), (-1, -1, -1))) > 0
    assert words(native, n=(0,), c=(0,), table=((-1,),)) > 0
    assert words(native, page=1 << 20, n_pages=2000) > 0
    assert words(native, n=(1, 1), c=(40, 40), table=((7, 2, 5), (7, 2, 6))) > 0  # shared pages


def test_null_and_short_buffers(native):
    b = batch(native)
    w = native.lib.orca_paged_plan_words(None, C.byref(b))
    buf = np.zeros(w, np.int32)
    assert native.lib.orca_paged_plan_words(None, None) == native.ERR_INVALID
    assert native.lib.orca_paged_plan_build(None, C.byref(b), None, w) == native.ERR_INVALID
    assert native.lib.orca_paged_plan_build(None, C.byref(b), buf.ctypes.data, w - 1) == native.ERR_INVALID
    assert not buf.any()
    assert native.lib.orca_paged_workspace_bytes(None) == native.ERR_INVALID
    assert native.lib.orca_paged_workspace_bytes(np.zeros(64, np.int32).ctypes.data) == native.ERR_INVALID


def test_operators_need_an_engine(native):
    p = plan(native)
    assert native.lib.orca_op_paged_append(None, 16, 768, 16, p.ctypes.data, 16, None, 0, 0, 0, 16, 512) == \
        native.ERR_INVALID
    assert native.lib.orca_op_paged_attention(None, 16, 512, 16, p.ctypes.data, 16, 0.0, 16, 16, 512) == \
        native.ERR_INVALID


def test_oracle_by_hand():
    x = np.arange(8, dtype=np.float64).reshape(1, 1, 8)
    turn = np.array([[0.0, 1.0, 1.0, 0.0]])  # pair 0 by a quarter, pair 1 not at all
    assert paged.rotate(x, turn, 4, False)[0, 0].tolist() == [-2, 1, 0, 3, 4, 5, 6, 7]
    assert paged.rotate(x, turn, 4, True)[0, 0].tolist() == [-1, 0, 2, 3, 4, 5, 6, 7]
    assert paged.slots([7, 2], 16, 14, 4).tolist() == [126, 127, 32, 33]
    # two keys of equal score, the second row alone sees both
    q, k = np.ones((2, 2, 1)), np.ones((1, 2, 1))
    out, spread = paged.attention(q, k, np.array([[[1.0], [3.0]]]), 0, 1.0)
    assert out[:, :, 0].tolist() == [[1, 1], [2, 2]] and spread[1, 0, 0] == pytest.approx(np.sqrt(0.5))
    # a rotation keeps products of rows at equal distance
    g = np.random.default_rng(0)
    a, b = g.standard_normal((1, 1, 32)), g.standard_normal((1, 1, 32))
    t = paged.rope_table(50, 24)
    for nb in (False, True):
        p = [(paged.rotate(a, t[i:i + 1], 24, nb) * paged.rotate(b, t[i + 7:i + 8], 24, nb)).sum() for i in (0, 13, 40)]
        assert np.ptp(p) < 1e-5


# words of a plan's header (k_paged.cu)
O_ROWS, O_REQS, O_TILES, ITEMS, PARTS, JOINS, JOINROWS, O_ITEMS, O_JOINS = 10, 11, 12, 14, 17, 18, 19, 20, 21
PITEMS, PPARTS, PJOINS, PJOINROWS, O_PITEMS, O_PJOINS, PACK, BOX = 22, 23, 24, 25, 26, 27, 28, 29
O_DEAL = 30


def cover(native, p, n, c, table, page, group, kv_heads):
    """What a plan's items read and write: every row and head sees its keys once, and nothing leaves its buffer."""
    words, rows = len(p), sum(n)
    first = np.concatenate([[0], np.cumsum(n)])
    req_of = np.repeat(np.arange(len(n)), n)
    keys_of, written = {}, {}  # by (row, head of the tile or of the group): spans of keys, partial columns

    def keys_ok(i, tile, keys):
        k0 = 16 * (tile - int(p[p[O_REQS] + i]))
        assert keys >= 1 and 0 <= k0 and k0 + keys <= c[i] + n[i]
        slots = p[tile:tile + (keys + 15) // 16]
        assert tile + len(slots) <= words
        assert (slots == paged.slots(table[i], page, k0, keys)[::16] // 16).all()
        return k0

    at = p[O_ITEMS]
    for cl in range(3):
        for r in p[at:at + 8 * p[ITEMS + cl]].reshape(-1, 8):
            tile, keys, row0, col0, cols, last0, part = (int(x) for x in r[:7])
            i = int(req_of[row0])
            assert row0 == first[i] and 1 <= cols <= 8 << cl and col0 + cols <= n[i] * group
            k0 = keys_ok(i, tile, keys)
            assert last0 == c[i] - k0 and (part < 0 or part + (8 << cl) <= p[PARTS])
            for x in range(cols):
                j = (col0 + x) // group
                key = (row0 + j, (col0 + x) % group)
                keys_of.setdefault(key, []).append((k0, k0 + max(0, min(keys, last0 + j + 1))))
                written.setdefault(key, []).append(("c", part + x) if part >= 0 else None)
        at += 8 * p[ITEMS + cl]
    pack, box = int(p[PACK]), int(p[BOX])
    assert group % pack == 0 and box % 16 == 0 and 64 % box == 0 and page % box == 0
    for r in p[p[O_PITEMS]:p[O_PITEMS] + 8 * p[PITEMS]].reshape(-1, 8):
        tile, keys, row0, nr, sees, part = (int(x) for x in r[:6])
        i, per = int(req_of[row0]), 128 // pack
        assert 1 <= nr <= 2 * per and row0 + nr <= first[i + 1]
        k0 = keys_ok(i, tile, keys)
        assert k0 % 64 == 0 and sees == c[i] + row0 - first[i] + 1 - k0 and sees + nr - 1 >= 1
        assert keys <= sees + nr - 1 and (part < 0 or part + 256 <= p[PPARTS])
        for j in range(nr):
            for g in range(group):  # (packed one by one: every head has the item's columns of its own)
                x = j // per * 128 + j % per * pack + (g if pack == group else 0)
                keys_of.setdefault((row0 + j, g), []).append((k0, k0 + max(0, min(keys, sees + j))))
                written.setdefault((row0 + j, g), []).append(("p", part + x) if part >= 0 else None)
    assert len(keys_of) == rows * group
    for (r, g), spans in keys_of.items():
        spans = sorted(s for s in spans if s[0] < s[1])
        assert spans[0][0] == 0 and spans[-1][1] == c[req_of[r]] + r - first[req_of[r]] + 1
        assert all(a[1] == b[0] for a, b in zip(spans, spans[1:]))
    joined = {}
    per = 512 // int(p[4])  # columns that a block joins, if they have few parts
    for kind, off, count, most, unit in (("c", O_JOINS, JOINS, JOINROWS, group), ("p", O_PJOINS, PJOINS, PJOINROWS, pack)):
        for r in p[p[off]:p[off] + 8 * p[count]].reshape(-1, 8):
            row0, col0, cols, parts, part, step, tc = (int(v) for v in r[:7])
            assert p[most] >= (cols if parts >= 16 else -(-cols // per))
            for col in range(cols):
                x = col // tc * 128 + col % tc
                assert x < step
                for g in range(group // unit):
                    key = (row0 + (col0 + col) // unit, g * unit + (col0 + col) % unit if unit == group else g)
                    assert key not in joined
                    joined[key] = [(kind, part + y * step + x) for y in range(parts)]
    for key, w in written.items():
        assert joined.get(key) == w if w[0] is not None else (len(w) == 1 and key not in joined)
    if pack == group:
        flat = [w for ws in written.values() for w in ws if w is not None]
        assert len(flat) == len(set(flat))
    assert native.lib.orca_paged_workspace_bytes(p.ctypes.data) == \
        (int(p[PARTS]) * kv_heads + int(p[PPARTS]) * (group * kv_heads // pack)) * (int(p[4]) + 2) * 4


@pytest.mark.parametrize("seed", range(60))
def test_plans_cover_every_key_once(native, seed):
    g = np.random.default_rng(seed)
    reqs = int(g.integers(1, 12))
    n = [int(g.choice([0, 1, 1, 1, 2, 7, 33, 200])) for _ in range(reqs)]
    c = [int(g.choice([0, 1, 15, 16, 300, 700, 5000])) for _ in range(reqs)]
    n[0] = max(1, n[0])
    page, group, kv = int(g.choice([16, 48, 128])), int(g.choice([1, 3, 8, 17, 40, 70])), int(g.choice([1, 4]))
    need = [-(-(a + b) // page) for a, b in zip(n, c)]
    order, table, at = g.permutation(sum(need)), np.zeros((reqs, max(need)), np.int32), 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    p = plan(native, dtype=seed % 2, heads=group * kv, kv_heads=kv, d=int(g.choice([16, 64, 128])), page=page,
             n_pages=sum(need), n=n, c=c, table=table)
    cover(native, p, n, c, table, page, group, kv)


def test_kernels_of_one_call_start_behind_what_is_in_front_of_it():
    """The first kernel of an attention triggers behind its wait, so the second, which does not wait at its start, finds
    all that was in front of the call; it waits before it ends, so that behind it both have ended."""
    from test_launch_order import body, triggers_behind_wait
    assert triggers_behind_wait("k_paged.cu", "paged_cols_kernel") and triggers_behind_wait("k_paged.cu", "paged_prompt_kernel")
    b = body("k_paged.cu", "paged_cols_kernel")
    assert b.find("if (!a.beside) pdl_wait();") < b.find("a.items[") and b.rfind("if (a.beside) pdl_wait();") > b.find("a.out")
    assert b.find("if (!a.beside) pdl_wait();") < b.find("pdl_trigger();")
    for kernel in ("paged_append_kernel", "paged_append_odd_kernel", "paged_join_kernel"):
        b = body("k_paged.cu", kernel)
        assert 0 <= b.find("pdl_wait();") < b.find("blockIdx")


@pytest.mark.parametrize("heads,kv_heads,n,c", [(40, 8, (1024,) * 4, (1000,) * 4), (16, 2, (2047, 1500, 300), (0, 7, 0)),
                                                (2, 2, (200,), (0,)), (70, 1, (100,), (900,))])
def test_prompt_items_are_dealt_evenly(native, heads, kv_heads, n, c):
    need = max(-(-(a + b) // 16) for a, b in zip(n, c))
    p = plan(native, heads=heads, kv_heads=kv_heads, d=128, n=n, c=c, n_pages=need * len(n),
             table=np.arange(need * len(n)).reshape(len(n), need))
    tile_heads = heads // int(p[PACK])
    total = int(p[PITEMS]) * tile_heads
    blocks = min(152, total)
    first = p[p[O_DEAL]:p[O_DEAL] + blocks + 1]
    entry = p[p[O_DEAL] + blocks + 1:p[O_DEAL] + blocks + 1 + total]
    assert first[0] == 0 and first[-1] == total and (np.diff(first) >= 1).all()
    assert (np.sort(entry) == np.arange(total)).all() and p[O_DEAL] + blocks + 1 + total <= len(p)
    assert (entry[first[:-1]] == np.arange(blocks)).all()  # a block knows its first without reading it
    keys = p[p[O_PITEMS]:p[O_PITEMS] + 8 * p[PITEMS]].reshape(-1, 8)[:, 1]
    cost = -(-keys[entry // tile_heads] // 64) + 3
    load = np.add.reduceat(cost, first[:-1])
    # the longest first to the least busy block: no block is above the mean by more than one item
    assert load.max() <= cost.sum() / blocks + cost.max()
    for a, b in zip(first, first[1:]):
        assert (np.diff(cost[a:b]) <= 0).all()


@pytest.mark.parametrize("dtype,n,c,want", [
    (1, (1, 1), (100, 50), (2, 0, 0)),
    (1, (1, 3), (99, 98), (0, 2, 0)),         # 100 keys beside 101: along with the wider class
    (1, (1, 3), (101, 98), (1, 1, 0)),        # 102 beside 101: a launch of their own
    (1, (1, 7), (106, 100), (0, 0, 2)),
    (1, (1, 3, 7), (150, 60, 120), (0, 0, 3)),  # 63 into 127, then 151 into these 190
    (1, (1, 3, 7), (50, 130, 120), (0, 2, 1)),
    (1, (1, 3, 7), (150, 50, 70), (1, 0, 2)),
    (0, (1, 3), (50, 150), (1, 1, 0)),        # fp32: each its own
])
def test_narrow_requests_go_along_with_wider_ones(native, dtype, n, c, want):
    p = plan(native, dtype=dtype, heads=8, kv_heads=2, d=32, n=n, c=c, n_pages=40,
             table=np.arange(30).reshape(3, 10)[:len(n)])
    assert tuple(p[ITEMS:ITEMS + 3]) == want


@pytest.mark.parametrize("heads,d,n,c,want", [
    (8, 64, (5,), (50,), (0, 0, 0, 1)),                 # 20 columns
    (8, 64, (4,), (50,), (0, 1, 0, 0)),
    (8, 32, (5,), (50,), (0, 0, 1, 0)),
    (8, 64, (5, 4), (50, 51), (0, 0, 0, 2)),            # 55 keys go along with 55
    (8, 64, (5, 4), (50, 52), (0, 1, 0, 1)),            # 56 do not
    (8, 64, (5, 4), (50, 106), (0, 1, 0, 1)),
    (8, 64, (5, 4), (50, 107), (0, 1, 1, 0)),           # twice the prompts' keys: these are tiles, of 64 columns at most
    (8, 64, (17, 4), (50, 140), (0, 1, 0, 1)),          # 68 columns: a prompt whatever is beside it
    (8, 64, (9, 1, 3), (50, 60, 50), (0, 0, 0, 3)),      # 53 into 59, then 61 into 112
    (142, 64, (32,), (50,), (0, 0, 71, 0)),             # 71 heads over one: tiles of a head's rows
    (142, 64, (33,), (50,), (0, 0, 0, 1)),
])
def test_which_requests_are_prompts(native, heads, d, n, c, want):
    p = plan(native, heads=heads, kv_heads=2, d=d, n=n, c=c, n_pages=40, table=np.arange(30).reshape(3, 10)[:len(n)])
    assert tuple(p[ITEMS:ITEMS + 3]) + (p[PITEMS],) == want


def test_tensor_memory_is_taken_once_the_kernel_in_front_has_ended():
    """A kernel in front that triggers ahead of its own allocation would wait for the columns, and they for its end; what
    follows this one starts when all its blocks have theirs."""
    from test_launch_order import body
    b = body("k_paged.cu", "paged_prompt_kernel")
    assert 0 <= b.find("pdl_wait();") < b.find("tmem_alloc(") < b.find("__syncthreads();") < b.find("pdl_trigger();")


def test_a_wait_that_gave_up_ends_the_softmax_role():
    """Of the prompt kernel, once a wait has run out: the role ends at the item's last wait, in front of its output, no row
    is computed key by key (which takes seconds over long contexts and holds up the other waits' limits), and values that
    may still be landing are left alone."""
    from test_launch_order import body
    b = body("k_paged.cu", "paged_prompt_kernel")
    b = b[b.index("warp < kPpTma)"):]
    end = b.index("if (!__all_sync(kFull, wait(&bar.o_done[t][1], n_last++))) break;")
    assert end < min(b.index("a.out"), b.index("part + x"), b.index("a.part_ml"))
    assert b[end:].count("wait(") == 1  # the last of the item's waits
    loop = b.index("pp_row<D>")
    assert b[b.rindex("for (", 0, loop):loop].count("__any_sync(kFull, *abort != 0)") == 1
    zero = b.index("make_uint4(0, 0, 0, 0)")
    assert "landed = wait(&bar.full[1]" in b[:zero] and "if (landed &&" in b[b.index("landed = "):zero]


@pytest.mark.parametrize("seed", range(20))
def test_narrow_requests_are_marked_in_every_launch(native, seed):
    """Up to 16 rows x heads of a key/value head, whichever class they go along with: weights of 16 bits."""
    g = np.random.default_rng(100 + seed)
    n = [int(x) for x in g.choice([1, 1, 2, 3, 4, 5, 9, 16, 17, 40, 150], int(g.integers(2, 9)))]
    c = [int(x) for x in g.choice([0, 20, 300, 2000], len(n))]
    group, need = int(g.choice([1, 3, 4, 5, 8, 16, 71])), [-(-(a + b) // 16) for a, b in zip(n, c)]
    first, table = np.concatenate([[0], np.cumsum(need)]), np.zeros((len(n), max(need)), np.int32)
    for i, m in enumerate(need):
        table[i, :m] = first[i] + np.arange(m)
    p = plan(native, heads=2 * group, kv_heads=2, d=int(g.choice([16, 64, 128])), n=n, c=c, n_pages=sum(need), table=table)
    req_of, seen = np.repeat(np.arange(len(n)), n), set()
    for off, count, mark in ((O_ITEMS, p[ITEMS:ITEMS + 3].sum(), 7), (O_PITEMS, p[PITEMS], 6)):
        for r in p[p[off]:p[off] + 8 * count].reshape(-1, 8):
            i = int(req_of[r[2]])
            assert r[mark] == (n[i] * group <= 16)
            seen.add(i)
    assert seen == set(range(len(n)))
