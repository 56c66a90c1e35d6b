"""The paged K/V cache on the GPU: append with rotated positions and attention over
the pages, against the float64 oracle (oracle/paged.py).

Tolerances.  u is half a step of the type (bf16 2^-8, fp32 2^-24).
Append: a rotated component is a c - b s in fp32, two products and a sum (2^-24
of |a c| + |b s| each at most), then rounded once to the type: u |ref| + 2^-22
(|a c| + |b s|).  What is not rotated is exact.
Attention: a score is a sum of D products with a running rounding of 2^-23 at
most each (tensor cores cut sums off instead of rounding), (D + 16) 2^-23 sum |q_i
k_i| scale, and moves a weight by that factor; numerator and denominator both
move: 2 of it times max |v|, and 2^-20 for the exponential (its argument is held
to 2^-24 of its size, which the score's term covers too).  bf16: weights enter the second product rounded
to bf16, independently of each other, |d_t| <= 2^-8, so that the output moves by
sum w_t d_t (v_t - out): more than 7 * 2^-8 sqrt(sum w_t^2 (v_t - out)^2) has a
probability of 2 exp(-24.5) = 5e-11 (Hoeffding).  Sums over T keys: T 2^-23
relative at most.  fp32: the products of parts of 11 bits leave 2^-21 of each
product.  Then u |ref|."""

import numpy as np
import pytest
import torch

from oracle import paged

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TYPES = [("bf16", 128), ("bf16", 64), ("bf16", 32), ("bf16", 16), ("fp32", 128), ("fp32", 64), ("fp32", 32),
         ("fp32", 16)]


@pytest.fixture(scope="module")
def native():
    from iteration_level_scheduling_gb300 import build
    build.build()
    from iteration_level_scheduling_gb300 import native as n
    return n


@pytest.fixture(scope="module")
def eng(native):
    e = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None,
                      torch.cuda.current_stream().cuda_stream)
    yield e
    e.close()


def rounded(x, dtype):
    """float32 values of the type."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TD[dtype]).float().numpy()


def limits(dtype, q, k, v, c, scale=None, equal=False):
    """The oracle's output for q [n, heads, d] over k, v [kv_heads, keys, d], and what it may be off by."""
    heads, d = q.shape[1:]
    group, scale = heads // k.shape[0], scale or 1 / np.sqrt(d)
    ref, spread = paged.attention(q, k, v, c, scale)
    fin = np.abs(np.where(np.isfinite(k), k, 0))  # (a key of -inf has no weight)
    size = 0 if equal else max((np.abs(q[:, h]) @ fin[h // group].T).max() for h in range(heads)) * scale
    tol = 2 * (d + 16) * 2.0 ** -23 * size + 3 * 2.0 ** -20 + k.shape[1] * 2.0 ** -23
    if dtype == "fp32":
        tol += 2 * 2.0 ** -21 * size + 2.0 ** -21
    lim = U[dtype] * np.abs(ref) + tol * np.abs(v).max()
    return ref, lim + 7 * 2.0 ** -8 * spread if dtype == "bf16" else lim


class Case:
    """Requests (rows, ctx) over pages in random order; every slot that no request covers is NaN."""

    def __init__(self, native, eng, seed, dtype, heads, kv_heads, d, page, reqs, std=1.0, pad=0, table=None, n_pages=0):
        g = self.g = np.random.default_rng(seed)
        self.native, self.eng, self.dtype, self.page, self.reqs = native, eng, dtype, page, reqs
        self.heads, self.kv_heads, self.d, self.pad = heads, kv_heads, d, pad
        self.n, self.c = [n for n, _ in reqs], [c for _, c in reqs]
        need = [(n + c + page - 1) // page for n, c in reqs]
        self.n_pages = n_pages or sum(need) + 2
        if table is None:
            order, table, at = g.permutation(self.n_pages), np.full((len(reqs), max(need + [1])), -1), 0
            for i, m in enumerate(need):
                table[i, :m] = order[at:at + m]
                at += m
        self.table = np.ascontiguousarray(table, np.int32)
        self.rows, self.H = sum(self.n), heads * d
        self.slots = self.n_pages * page
        self.host = np.full((2, kv_heads, self.slots, d), np.nan, np.float32)
        for (n, c), t in zip(reqs, self.table):
            s = paged.slots(t, page, 0, n + c) if n else np.zeros(0, np.int64)
            self.host[:, :, s] = rounded(g.standard_normal((2, kv_heads, len(s), d)) * std, dtype)
        self.q = rounded(g.standard_normal((self.rows, heads, d)), dtype)
        code = native.DTYPE_BF16 if dtype == "bf16" else native.DTYPE_FP32
        self.plan = eng.paged_plan(code, heads, kv_heads, d, page, self.n_pages, self.n, self.c, self.table)
        self.dplan = torch.from_numpy(self.plan).cuda()
        self.work = torch.full((max(16, eng.paged_workspace_bytes(self.plan)),), 0xFF, dtype=torch.uint8, device="cuda")
        self.upload()

    def padded(self, x, pad):
        """Device rows of x [rows, ...] with `pad` NaN behind each, and two rows of NaN behind the last."""
        x = x.reshape(len(x), int(np.prod(x.shape[1:])))
        t = torch.full((len(x) + 2, x.shape[1] + pad), float("nan"), dtype=TD[self.dtype], device="cuda")
        t[:len(x), :x.shape[1]] = torch.from_numpy(np.ascontiguousarray(x)).cuda().to(TD[self.dtype])
        return t

    def upload(self):
        self.layer = torch.from_numpy(self.host).cuda().to(TD[self.dtype])
        self.dq = self.padded(self.q, self.pad)

    def attention(self, work=None, dplan=None, **kw):
        out = torch.full((self.rows + 2, self.H + self.pad), 768.0, dtype=TD[self.dtype], device="cuda")
        self.eng.op_paged_attention(self.dq.data_ptr(), self.layer.data_ptr(), self.plan,
                                    (self.dplan if dplan is None else dplan).data_ptr(),
                                    (self.work if work is None else work).data_ptr(), out.data_ptr(),
                                    ld_q=self.H + self.pad, ld_out=self.H + self.pad, **kw)
        return out

    def limits(self, scale=None, equal=False):
        """Oracle's output and tolerance of every row (equal: all scores of a row are the same bits)."""
        ref, lim, r = np.zeros((self.rows, self.heads, self.d)), np.zeros((self.rows, self.heads, self.d)), 0
        for (n, c), t in zip(self.reqs, self.table):
            if n:
                k, v = self.host[:, :, paged.slots(t, self.page, 0, n + c)]
                ref[r:r + n], lim[r:r + n] = limits(self.dtype, self.q[r:r + n], k, v, c, scale, equal)
            r += n
        return ref, lim

    def check(self, out, **kw):
        ref, lim = self.limits(**kw)
        o = out.float().cpu().numpy()
        assert (o[self.rows:] == 768).all() and (o[:, self.H:] == 768).all()  # what is behind the rows stays
        got = o[:self.rows, :self.H].reshape(ref.shape).astype(np.float64)
        off = np.abs(got - ref)
        assert np.isfinite(got).all() and (off <= lim).all(), float((off / lim).max())


# --------------------------------------------------------------------------- #
# append
# --------------------------------------------------------------------------- #
def append_case(native, eng, seed, dtype, heads, kv_heads, d, page, reqs, rot, neighbours, pad=0, std=1.0):
    s = Case(native, eng, seed, dtype, heads, kv_heads, d, page, reqs)
    W = heads + 2 * kv_heads
    s.qkv = rounded(s.g.standard_normal((s.rows, W, d)) * std, dtype)
    s.dqkv = s.padded(s.qkv, pad)
    s.rot, s.nb, s.apad = rot, neighbours, pad
    s.rope = paged.rope_table(max(n + c for n, c in reqs) + 1, rot)
    s.drope = torch.from_numpy(s.rope).cuda()
    s.q_out = torch.full((s.rows + 2, s.H + pad), 512.0, dtype=TD[dtype], device="cuda")
    return s


def do_append(s, q_out=True, **kw):
    s.eng.op_paged_append(s.dqkv.data_ptr(), s.layer.data_ptr(), s.plan, s.dplan.data_ptr(),
                          q_out=s.q_out.data_ptr() if q_out else 0, rope=s.drope.data_ptr() if s.rot else 0,
                          rope_len=len(s.rope) if s.rot else 0, rot_dim=s.rot, neighbours=s.nb,
                          ld_qkv=s.dqkv.shape[1], ld_q=s.q_out.shape[1], **kw)


def check_append(s, q=True):
    pos = np.concatenate([np.arange(c, c + n) for n, c in s.reqs])
    qk = s.heads + s.kv_heads
    ref = s.qkv.astype(np.float64)
    lim = np.zeros(ref.shape)
    if s.rot:
        ref[:, :qk] = paged.rotate(s.qkv[:, :qk], s.rope[pos], s.rot, s.nb)
        big = np.abs(s.qkv[:, :qk, :s.rot]).max(-1, keepdims=True) * 2  # |a c| + |b s| of any pair of the head
        lim[:, :qk, :s.rot] = U[s.dtype] * np.abs(ref[:, :qk, :s.rot]) + 2.0 ** -22 * big
    if q:
        got = s.q_out.float().cpu().numpy()
        assert (got[s.rows:] == 512).all() and (got[:, s.H:] == 512).all()
        got = got[:s.rows, :s.H].reshape(s.rows, s.heads, s.d)
        assert (np.abs(got - ref[:, :s.heads]) <= lim[:, :s.heads]).all()
    want, tol = s.host.astype(np.float64), np.zeros(s.host.shape)
    r = 0
    for (n, c), t in zip(s.reqs, s.table):
        for j in range(n):
            at = paged.slots(t, s.page, c + j, 1)[0]
            for x in (0, 1):
                h = s.heads + x * s.kv_heads
                want[x, :, at], tol[x, :, at] = ref[r, h:h + s.kv_heads], lim[r, h:h + s.kv_heads]
            r += 1
    got = s.layer.float().cpu().numpy()
    assert (np.isnan(got) == np.isnan(want)).all()  # no other slot is touched
    assert (np.nan_to_num(np.abs(got - want)) <= tol).all()


REQS = [(1, 0), (7, 3), (1, 12), (66, 0), (2, 31), (3, 47), (1, 16), (0, 5), (1, 15)]


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("dtype,d", TYPES)
def test_append(native, eng, dtype, d, neighbours):
    for rot in sorted({0, d, d // 2, 2, 6, d - 2}):
        s = append_case(native, eng, rot, dtype, 6, 3, d, 32, REQS, rot, neighbours, pad=8)
        do_append(s)
        check_append(s)


@pytest.mark.parametrize("heads,kv_heads,page", [(1, 1, 16), (5, 1, 48), (40, 8, 16), (7, 7, 256), (71, 1, 128)])
def test_append_shapes(native, eng, heads, kv_heads, page):
    for dtype in ("bf16", "fp32"):
        s = append_case(native, eng, 3, dtype, heads, kv_heads, 64, page, [(33, 100), (1, 0), (130, 7)], 64, False)
        do_append(s)
        check_append(s)


@pytest.mark.parametrize("rot,neighbours", [(64, False), (20, False), (22, True), (0, False)])
def test_append_in_place_and_without_queries(native, eng, rot, neighbours):
    s = append_case(native, eng, 4, "bf16", 6, 2, 64, 16, REQS, rot, neighbours)
    do_append(s, q_out=False)
    check_append(s, q=False)
    assert (s.q_out == 512).all()
    before = s.dqkv.clone()
    s.eng.op_paged_append(s.dqkv.data_ptr(), s.layer.data_ptr(), s.plan, s.dplan.data_ptr(), q_out=s.dqkv.data_ptr(),
                          rope=s.drope.data_ptr() if rot else 0, rope_len=len(s.rope) if rot else 0, rot_dim=rot,
                          neighbours=neighbours, ld_q=s.dqkv.shape[1])
    assert torch.equal(s.dqkv[:s.rows, s.H:], before[:s.rows, s.H:])
    s.q_out[:s.rows, :s.H] = s.dqkv[:s.rows, :s.H]
    check_append(s)


def test_append_of_infinities_and_nan(native, eng):
    """They stay in their pair."""
    s = append_case(native, eng, 5, "bf16", 2, 1, 64, 16, [(3, 2)], 64, False)
    s.qkv[0, 0, 5], s.qkv[1, 2, 7], s.qkv[2, 3, 9] = np.inf, np.nan, -np.inf
    s.dqkv = s.padded(s.qkv, 0)
    do_append(s)
    q = s.q_out[:3, :128].float().cpu().numpy().reshape(3, 2, 64)
    assert not np.isfinite(q[0, 0, [5, 37]]).any() and np.isfinite(np.delete(q[0, 0], [5, 37])).all()
    at = paged.slots(s.table[0], 16, 3, 2)
    k = s.layer[0, 0, at[0]].float().cpu().numpy()
    assert np.isnan(k[[7, 39]]).all() and np.isfinite(np.delete(k, [7, 39])).all()
    v = s.layer[1, 0, at[1]].float().cpu().numpy()
    assert v[9] == -np.inf and np.isfinite(np.delete(v, 9)).all()


# --------------------------------------------------------------------------- #
# attention
# --------------------------------------------------------------------------- #
EDGES = [(1, c) for c in (0, 1, 14, 15, 16, 17, 31, 32, 47, 63, 64, 65, 127, 128, 255, 256, 300, 511, 512, 700)]


@pytest.mark.parametrize("heads,kv_heads", [(3, 3), (8, 2), (5, 1)])
@pytest.mark.parametrize("dtype,d", TYPES)
def test_single_rows(native, eng, dtype, d, heads, kv_heads):
    s = Case(native, eng, 1, dtype, heads, kv_heads, d, 16, EDGES, pad=8)
    s.check(s.attention())


@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (8, 2), (16, 1), (24, 1), (40, 1), (7, 1), (71, 1)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("fp32", 64), ("fp32", 128)])
def test_shared_heads(native, eng, dtype, d, heads, kv_heads):
    s = Case(native, eng, 2, dtype, heads, kv_heads, d, 48, [(1, 200), (2, 30), (5, 77), (0, 3), (1, 0), (33, 64)])
    s.check(s.attention())


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 144, 256, 1024])
def test_page_sizes(native, eng, page):
    for dtype, d in (("bf16", 128), ("bf16", 64), ("fp32", 32)):
        s = Case(native, eng, page, dtype, 4, 2, d, page, [(1, 900), (1, page - 1), (1, page), (4, page - 2), (150, 333)])
        s.check(s.attention())


@pytest.mark.parametrize("dtype,d", TYPES)
def test_several_rows(native, eng, dtype, d):
    s = Case(native, eng, 3, dtype, 6, 2, d, 16, [(2, 0), (17, 0), (9, 100), (64, 0), (130, 1), (33, 500), (128, 128)])
    s.check(s.attention())


@pytest.mark.parametrize("dtype,d,heads,kv_heads", [("bf16", 128, 4, 4), ("bf16", 128, 8, 1), ("bf16", 64, 5, 1),
                                                     ("bf16", 64, 6, 2), ("bf16", 128, 40, 1), ("fp32", 128, 4, 1),
                                                     ("bf16", 16, 3, 1)])
def test_prompts(native, eng, dtype, d, heads, kv_heads):
    s = Case(native, eng, 4, dtype, heads, kv_heads, d, 32, [(300, 0), (257, 600), (128, 0), (1, 2000), (700, 13)], pad=8)
    s.check(s.attention())


@pytest.mark.parametrize("dtype,d,kv_heads,reqs", [
    ("bf16", 128, 1, [(1, 40000)]), ("bf16", 64, 2, [(1, 30001), (1, 5)]), ("fp32", 64, 1, [(1, 20000)]),
    ("bf16", 128, 1, [(7, 20000), (1, 9000)]), ("bf16", 128, 1, [(70, 9000)]), ("fp32", 128, 1, [(20, 5000)])])
def test_long_contexts(native, eng, dtype, d, kv_heads, reqs):
    s = Case(native, eng, 5, dtype, 4 * kv_heads, kv_heads, d, 64, reqs)
    s.check(s.attention())


@pytest.mark.parametrize("scale", [1.0, 0.03, 1e-30])
def test_scales(native, eng, scale):
    for dtype in ("bf16", "fp32"):
        s = Case(native, eng, 6, dtype, 4, 2, 64, 16, [(1, 333), (3, 40), (140, 20)])
        s.check(s.attention(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 16), ("fp32", 64)])
def test_large_scores(native, eng, dtype, d):
    """Rows that grow along the context: the maximum moves all the time, most weights vanish."""
    s = Case(native, eng, 7, dtype, 4, 2, d, 16, [(1, 700), (9, 200), (200, 100)])
    for (n, c), t in zip(s.reqs, s.table):
        at = paged.slots(t, 16, 0, n + c)
        s.host[0][:, at] = rounded(s.host[0][:, at] * np.linspace(0, 30, n + c)[None, :, None], dtype)
    s.upload()
    s.check(s.attention())


@pytest.mark.parametrize("dtype,d", TYPES)
def test_scores_far_from_zero(native, eng, dtype, d):
    """All scores of a row near the type's lowest or highest values that still have a softmax."""
    for sign in (1.0, -1.0):
        s = Case(native, eng, 8, dtype, 2, 1, d, 16, [(1, 100), (5, 40), (140, 20)])
        s.q[:], big = 0, rounded(np.full(1, 1e18), dtype)[0]
        s.q[..., 0] = sign * big
        for (n, c), t in zip(s.reqs, s.table):
            s.host[0][:, paged.slots(t, 16, 0, n + c)] = 0
            s.host[0][:, paged.slots(t, 16, 0, n + c), 0] = big
        s.upload()
        s.check(s.attention(), equal=True)  # (the mean of the values)


NONFINITE = [("bf16", 128), ("bf16", 64), ("bf16", 32), ("fp32", 64)]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,d", NONFINITE)
def test_values_that_are_not_finite(native, eng, dtype, d, bad):
    """They reach the rows that see their key, and no others, whichever key it is."""
    for reqs, key in (([(1, 100)], 100), ([(9, 50)], 54), ([(150, 60)], 60 + 33), ([(150, 0)], 149), ([(40, 300)], 310)):
        s = Case(native, eng, 9, dtype, 4, 2, d, 16, reqs)
        n, c = reqs[0]
        at = paged.slots(s.table[0], 16, key, 1)[0]
        s.host[1, 1, at, 3] = bad
        s.upload()
        out = s.attention().float().cpu().numpy()[:s.rows, :s.H].reshape(n, 4, d)
        sees = np.arange(n) + c >= key
        hit = np.zeros((n, 4), bool)
        hit[sees, 2:] = True
        assert (~np.isfinite(out[..., 3]) == hit).all()
        assert np.isfinite(out[~hit]).all()
        s.host[1, 1, at, 3] = 0
        ref, lim = s.limits()
        assert (np.abs(out - ref) <= lim)[~hit].all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,d", NONFINITE)
def test_keys_that_are_not_finite(native, eng, dtype, d, bad):
    for reqs, key in (([(1, 100)], 37), ([(9, 50)], 54), ([(150, 60)], 60 + 33), ([(150, 0)], 149)):
        s = Case(native, eng, 10, dtype, 4, 2, d, 16, reqs)
        n, c = reqs[0]
        s.host[0, 0, paged.slots(s.table[0], 16, key, 1)[0], 5] = bad
        s.q[..., 5] = np.abs(s.q[..., 5]) + 1  # (a score of +inf, whose softmax is NaN, not one of -inf)
        s.upload()
        out = s.attention().float().cpu().numpy()[:s.rows, :s.H].reshape(n, 4, d)
        hit = np.zeros((n, 4), bool)
        hit[np.arange(n) + c >= key, :2] = True
        assert np.isnan(out[hit]).all() and np.isfinite(out[~hit]).all()


@pytest.mark.parametrize("dtype,d", NONFINITE)
def test_keys_that_hide_themselves(native, eng, dtype, d):
    """Scores of -inf take their key out; a row of nothing else has no softmax."""
    for reqs in ([(1, 100)], [(9, 50)], [(150, 60)]):
        s = Case(native, eng, 11, dtype, 2, 1, d, 16, reqs)
        n, c = reqs[0]
        s.q[..., 0] = 1.0
        at = paged.slots(s.table[0], 16, 0, n + c)
        hidden = np.arange(n + c) % 3 != 1
        s.host[0][:, at[hidden], 0] = -np.inf
        s.upload()
        s.check(s.attention())
        s.host[0][:, at, 0] = -np.inf
        s.upload()
        assert torch.isnan(s.attention()[:s.rows, :s.H]).all()


def test_empty_batches(native, eng):
    s = Case(native, eng, 12, "bf16", 4, 2, 64, 16, [(0, 5), (0, 0)])
    out = s.attention()
    assert (out == 768).all()
    s = append_case(native, eng, 12, "bf16", 4, 2, 64, 16, [(0, 5), (0, 0)], 64, False)
    do_append(s)
    assert (s.q_out == 512).all() and torch.isnan(s.layer).all()


def test_shared_pages(native, eng):
    """Requests with a common beginning read its pages together; the second writes into pages of its own."""
    table = [[4, 1, 0], [4, 1, 5], [4, 1, 3]]
    s = Case(native, eng, 13, "bf16", 8, 2, 128, 32, [(1, 70), (5, 64), (1, 90)], table=table, n_pages=7)
    s.check(s.attention())
    for at, ok in ((70, True), (69, True), (68, False), (64, False), (63, True)):  # beside rows 64 .. 68 of one page
        a = append_case(native, eng, 13, "bf16", 8, 2, 128, 32, [(1, at), (5, 64)], 128, False)
        a.table = np.array([[4, 1, 0], [4, 1, 0]], np.int32)
        a.plan = eng.paged_plan(1, 8, 2, 128, 32, a.n_pages, a.n, a.c, a.table)
        a.dplan = torch.from_numpy(a.plan).cuda()
        if ok:
            do_append(a)
            continue
        with pytest.raises(native.OrcaError) as e:
            do_append(a)
        assert e.value.code == native.ERR_INVALID
    # the same request's two rows in one slot, by a page that its table names twice
    b = native.Engine.paged_plan(eng, 1, 8, 2, 128, 16, 4, [32], [0], np.array([[1, 1]], np.int32))
    x = torch.zeros(32 * 12 * 128, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(2 * 2 * 64 * 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(native.OrcaError):
        eng.op_paged_append(x.data_ptr(), y.data_ptr(), b, torch.from_numpy(b).cuda().data_ptr())


def test_refusals(native, eng):
    s = append_case(native, eng, 14, "bf16", 4, 2, 64, 16, [(2, 20)], 64, False)
    ok = dict(qkv=s.dqkv.data_ptr(), layer=s.layer.data_ptr(), plan=s.plan, dev_plan=s.dplan.data_ptr(),
              q_out=s.q_out.data_ptr(), rope=s.drope.data_ptr(), rope_len=len(s.rope), rot_dim=64, neighbours=False)
    eng.op_paged_append(**ok)
    for bad in (dict(qkv=0), dict(qkv=ok["qkv"] + 2), dict(layer=0), dict(layer=ok["layer"] + 8), dict(dev_plan=0),
                dict(dev_plan=ok["dev_plan"] + 4), dict(q_out=ok["q_out"] + 8), dict(rope=0), dict(rope=ok["rope"] + 4),
                dict(rope_len=21), dict(rot_dim=66), dict(rot_dim=3), dict(rot_dim=-2), dict(neighbours=2),
                dict(ld_qkv=504), dict(ld_qkv=516), dict(ld_q=248), dict(ld_q=260), dict(ld_qkv=2 ** 31),
                dict(q_out=ok["qkv"]), dict(q_out=ok["qkv"] + 16), dict(q_out=ok["layer"] + 1024),
                dict(qkv=ok["layer"] + 1024), dict(plan=np.zeros(64, np.int32) + s.plan[1])):
        with pytest.raises(native.OrcaError) as e:
            eng.op_paged_append(**{**ok, **bad})
        assert e.value.code == native.ERR_INVALID, bad
    out = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda")
    ok = dict(q=s.q_out.data_ptr(), layer=s.layer.data_ptr(), plan=s.plan, dev_plan=s.dplan.data_ptr(),
              workspace=s.work.data_ptr(), out=out.data_ptr())
    eng.op_paged_attention(**ok)
    for bad in (dict(q=0), dict(q=ok["q"] + 2), dict(layer=0), dict(layer=ok["layer"] + 8), dict(dev_plan=0),
                dict(dev_plan=ok["dev_plan"] + 4), dict(workspace=ok["workspace"] + 8), dict(out=0),
                dict(out=ok["out"] + 8), dict(ld_q=248), dict(ld_q=260), dict(ld_out=248), dict(ld_out=260),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=ok["q"]),
                dict(out=ok["layer"]), dict(plan=np.zeros(64, np.int32) + s.plan[1])):
        with pytest.raises(native.OrcaError) as e:
            eng.op_paged_attention(**{**ok, **bad})
        assert e.value.code == native.ERR_INVALID, bad
    s = Case(native, eng, 14, "bf16", 4, 1, 128, 16, [(1, 30000)])
    if eng.paged_workspace_bytes(s.plan):  # split keys: a workspace is needed
        with pytest.raises(native.OrcaError):
            eng.op_paged_attention(s.dq.data_ptr(), s.layer.data_ptr(), s.plan, s.dplan.data_ptr(), 0, s.dq.data_ptr())


MIX = [(1, 700), (1, 20000), (6, 300), (150, 200), (40, 3000), (1, 0)]


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 64)])
def test_calls_repeat_bit_for_bit(native, eng, dtype, d):
    """Twice in a row, captured and replayed, on a stream of another engine, with work of another call in the
    workspace: the same bits."""
    s = Case(native, eng, 15, dtype, 8, 2, d, 64, MIX)
    first = s.attention()
    s.check(first)
    assert torch.equal(first, s.attention())
    s.work.fill_(0x7F)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        e2 = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None, side.cuda_stream)
    side.wait_stream(torch.cuda.current_stream())
    s.eng = e2
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = s.attention(sync=False)
        for _ in range(3):
            out.zero_()
            graph.replay()
            side.synchronize()
            assert torch.equal(first[:s.rows, :s.H], out[:s.rows, :s.H])
    s.eng = eng
    del graph
    e2.close()


def test_two_streams_share_a_plan(native, eng):
    s = Case(native, eng, 16, "bf16", 8, 2, 128, 64, MIX)
    first = s.attention()
    side = torch.cuda.Stream()
    e2 = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None, side.cuda_stream)
    work2, outs = torch.empty_like(s.work), []
    torch.cuda.synchronize()
    for i in range(6):
        s.eng = e2 if i % 2 else eng
        with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
            outs.append(s.attention(work=work2 if i % 2 else None, sync=False))
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    s.eng = eng
    e2.close()


def test_a_prompt_and_its_tokens(native, eng):
    """As a serving program uses them: a prompt in two chunks, then tokens one by one, against one prompt in 64 bits."""
    heads, kv, d, page, N = 8, 2, 64, 16, 90
    g = np.random.default_rng(17)
    rope = paged.rope_table(N, d)
    drope = torch.from_numpy(rope).cuda()
    for dtype in ("bf16", "fp32"):
        qkv = rounded(g.standard_normal((N, heads + 2 * kv, d)), dtype)
        dqkv = torch.from_numpy(qkv.reshape(N, -1)).cuda().to(TD[dtype])
        layer = torch.full((2, kv, 10 * page, d), float("nan"), dtype=TD[dtype], device="cuda")
        table = g.permutation(10)[None, :6].astype(np.int32)
        out = torch.empty((N, heads * d), dtype=TD[dtype], device="cuda")
        q = torch.empty_like(out)
        for at, n in [(0, 40), (40, 37)] + [(t, 1) for t in range(77, N)]:
            plan = eng.paged_plan(1 if dtype == "bf16" else 0, heads, kv, d, page, 10, [n], [at], table)
            dev = torch.from_numpy(plan).cuda()
            work = torch.empty(max(16, eng.paged_workspace_bytes(plan)), dtype=torch.uint8, device="cuda")
            eng.op_paged_append(dqkv[at:].data_ptr(), layer.data_ptr(), plan, dev.data_ptr(), q_out=q[at:].data_ptr(),
                                rope=drope.data_ptr(), rope_len=N, rot_dim=d, sync=False)
            eng.op_paged_attention(q[at:].data_ptr(), layer.data_ptr(), plan, dev.data_ptr(), work.data_ptr(),
                                   out[at:].data_ptr())
        # rotated rows against the oracle's, then attention over the very rows that were written
        at = paged.slots(table[0], page, 0, N)
        rot = torch.cat([q.view(N, heads, d), layer[0][:, at].transpose(0, 1)], 1).float().cpu().numpy()
        want = paged.rotate(qkv[:, :heads + kv], rope, d, False)
        big = 2 * np.abs(qkv[:, :heads + kv]).max(-1, keepdims=True)
        assert (np.abs(rot - want) <= U[dtype] * np.abs(want) + 2.0 ** -22 * big).all()
        assert torch.equal(layer[1][:, at], dqkv.view(N, -1, d)[:, heads + kv:].transpose(0, 1))
        ref, lim = limits(dtype, rot[:, :heads], rot[:, heads:].transpose(1, 0, 2),
                          qkv[:, heads + kv:].transpose(1, 0, 2), 0)
        got = out.float().cpu().numpy().reshape(N, heads, d)
        assert (np.abs(got - ref) <= lim).all()


def test_slots_beyond_32_bits(native, eng):
    """A layer of more than 2^32 elements, of which the last pages are used."""
    kv, d, page, n_pages = 4, 128, 64, 70000  # 4.6e9 elements, 9 GB
    g = np.random.default_rng(18)
    layer = torch.empty((2, kv, n_pages * page, d), dtype=torch.bfloat16, device="cuda")
    for dtype, heads, reqs in (("bf16", 8, [(1, 300), (5, 100), (150, 40)]),):
        n, c = [a for a, _ in reqs], [b for _, b in reqs]
        need = [-(-(a + b) // page) for a, b in reqs]
        last, at = n_pages - 1 - g.permutation(sum(need)), 0
        table = np.zeros((len(reqs), max(need)), np.int32)
        for i, m in enumerate(need):
            table[i, :m] = last[at:at + m]
            at += m
        plan = eng.paged_plan(1, heads, kv, d, page, n_pages, n, c, table)
        dev = torch.from_numpy(plan).cuda()
        work = torch.empty(max(16, eng.paged_workspace_bytes(plan)), dtype=torch.uint8, device="cuda")
        keys = []
        for i, (a, b) in enumerate(reqs):
            s = torch.from_numpy(paged.slots(table[i], page, 0, a + b)).cuda()
            x = rounded(g.standard_normal((2, kv, a + b, d)), dtype)
            layer[:, :, s] = torch.from_numpy(x).cuda().bfloat16()
            keys.append(x)
        qkv = rounded(g.standard_normal((sum(n), heads + 2 * kv, d)), dtype)
        r = 0
        for i, (a, b) in enumerate(reqs):  # the rows' own keys and values, to be appended
            keys[i][0, :, b:] = qkv[r:r + a, heads:heads + kv].transpose(1, 0, 2)
            keys[i][1, :, b:] = qkv[r:r + a, heads + kv:].transpose(1, 0, 2)
            r += a
        dq = torch.from_numpy(qkv.reshape(len(qkv), -1)).cuda().bfloat16()
        out = torch.empty((sum(n), heads * d), dtype=torch.bfloat16, device="cuda")
        eng.op_paged_append(dq.data_ptr(), layer.data_ptr(), plan, dev.data_ptr())
        eng.op_paged_attention(dq.data_ptr(), layer.data_ptr(), plan, dev.data_ptr(), work.data_ptr(), out.data_ptr(),
                               ld_q=dq.shape[1])
        got, r = out.float().cpu().numpy().reshape(-1, heads, d), 0
        for i, (a, b) in enumerate(reqs):
            ref, lim = limits(dtype, qkv[r:r + a, :heads], *keys[i], b)
            assert (np.abs(got[r:r + a] - ref) <= lim).all()
            r += a


def test_steps_queued_behind_one_another(native, eng):
    """Several layers' appends and attentions, over growing contexts, in one graph: the bits of the same calls one by
    one.  (Kernels start early behind the ones in front of them; the next plan's rows are read behind the wait.)"""
    heads, kv, d, page, steps, B = 8, 2, 128, 16, 6, 5
    g = np.random.default_rng(19)
    ctx0 = [3, 700, 40, 15, 1300]
    need = [-(-(c + steps) // page) for c in ctx0]
    table, at = np.zeros((B, max(need)), np.int32), 0
    order = g.permutation(sum(need))
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    rope = torch.from_numpy(paged.rope_table(2000, d)).cuda()
    first = torch.from_numpy(rounded(g.standard_normal((2, kv, sum(need) * page, d)), "bf16")).cuda().bfloat16()
    plans = [eng.paged_plan(1, heads, kv, d, page, sum(need), [1] * B, [c + s for c in ctx0], table) for s in range(steps)]
    devs = [torch.from_numpy(p).cuda() for p in plans]
    work = torch.empty(max(max(16, eng.paged_workspace_bytes(p)) for p in plans), dtype=torch.uint8, device="cuda")
    qkv = [torch.from_numpy(rounded(g.standard_normal((B, (heads + 2 * kv) * d)), "bf16")).cuda().bfloat16()
           for _ in range(steps)]

    def run(e, sync):
        layer, q = first.clone(), torch.empty((B, heads * d), dtype=torch.bfloat16, device="cuda")
        outs = [torch.empty_like(q) for _ in range(steps)]

        def go():
            for s in range(steps):
                e.op_paged_append(qkv[s].data_ptr(), layer.data_ptr(), plans[s], devs[s].data_ptr(), q_out=q.data_ptr(),
                                  rope=rope.data_ptr(), rope_len=2000, rot_dim=d, sync=sync)
                e.op_paged_attention(q.data_ptr(), layer.data_ptr(), plans[s], devs[s].data_ptr(), work.data_ptr(),
                                     outs[s].data_ptr(), sync=sync)
        return go, layer, outs

    go, layer, want = run(eng, True)
    go()
    side = torch.cuda.Stream()
    e2 = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None, side.cuda_stream)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go2, layer2, got = run(e2, False)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            go2()
        for _ in range(20):
            layer2.copy_(first)
            for o in got:
                o.zero_()
            graph.replay()
            side.synchronize()
            assert torch.equal(layer, layer2) and all(torch.equal(a, b) for a, b in zip(want, got))
    del graph
    e2.close()


@pytest.mark.parametrize("d", [64, 128])
def test_beside_the_engines_own_attention(native, eng, d):
    """Pages in a row are a request's contiguous slots: the two attentions over one layer agree."""
    heads, reqs, page = 4, [(1, 200), (40, 7), (1, 0), (130, 64)], 16
    n, c = [a for a, _ in reqs], [b for _, b in reqs]
    need = [-(-(a + b) // page) for a, b in reqs]
    begin = np.concatenate([[0], np.cumsum(need)])[:-1]
    table = np.zeros((len(reqs), max(need)), np.int32)
    for i, m in enumerate(need):
        table[i, :m] = begin[i] + np.arange(m)
    s = Case(native, eng, 20, "bf16", heads, heads, d, page, reqs, table=table, n_pages=sum(need))
    qkv = rounded(s.g.standard_normal((s.rows, 3, heads, d)), "bf16")
    s.q, r = qkv[:, 0].copy(), 0
    dq = torch.from_numpy(qkv.reshape(s.rows, -1)).cuda().bfloat16()
    s.eng.op_paged_append(dq.data_ptr(), s.layer.data_ptr(), s.plan, s.dplan.data_ptr())
    for (a, b), t in zip(reqs, table):
        s.host[:, :, paged.slots(t, page, b, a)] = qkv[r:r + a, 1:].transpose(1, 2, 0, 3)
        r += a
    out, own = (torch.full((s.rows + 2, heads * d), 768.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s.eng.op_paged_attention(dq.data_ptr(), s.layer.data_ptr(), s.plan, s.dplan.data_ptr(), s.work.data_ptr(),
                             out.data_ptr(), ld_q=dq.shape[1])
    e2 = native.Engine(1, heads * d, heads, 64, 64, 4096, native.DTYPE_BF16, 1024, 8, 64, None,
                       torch.cuda.current_stream().cuda_stream)
    e2.op_attention(1, dq.data_ptr(), s.layer.data_ptr(), s.slots, heads, d, n, c, begin * page, own.data_ptr())
    e2.close()
    s.check(out)
    s.check(own)


@pytest.mark.parametrize("reqs", [[(1, 300), (3, 700), (6, 900), (1, 0)],
                                  [(1, 40), (4, 90), (1, 15)],
                                  [(2, 500), (7, 100), (3, 450), (1, 20)]])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 16), ("fp32", 64)])
def test_requests_of_few_rows_in_a_wider_launch(native, eng, dtype, d, reqs):
    s = Case(native, eng, 31, dtype, 8, 2, d, 16, reqs)
    s.check(s.attention())


def test_a_workspace_that_overlaps_is_refused(native, eng):
    s = Case(native, eng, 32, "bf16", 4, 1, 128, 16, [(1, 30000)])
    size = eng.paged_workspace_bytes(s.plan)
    assert size > 0
    out = torch.zeros((1, 512), dtype=torch.bfloat16, device="cuda")
    both = torch.zeros(size + 4096, dtype=torch.uint8, device="cuda")
    ok = dict(q=s.dq.data_ptr(), layer=s.layer.data_ptr(), plan=s.plan, dev_plan=s.dplan.data_ptr(),
              workspace=both.data_ptr(), out=out.data_ptr())
    for bad in (dict(workspace=ok["layer"]), dict(workspace=ok["layer"] + 1024), dict(out=both.data_ptr()),
                dict(out=both.data_ptr() + size - 16), dict(q=both.data_ptr()), dict(q=both.data_ptr() + size - 16),
                dict(scale=2.0 ** 127.5)):
        with pytest.raises(native.OrcaError) as e:
            eng.op_paged_attention(**{**ok, **bad})
        assert e.value.code == native.ERR_INVALID, bad
    up = (size + 15) // 16 * 16
    eng.op_paged_attention(**{**ok, "out": both.data_ptr() + up})  # right behind it
    eng.sync()


@pytest.mark.parametrize("heads,kv,reqs", [(8, 2, [(40, 300), (8, 200), (1, 100), (1, 0)]),
                                           (8, 2, [(9, 70), (8, 30), (1, 15)]),
                                           (8, 2, [(9, 70), (8, 300), (8, 200)]), (71, 1, [(33, 40), (1, 30), (7, 0)]),
                                           (71, 1, [(32, 40), (1, 300)]), (16, 16, [(130, 5), (20, 100), (1, 60)])])
@pytest.mark.parametrize("d", [64, 128])
def test_requests_of_few_rows_as_prompts(native, eng, d, heads, kv, reqs):
    s = Case(native, eng, 33, "bf16", heads, kv, d, 16, reqs)
    s.check(s.attention())


def test_rows_that_take_seconds_hold_nobody_up(native, eng):
    """Rows over a value that is not finite are computed once more, key by key: over 600,000 keys that is longer than a
    wait may last, and the requests behind them on the same block still come out."""
    d, page, ctx, rows, sms = 128, 64, 600000, 250, torch.cuda.get_device_properties(0).multi_processor_count
    pages = -(-(ctx + rows) // page)
    table = np.tile(np.arange(1, pages + 1, dtype=np.int32), (2 * sms, 1))
    table[:sms, 0] = 0  # the first half of the requests begins with a page of its own
    layer = torch.zeros((2, 1, (pages + 1) * page, d), dtype=torch.bfloat16, device="cuda")
    layer[1] = 1
    layer[1, 0, 3, 5] = float("nan")
    plan = eng.paged_plan(1, 1, 1, d, page, pages + 1, [rows] * (2 * sms), [ctx] * (2 * sms), table)
    dplan = torch.from_numpy(plan).cuda()
    q = torch.ones((2 * sms * rows, d), dtype=torch.bfloat16, device="cuda")
    out, work = torch.zeros_like(q), torch.zeros(eng.paged_workspace_bytes(plan) + 16, dtype=torch.uint8, device="cuda")
    eng.op_paged_attention(q.data_ptr(), layer.data_ptr(), plan, dplan.data_ptr(), work.data_ptr(), out.data_ptr())
    eng.sync()
    want = torch.ones_like(out)
    want[:sms * rows, 5] = float("nan")
    assert torch.equal(torch.nan_to_num(out, 7.0), torch.nan_to_num(want, 7.0))


# --------------------------------------------------------------------------- #
# what a row's bits may depend on
# --------------------------------------------------------------------------- #
def fill_shared_memory(native, eng, word):
    """An attention of fp32 rows on every SM whose queries, keys and values are `word` throughout: what the kernels after it
    find in shared memory that they do not write themselves."""
    sms, ctx = torch.cuda.get_device_properties(0).multi_processor_count, 255
    n_pages = 4 * sms * (ctx + 1) // 16
    plan = eng.paged_plan(native.DTYPE_FP32, 1, 1, 128, 16, n_pages, [1] * 4 * sms, [ctx] * 4 * sms,
                          np.arange(n_pages).reshape(4 * sms, -1))
    layer, q = (torch.full(s, word, dtype=torch.int32, device="cuda") for s in ((2, n_pages * 16, 128), (4 * sms, 128)))
    dev, out = torch.from_numpy(plan).cuda(), torch.empty((4 * sms, 128), device="cuda")
    work = torch.empty(max(16, eng.paged_workspace_bytes(plan)), dtype=torch.uint8, device="cuda")
    eng.op_paged_attention(q.data_ptr(), layer.data_ptr(), plan, dev.data_ptr(), work.data_ptr(), out.data_ptr())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(40, 8), (6, 2), (7, 1), (12, 2), (44, 1)])
def test_bits_do_not_depend_on_what_ran_before(native, eng, heads, kv_heads, d):
    """Groups that do not divide 128 leave rows of a prompt's tile without a query.  Words that are large, or NaN, as
    two bf16 numbers lie there; zero is the calm case."""
    s = Case(native, eng, 41, "bf16", heads, kv_heads, d, 16, [(150, 90), (64, 300), (257, 0)])
    outs = []
    for word in (0, 0x70007000, 0x7FC07FC0, 0x71007F80 - (1 << 31)):
        fill_shared_memory(native, eng, word)
        outs.append(s.attention())
    s.check(outs[0])
    for o in outs[1:]:
        assert torch.equal(outs[0], o)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (40, 8), (16, 16)])
def test_bits_do_not_depend_on_the_next_requests_rows(native, eng, heads, kv_heads, d):
    """A request's last tile is filled up with rows of the next request, which are not its own."""
    s = Case(native, eng, 42, "bf16", heads, kv_heads, d, 16, [(30, 100), (45, 200), (70, 130)])
    want, calm = s.attention(), s.q[30:].copy()
    s.check(want)
    for factor in (1e30, -1e36, np.nan):
        s.q[30:] = rounded(calm * factor, "bf16")
        s.upload()
        assert torch.equal(want[:30], s.attention()[:30])


def narrow_limits(q, k, v, c):
    """limits() where weights enter the second product with 16 bits: rounded to bf16 and what is left of them rounded again,
    so that each is off by 2^-8 2^-8 of itself at most and the output by 2^-16 sum w |v| <= 2^-16 max |v|."""
    heads, d = q.shape[1:]
    ref, _ = paged.attention(q, k, v, c, 1 / np.sqrt(d))
    size = max((np.abs(q[:, h]) @ np.abs(k[h // (heads // len(k))]).T).max() for h in range(heads)) / np.sqrt(d)
    tol = 2 * (d + 16) * 2.0 ** -23 * size + 3 * 2.0 ** -20 + k.shape[1] * 2.0 ** -23 + 2.0 ** -16
    return ref, U["bf16"] * np.abs(ref) + tol * np.abs(v).max()


def one_part(q, k, v, c):
    """The output where weights are rounded to bf16 once: what narrow_limits() has to tell from it."""
    n, heads, d = q.shape
    out = np.zeros(q.shape)
    for h in range(heads):
        kk, vv = (x[h // (heads // len(k))].astype(np.float64) for x in (k, v))
        s = q[:, h].astype(np.float64) @ kk.T / np.sqrt(d)
        s = np.where(np.arange(kk.shape[0])[None] <= c + np.arange(n)[:, None], s, -np.inf)
        w = np.exp(s - s.max(1, keepdims=True))
        out[:, h] = rounded(w, "bf16") @ vv / w.sum(1, keepdims=True)
    return rounded(out, "bf16")


# Requests of at most 16 rows x heads of a key/value head, alone, beside one another and beside wider ones: prompts, and
# (at head_dim 16 and 32, or where there are few of them) tiles of 32 columns.
COMPANY = [(8, 2, [(1, 40)], 1), (8, 2, [(1, 40), (4, 30), (2, 60)], 3), (8, 2, [(1, 40), (4, 30), (2, 60), (200, 100)], 3),
           (8, 2, [(1, 40), (3, 20), (9, 50)], 2), (8, 2, [(1, 40), (4, 20), (5, 30), (7, 20)], 2),
           (8, 2, [(4, 20), (1, 100), (1, 90), (6, 30)], 3), (12, 4, [(5, 33), (1, 64), (1, 20), (300, 0)], 3),
           (4, 4, [(16, 30), (1, 70), (128, 0), (500, 20)], 2),
           (40, 8, [(1, 50), (3, 40), (1, 300), (260, 300)], 3), (16, 1, [(1, 60), (20, 50)], 1)]


@pytest.mark.parametrize("heads,kv_heads,reqs,narrow", COMPANY)
@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_narrow_requests_keep_16_bits_of_their_weights(native, eng, d, heads, kv_heads, reqs, narrow):
    s = Case(native, eng, 43, "bf16", heads, kv_heads, d, 16, reqs)
    s.q = rounded(s.q / 4, "bf16")
    s.host[1] = np.where(np.isnan(s.host[1]), np.nan, rounded(s.g.uniform(-1, 1, s.host[1].shape), "bf16"))
    s.upload()
    out = s.attention()
    s.check(out)
    got, r, told = out.float().cpu().numpy()[:s.rows, :s.H].reshape(s.rows, heads, d), 0, 0
    for i, ((n, c), t) in enumerate(zip(reqs, s.table)):
        if i < narrow:
            k, v = s.host[:, :, paged.slots(t, 16, 0, n + c)]
            ref, lim = narrow_limits(s.q[r:r + n], k, v, c)
            assert (np.abs(got[r:r + n] - ref) <= lim).all(), float((np.abs(got[r:r + n] - ref) / lim).max())
            told += (np.abs(one_part(s.q[r:r + n], k, v, c) - ref) > lim).sum()
        r += n
    assert told  # (one part would be seen)


@pytest.mark.parametrize("jump", [60.0, 100.0, 125.0, 126.0, 126.5, 127.0, 127.5])
@pytest.mark.parametrize("reqs,first,second", [([(150, 100)], 70, 130), ([(150, 100)], 70, 98), ([(33, 217)], 130, 195),
                                               ([(40, 3000)], 250, 256), ([(40, 3000)], 200, 700),
                                               ([(40, 3000)], 10, 2600), ([(40, 3000)], 250, 2999)])
@pytest.mark.parametrize("d", [64, 128])
def test_sums_near_the_end_of_fp32(native, eng, d, reqs, first, second, jump):
    """Two keys that are 2^jump above all others: in tiles or in parts of the keys that follow one another, whose weights are
    as large as fp32 holds over the maximum in front of them, and one when it has followed."""
    s = Case(native, eng, 44, "bf16", 8, 2, d, 16, reqs)
    (n, c), at = reqs[0], paged.slots(s.table[0], 16, 0, sum(reqs[0]))
    s.q[:], s.q[..., 0] = 0, 1
    s.host[0][:, at] = 0
    s.host[0][:, at[[first, second]], 0] = jump
    s.host[1][:, at] = rounded(s.g.uniform(-1, 1, s.host[1][:, at].shape), "bf16")
    s.upload()
    s.check(s.attention(scale=float(np.log(2.0))), scale=float(np.log(2.0)))


# --------------------------------------------------------------------------- #
# what one request may cost the others
# --------------------------------------------------------------------------- #
def microseconds(call):
    best = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        b.synchronize()
        best.append(a.elapsed_time(b) * 1e3)
    return min(best)


def growing(s, i, per_tile):
    """Request i's queries and keys positive, its keys growing by `per_tile` with every 64 of them."""
    r, (n, c) = sum(s.n[:i]), s.reqs[i]
    at = paged.slots(s.table[i], s.page, 0, n + c)
    s.q[r:r + n] = np.abs(s.q[r:r + n])
    s.host[0][:, at] = rounded(np.abs(s.host[0][:, at]) * (np.arange(n + c) // 64 * per_tile)[None, :, None], s.dtype)
    s.upload()


@pytest.mark.parametrize("per_tile", [0.5, 3.0, 20.0, 1e6, 1e25])
@pytest.mark.parametrize("reqs", [[(150, 700)], [(40, 3000), (2, 900)], [(3, 500), (130, 100)]])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_outgrow_the_maximum(native, eng, d, reqs, per_tile):
    """Every tile of 64 keys is by far above the ones before it (also by more than fp32 holds as a weight)."""
    s = Case(native, eng, 51, "bf16", 8, 2, d, 16, reqs)
    growing(s, 0, per_tile)
    s.check(s.attention())


@pytest.mark.parametrize("heads,kv_heads,d", [(40, 8, 128), (16, 2, 64)])
def test_one_request_does_not_hold_up_the_others(native, eng, heads, kv_heads, d):
    """A key or a value that is not finite but seen by all rows takes about the time of others (a row at a time, key by key,
    took some 500 times as long)."""
    s = Case(native, eng, 52, "bf16", heads, kv_heads, d, 16, [(700, 900), (600, 800), (500, 300)])
    calm_keys = s.host.copy()
    s.q[..., 5] = np.abs(s.q[..., 5]) + 1  # (a key of +inf gives scores of +inf)
    s.upload()
    s.attention()
    calm = microseconds(lambda: s.attention(sync=False))
    for which, bad in ((1, np.nan), (1, np.inf), (0, np.nan), (0, np.inf)):
        s.host[:] = calm_keys
        s.host[which, :, paged.slots(s.table[0], 16, 100, 1)[0], 5] = bad
        s.upload()
        if which or np.isnan(bad):  # (a score of +inf cannot be told from one that outgrew fp32)
            assert microseconds(lambda: s.attention(sync=False)) < 20 * calm
        out = s.attention()
        assert not torch.isfinite(out[:700, 5]).all() and torch.isfinite(out[700:]).all()
        assert torch.isfinite(out[:700, 6]).all() == (which == 1)


def test_rows_beside_a_value_that_is_not_theirs_hold_nobody_up(native, eng):
    """Rows in front of a value that is not finite, in one tile with it, are computed once more, key by key: over 600,000
    keys that is longer than a wait may last, and the requests behind them on the same block still come out."""
    d, page, ctx, rows, sms = 128, 64, 600000, 250, torch.cuda.get_device_properties(0).multi_processor_count
    pages = -(-(ctx + rows) // page)
    table = np.tile(np.arange(1, pages + 2, dtype=np.int32), (2 * sms, 1))[:, :pages]
    table[:sms, -1] = 0  # the first half of the requests ends with a page of its own
    layer = torch.zeros((2, 1, (pages + 2) * page, d), dtype=torch.bfloat16, device="cuda")
    layer[1] = 1
    last = (ctx + rows - 1) % page
    layer[1, 0, last, 5] = float("nan")
    plan = eng.paged_plan(1, 1, 1, d, page, pages + 2, [rows] * (2 * sms), [ctx] * (2 * sms), table)
    dplan = torch.from_numpy(plan).cuda()
    q = torch.ones((2 * sms * rows, d), dtype=torch.bfloat16, device="cuda")
    out, work = torch.zeros_like(q), torch.zeros(eng.paged_workspace_bytes(plan) + 16, dtype=torch.uint8, device="cuda")
    eng.op_paged_attention(q.data_ptr(), layer.data_ptr(), plan, dplan.data_ptr(), work.data_ptr(), out.data_ptr())
    eng.sync()
    want = torch.ones_like(out)
    want[rows - 1:sms * rows:rows, 5] = float("nan")
    assert torch.equal(torch.nan_to_num(out, 7.0), torch.nan_to_num(want, 7.0))


def test_tables_that_are_written_are_refused(native, eng):
    """The plan and the cosines are read while the rows are written."""
    s = append_case(native, eng, 61, "bf16", 4, 1, 128, 16, [(1, 30000), (2, 5)], 128, False)
    size, words = eng.paged_workspace_bytes(s.plan), len(s.plan)
    assert size > 0
    room = torch.zeros(4 * words + size + 2 * s.layer.numel() + 65536, dtype=torch.uint8, device="cuda")
    at = room.data_ptr()
    room[:4 * words] = s.dplan.view(torch.uint8)
    ok = dict(qkv=s.dqkv.data_ptr(), layer=s.layer.data_ptr(), plan=s.plan, dev_plan=at, q_out=s.q_out.data_ptr(),
              rope=s.drope.data_ptr(), rope_len=len(s.rope), rot_dim=128, ld_q=s.q_out.shape[1])
    rope_end = ok["rope"] + s.drope.numel() * 4
    for bad in (dict(q_out=at), dict(q_out=at + 4 * words - 16), dict(layer=at), dict(layer=at + 4 * words - 16),
                dict(q_out=ok["rope"]), dict(q_out=rope_end - 16), dict(layer=ok["rope"]), dict(layer=rope_end - 16)):
        with pytest.raises(native.OrcaError) as e:
            eng.op_paged_append(**{**ok, **bad})
        assert e.value.code == native.ERR_INVALID, bad
    up = at + (4 * words + 15) // 16 * 16
    q = dict(q=s.q_out.data_ptr(), layer=s.layer.data_ptr(), plan=s.plan, dev_plan=at, workspace=up,
             out=up + (size + 15) // 16 * 16)
    for bad in (dict(out=at), dict(out=at + 4 * words - 16), dict(workspace=at), dict(workspace=at + 4 * words - 16)):
        with pytest.raises(native.OrcaError) as e:
            eng.op_paged_attention(**{**q, **bad})
        assert e.value.code == native.ERR_INVALID, bad
    eng.op_paged_append(**ok)
    eng.op_paged_attention(**q)  # right behind one another
    eng.sync()


def test_split_keys_need_a_workspace(native, eng):
    s = Case(native, eng, 62, "bf16", 4, 1, 128, 16, [(1, 30000)])
    assert eng.paged_workspace_bytes(s.plan) > 0
    out = torch.full((1, s.H), 768.0, dtype=torch.bfloat16, device="cuda")
    call = lambda work: eng.op_paged_attention(s.dq.data_ptr(), s.layer.data_ptr(), s.plan, s.dplan.data_ptr(), work,
                                               out.data_ptr())
    with pytest.raises(native.OrcaError) as e:
        call(0)
    assert e.value.code == native.ERR_INVALID
    eng.sync()
    assert (out == 768).all()
    call(s.work.data_ptr())
    assert (out != 768).all()


@pytest.mark.parametrize("reqs,key", [([(150, 100)], 70), ([(40, 3000)], 300), ([(40, 3000)], 3000), ([(33, 217)], 130),
                                      ([(5, 100), (200, 0)], 70), ([(7, 90), (1, 50), (2, 300)], 85)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("fp32", 64)])
def test_one_weight_above_all_others(native, eng, dtype, d, reqs, key):
    """A key of 2^20 times the others' weight, its own a number that bf16 rounds by half a step (2^20 (1 + 2^-8)): what is
    rounded of it goes out of the sum as well, so that the output is the key's value."""
    s = Case(native, eng, 45, dtype, 8, 2, d, 16, reqs)
    s.q[:], s.q[..., :2] = 0, 1
    for (n, c), t in zip(reqs, s.table):
        at = paged.slots(t, 16, 0, n + c)
        s.host[0][:, at] = 0
        s.host[0][:, at[min(key, c)], :2] = rounded(np.array([20, np.log2(1 + 2.0 ** -8)]), dtype)
    s.upload()
    s.check(s.attention(scale=float(np.log(2.0))), scale=float(np.log(2.0)))
