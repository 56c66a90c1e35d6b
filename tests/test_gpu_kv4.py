"""The 4-bit K/V cache on the GPU: the bytes an append writes, the values a read
gives and attention over them, against the float64 oracle (oracle/kv4.py).

Tolerances.  Bytes and read values are exact (a read rounds once to the plan's
type, as the oracle's value is rounded).  Attention: with B = D 2^-24 max_k
sum |q_i k_i| log2(e) / sqrt(D) the fp32 rounding of a score of D terms (a few
more for the group sums: (D + 16) is used), a weight is off by a factor within
1 +- (2 B + 2^-21), numerator and denominator both, sums add 2^-24 per key and
the last rounding is eps / 2: so
  |out - ref| <= eps / 2 |ref| + (4 B + 2^-19 + T 2^-24) max |v|.
The tensor-core path splits a weight times a scale into two bf16 (2^-16 left),
and prompts run on K and V rounded to fp16 with weights rounded to fp16: 2^-11
on each of the value and the weight (and 2^-25 of the largest for those that
fall below fp16's normal range) and 2^-11 sum |q k| log2(e) / sqrt(D) on a
score, whose natural exponential moves by ln 2 times that."""

import math

import numpy as np
import pytest
import torch

from oracle import kv4

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


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


def code(native, dtype):
    return native.DTYPE_BF16 if dtype == "bf16" else native.DTYPE_FP32


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(TD[dtype])


class Case:
    """Requests (rows, ctx) at odd and even offsets with gaps, over a layer whose unused bytes are all ones
    (codes 15, parameters NaN): nothing of them may reach an output."""

    def __init__(self, native, eng, seed, dtype, heads, d, reqs, std=1.0, shift=0.0):
        g = np.random.default_rng(seed)
        self.native, self.eng, self.dtype, self.heads, self.d, self.reqs = native, eng, dtype, heads, d, reqs
        self.off, at = [], int(g.integers(0, 4))
        for n, c in reqs:
            self.off.append(at)
            at += c + n + int(g.integers(0, 4))
        self.slots = at + 1
        self.n, self.c = [n for n, _ in reqs], [c for _, c in reqs]
        rows, H = sum(self.n), heads * d
        self.host = np.full(native.kv4_layer_bytes(heads, d, self.slots), 0xFF, np.uint8)
        self.layer = kv4.Layer(heads, d, self.slots, self.host)
        val = lambda *s: rounded((g.standard_normal(s) * std + shift).astype(np.float32), dtype).float().numpy()  # noqa: E731
        for (n, c), o in zip(reqs, self.off):
            kv = val(c, 2, heads, d)
            for t in range(c):
                self.layer.write(o + t, kv[t, 0], kv[t, 1])
        self.qkv = val(rows, 3, heads, d)
        self.qkv[:, 0] = rounded(g.standard_normal((rows, heads, d)).astype(np.float32), dtype).float().numpy()
        self.dev = torch.from_numpy(self.host.copy()).cuda()
        self.upload()
        self.plan = eng.kv4_plan(code(native, dtype), heads, d, self.slots, self.n, self.c, self.off)
        self.dplan = torch.from_numpy(self.plan).cuda()
        self.work = torch.full((max(1, eng.kv4_workspace_bytes(self.plan)),), 0xFF, dtype=torch.uint8, device="cuda")

    def upload(self):
        self.dqkv = rounded(self.qkv.reshape(len(self.qkv), -1), self.dtype).cuda()

    def append(self, **kw):
        self.eng.op_kv4_append(self.dqkv.data_ptr(), self.dev.data_ptr(), self.plan, self.dplan.data_ptr(), **kw)

    def append_oracle(self):
        r = 0
        for n, c, o in zip(self.n, self.c, self.off):
            for j in range(n):
                self.layer.write(o + c + j, self.qkv[r, 1], self.qkv[r, 2])
                r += 1

    def attention(self, **kw):
        out = torch.full((len(self.qkv), self.heads * self.d), float("nan"), dtype=TD[self.dtype], device="cuda")
        self.eng.op_kv4_attention(self.dqkv.data_ptr(), self.dev.data_ptr(), self.plan, self.dplan.data_ptr(),
                                  self.work.data_ptr(), out.data_ptr(), **kw)
        return out

    def check(self, out, rounded_operands=False):
        got = out.float().cpu().numpy().reshape(len(self.qkv), self.heads, self.d).astype(np.float64)
        eps = torch.finfo(TD[self.dtype]).eps / 2
        r = 0
        for n, c, o in zip(self.n, self.c, self.off):
            k, v = self.layer.read(o, c + n)
            q = self.qkv[r:r + n, 0].astype(np.float64)
            ref = kv4.attention(q, k, v, c)
            size = np.einsum("nhd,hkd->nhk", np.abs(q), np.abs(k)).max() * math.log2(math.e) / math.sqrt(self.d)
            tol = 4 * (self.d + 16) * 2.0 ** -24 * size + 2.0 ** -15 + (c + n) * 2.0 ** -24
            if rounded_operands:
                tol += 2 * 2.0 ** -11 + (c + n) * 2.0 ** -25 + 2 * 2.0 ** -11 * size * math.log(2)
            lim = eps * np.abs(ref) + tol * np.abs(v).max()
            d = np.abs(got[r:r + n] - ref)
            assert np.isfinite(got[r:r + n]).all() and (d <= lim).all(), (n, c, float((d / lim).max()))
            r += n


TYPES = [("bf16", 128), ("bf16", 64), ("bf16", 32), ("bf16", 16), ("fp32", 128), ("fp32", 64), ("fp32", 32),
         ("fp32", 16)]


@pytest.mark.parametrize("dtype,d", TYPES)
def test_append_writes_the_oracles_bytes(native, eng, dtype, d):
    s = Case(native, eng, 1, dtype, 5, d, [(1, 0), (7, 3), (1, 12), (66, 0), (2, 5), (3, 8)], std=2.0, shift=0.3)
    f = s.qkv
    f[0, 1, 0] = 0.25                      # a constant group
    f[1, 1, 1, :3] = [np.inf, 1, 2]        # groups that read back as NaN
    f[2, 2, 2, 1] = -np.inf
    f[3, 2, 0, 5] = np.nan
    f[4, 1, 3, :2] = [3e38, -3e38]         # a range beyond fp32
    f[5, 1] *= 1e-38                       # subnormal scales
    f[6, 2] = 0.0
    f[7, 1, 0, :8] = [0, 15, 0.5, 1.5, 2.5, 14.5, 13.5, 7.5]  # halves (where the group's minimum is 0)
    f[7, 1, 0] = np.clip(f[7, 1, 0], 0, 15)
    f[8, 2] = np.round(f[8, 2] * 16) / 16  # coarse values: borders are met exactly
    f[9, 1] += 1000.0                      # a range far from zero
    s.qkv = rounded(f, dtype).float().numpy()
    s.upload()
    s.append()
    s.append_oracle()
    want = torch.from_numpy(s.host)
    assert torch.equal(s.dev.cpu()[:s.layer.kc.size * 2], want[:s.layer.kc.size * 2])  # codes
    # parameters by value: a zero minimum may have either sign, NaN any payload
    a, b = (x[s.layer.kc.size * 2:].view(torch.bfloat16).float() for x in (s.dev.cpu(), want))
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_codes_at_borders(native, eng, dtype):
    """Values within a few ulp of every border between codes, for scales of all mantissas: the code is real
    arithmetic's, whichever way an fp32 quotient would round."""
    g = np.random.default_rng(5)
    heads, d, rows = 4, 128, 64
    s = Case(native, eng, 2, dtype, heads, d, [(rows, 0)])
    x = s.qkv[:, 1:].reshape(-1, 32)
    for i in range(len(x)):
        lo, span = np.float32(g.standard_normal() * 4), np.float32(np.exp(g.uniform(-6, 3)))
        lo = np.float32(kv4.bf16(lo).item()) if i % 2 else lo
        x[i, 0], x[i, 1] = lo, lo + span
        sc, m = kv4.bf16((x[i, 1] - x[i, 0]) / np.float32(15)).item(), kv4.bf16(lo).item()
        border = (m + sc * (np.arange(30) % 15 + 0.5)).astype(np.float32)
        step = np.spacing(np.abs(border)) * (g.integers(-2, 3, 30) if dtype == "fp32" else 0)
        x[i, 2:] = np.clip(border + step.astype(np.float32), lo, lo + span)
    s.qkv[:, 1:] = x.reshape(rows, 2, heads, d)
    s.qkv = rounded(s.qkv, dtype).float().numpy()
    s.upload()
    s.append()
    s.append_oracle()
    assert np.array_equal(s.dev.cpu().numpy(), s.host)


@pytest.mark.parametrize("dtype,d", TYPES)
def test_read_gives_the_values(native, eng, dtype, d):
    s = Case(native, eng, 3, dtype, 3, d, [(1, 0), (1, 1), (5, 60), (70, 130), (1, 63), (64, 64)])
    s.append()
    s.append_oracle()
    total = sum(s.n) + sum(s.c)
    out = torch.full((2, s.heads, total, d), float("nan"), dtype=TD[dtype], device="cuda")
    eng.op_kv4_read(s.dev.data_ptr(), s.plan, s.dplan.data_ptr(), out.data_ptr())
    at = 0
    for n, c, o in zip(s.n, s.c, s.off):
        for got, want in zip(out[:, :, at:at + n + c], s.layer.read(o, n + c)):
            assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(TD[dtype]))
        at += n + c


DECODE = [0, 1, 2, 14, 15, 16, 17, 31, 32, 33, 63, 64, 127, 128, 129, 500, 513, 1023, 2100]


@pytest.mark.parametrize("dtype,d", TYPES)
def test_decode(native, eng, dtype, d):
    s = Case(native, eng, 4, dtype, 3, d, [(1, c) for c in DECODE])
    s.append()
    s.append_oracle()
    s.check(s.attention())


@pytest.mark.parametrize("dtype,d,heads", [("bf16", 128, 40), ("bf16", 64, 1), ("fp32", 64, 20)])
def test_decode_far_from_zero(native, eng, dtype, d, heads):
    """K and V with a common offset many times their spread: codes and minimum have to meet without loss."""
    s = Case(native, eng, 5, dtype, heads, d, [(1, 40), (1, 333), (1, 900)], std=0.05, shift=6.0)
    s.append()
    s.append_oracle()
    s.check(s.attention())


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("std", [1e-6, 300.0])
def test_decode_small_and_large_values(native, eng, dtype, d, std):
    s = Case(native, eng, 6, dtype, 2, d, [(1, 40), (1, 333)], std=std)
    if std > 1:
        s.qkv[:, 0] = rounded(s.qkv[:, 0] / 256, dtype).float().numpy()
        s.upload()
    s.append()
    s.append_oracle()
    s.check(s.attention())


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("std", [1e-20, 1e15])
def test_magnitudes_far_from_one(native, eng, dtype, d, std):
    """Keys and values of any size (queries of the inverse size): increments, a few rows and a prompt."""
    s = Case(native, eng, 21, dtype, 2, d, [(1, 40), (1, 333), (5, 60), (40, 30)], std=std)
    s.qkv[:, 0] = rounded(s.qkv[:, 0] / np.float32(std), dtype).float().numpy()
    s.upload()
    s.append()
    s.append_oracle()
    s.check(s.attention(), rounded_operands=dtype == "bf16")


@pytest.mark.parametrize("dtype,d", TYPES)
def test_few_rows(native, eng, dtype, d):
    s = Case(native, eng, 7, dtype, 3, d, [(2, 0), (3, 1), (7, 130), (15, 64), (1, 77), (5, 700)])
    s.append()
    s.append_oracle()
    s.check(s.attention())


@pytest.mark.parametrize("std", [1.0, 1e-5, 3e4])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("bf16", 16), ("fp32", 64)])
def test_prompts(native, eng, dtype, d, std):
    s = Case(native, eng, 8, dtype, 3, d, [(130, 0), (64, 0), (127, 200), (257, 65), (1, 300), (4, 30), (33, 1)],
             std=std)
    s.qkv[:, 0] = rounded(s.qkv[:, 0] * min(1.0, 1 / std), dtype).float().numpy()
    s.upload()
    s.append()
    s.append_oracle()
    s.check(s.attention(), rounded_operands=dtype == "bf16")


@pytest.mark.parametrize("dtype,d,n", [("bf16", 128, 200), ("bf16", 64, 200), ("bf16", 32, 70), ("fp32", 64, 70),
                                       ("bf16", 128, 9)])
def test_nan_reaches_the_rows_that_see_it_and_no_other(native, eng, dtype, d, n):
    s = Case(native, eng, 20, dtype, 2, d, [(n, 20)])
    a, b = n // 3, n // 2
    s.qkv[a, 2, 0, 3] = np.nan   # a value of head 0 from row a on
    s.qkv[b, 1, 1, 5] = np.inf   # a key of head 1 from row b on
    s.upload()
    s.append()
    out = s.attention().float().reshape(n, 2, d)
    assert out[:a, 0].isfinite().all() and out[:b, 1].isfinite().all()
    assert out[a:, 0, :min(32, d)].isnan().all() and out[b:, 1].isnan().all()


def test_rows_do_not_depend_on_their_company(native, eng):
    """A row's output is the same bits alone and in a batch whose work is split alike, and call after call."""
    s = Case(native, eng, 9, "bf16", 4, 128, [(1, 900), (1, 1300), (1, 50)])
    s.append()
    a, b = s.attention(), s.attention()
    assert torch.equal(a, b)


def test_another_stream_and_graph_replay(native):
    """An engine on a stream of its own; append and attention captured, replayed over changed inputs."""
    st = torch.cuda.Stream()
    e = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None, st.cuda_stream)
    try:
        with torch.cuda.stream(st):
            s = Case(native, e, 10, "bf16", 8, 128, [(1, 700), (1, 33), (5, 260), (40, 90)])
            out = torch.zeros((len(s.qkv), s.heads * s.d), dtype=torch.bfloat16, device="cuda")

            def step():
                s.append(sync=False)
                e.op_kv4_attention(s.dqkv.data_ptr(), s.dev.data_ptr(), s.plan, s.dplan.data_ptr(), s.work.data_ptr(),
                                   out.data_ptr(), sync=False)
            step()
            e.sync()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=st):
                step()
            s.qkv = s.qkv[::-1].copy()
            s.dqkv.copy_(rounded(s.qkv.reshape(len(s.qkv), -1), "bf16").cuda())
            gr.replay()
            gr.replay()
            e.sync()
            s.append_oracle()
            s.check(out, rounded_operands=True)
    finally:
        e.close()


def test_offsets_past_32_bits(native, eng):
    """A layer of more than 4 GiB of codes per half: the last slots of the last head."""
    heads, d, slots = 64, 128, 1_200_003
    n, c, off = [1, 3], [70, 20], [slots - 71, slots - 171]
    nbytes = native.kv4_layer_bytes(heads, d, slots)
    assert heads * (slots + 13) // 16 * 16 * d // 2 > 2 ** 32
    layer = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    g = np.random.default_rng(11)
    small = Case(native, eng, 11, "bf16", heads, d, [(3, 20), (1, 70)])
    # the same contents: filled by appends of whole contexts at both places
    H = heads * d
    ctx = rounded(g.standard_normal((90, 3 * H)).astype(np.float32), "bf16").cuda()
    plan = eng.kv4_plan(native.DTYPE_BF16, heads, d, slots, [70, 20], [0, 0], off)
    dplan = torch.from_numpy(plan).cuda()
    eng.op_kv4_append(ctx.data_ptr(), layer.data_ptr(), plan, dplan.data_ptr())
    plan = eng.kv4_plan(native.DTYPE_BF16, heads, d, slots, n, c, off)
    dplan = torch.from_numpy(plan).cuda()
    work = torch.zeros(max(1, eng.kv4_workspace_bytes(plan)), dtype=torch.uint8, device="cuda")
    qkv = torch.cat([small.dqkv[3:], small.dqkv[:3]])
    out = torch.zeros((4, H), dtype=torch.bfloat16, device="cuda")
    eng.op_kv4_append(qkv.data_ptr(), layer.data_ptr(), plan, dplan.data_ptr())
    eng.op_kv4_attention(qkv.data_ptr(), layer.data_ptr(), plan, dplan.data_ptr(), work.data_ptr(), out.data_ptr())
    del layer
    # the reference: the same rows in a small layer
    ctx = ctx.float().cpu().numpy().reshape(90, 3, heads, d)
    for (t0, t1), o in (((0, 70), small.off[1]), ((70, 90), small.off[0])):
        for t in range(t0, t1):
            small.layer.write(o + t - t0, ctx[t, 1], ctx[t, 2])
    small.append_oracle()
    small.check(torch.cat([out[1:], out[:1]]))


def test_refusals(native, eng):
    s = Case(native, eng, 12, "bf16", 2, 64, [(1, 70), (1, 900)])  # (900 keys are split: a workspace is needed)
    E, L = native.ERR_INVALID, native.lib
    h, pl = eng.handle, s.plan.ctypes.data
    q, la, dp, w, o = s.dqkv.data_ptr(), s.dev.data_ptr(), s.dplan.data_ptr(), s.work.data_ptr(), s.dqkv.data_ptr()
    assert eng.kv4_workspace_bytes(s.plan) > 0
    junk = np.zeros(64, np.int32)
    for args in ((0, la, pl, dp), (q, 0, pl, dp), (q, la, 0, dp), (q, la, pl, 0), (q + 2, la, pl, dp),
                 (q, la + 4, pl, dp), (q, la, pl, dp + 4), (q, la, junk.ctypes.data, dp)):
        assert L.orca_op_kv4_append(h, *args) == E
    for args in ((0, pl, dp, o), (la, 0, dp, o), (la, pl, 0, o), (la, pl, dp, 0), (la, pl, dp, o + 2),
                 (la + 8, pl, dp, o)):
        assert L.orca_op_kv4_read(h, *args) == E
    for args in ((0, la, pl, dp, w, o), (q, 0, pl, dp, w, o), (q, la, 0, dp, w, o), (q, la, pl, 0, w, o),
                 (q, la, pl, dp, 0, o), (q, la, pl, dp, w, 0), (q, la, pl, dp, w + 4, o), (q + 8, la, pl, dp, w, o)):
        assert L.orca_op_kv4_attention(h, *args) == E
    twice = eng.kv4_plan(native.DTYPE_BF16, 2, 64, s.slots, [2, 3], [5, 0], [0, 6])  # slots 5, 6 and 6, 7, 8
    assert L.orca_op_kv4_append(h, q, la, twice.ctypes.data, dp) == E
    with pytest.raises(ValueError):
        eng.kv4_plan(native.DTYPE_BF16, 2, 64, 100, [1, 1], [0], [0, 1])


def test_shared_prefix(native, eng):
    """Two requests may read the same slots (a shared context); only written slots have to be apart."""
    s = Case(native, eng, 13, "fp32", 2, 64, [(1, 100)])
    s.append()
    s.append_oracle()
    plan = eng.kv4_plan(native.DTYPE_FP32, 2, 64, s.slots, [1, 1], [100, 57], [s.off[0], s.off[0]])
    dplan = torch.from_numpy(plan).cuda()
    work = torch.zeros(max(1, eng.kv4_workspace_bytes(plan)), dtype=torch.uint8, device="cuda")
    qkv, out = s.dqkv.repeat(2, 1), torch.zeros((2, 128), device="cuda")
    eng.op_kv4_attention(qkv.data_ptr(), s.dev.data_ptr(), plan, dplan.data_ptr(), work.data_ptr(), out.data_ptr())
    s.qkv = np.concatenate([s.qkv, s.qkv])
    s.n, s.c, s.off = [1, 1], [100, 57], s.off * 2
    s.check(out)


@pytest.mark.parametrize("n", [1, 9, 20, 40])
def test_nan_value_of_a_key_that_weighs_nothing(native, eng, n):
    """A key that a row sees, but whose weight underflows: 0 times its NaN value is NaN, as in the formula."""
    s = Case(native, eng, 22, "bf16", 2, 128, [(n, 20)])
    s.qkv[:, 0, 0], s.qkv[:, 1, 0] = 8.0, 8.0
    s.qkv[0, 1, 0] = -8.0          # head 0, row 0: a score of 8192 / sqrt(128) below the other rows'
    s.qkv[0, 2, 0, 3] = np.nan
    s.upload()
    s.append()
    out = s.attention().float().reshape(n, 2, 128)
    assert out[:, 0, :32].isnan().all() and out[:, 1].isfinite().all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 32), ("fp32", 64)])
def test_nothing_else_is_written(native, eng, dtype, d):
    """Rows behind the last one, what lies behind a read, slots outside the ranges and what follows a workspace."""
    s = Case(native, eng, 23, dtype, 3, d, [(1, 700), (5, 600), (150, 33), (1, 0)])
    H, rows, keys = s.heads * d, len(s.qkv), sum(s.n) + sum(s.c)
    need = eng.kv4_workspace_bytes(s.plan)
    s.work = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((rows + 200, H), float("nan"), dtype=TD[dtype], device="cuda")
    back = torch.full((2 * s.heads * keys + 200, d), float("nan"), dtype=TD[dtype], device="cuda")
    tail = torch.full((s.dev.numel() + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    tail[:s.dev.numel()] = s.dev
    s.dev = tail
    s.append()
    eng.op_kv4_attention(s.dqkv.data_ptr(), s.dev.data_ptr(), s.plan, s.dplan.data_ptr(), s.work.data_ptr(),
                         out.data_ptr())
    eng.op_kv4_read(s.dev.data_ptr(), s.plan, s.dplan.data_ptr(), back.data_ptr())
    s.append_oracle()
    assert np.array_equal(s.dev[:-4096].cpu().numpy(), s.host)
    assert (s.dev[-4096:] == 0xFF).all() and (s.work[need:] == 0xA5).all()
    assert out[rows:].isnan().all() and back[-200:].isnan().all() and back[:-200].isfinite().all()
    s.check(out[:rows], rounded_operands=dtype == "bf16")
    # and the plan is as it was: the next call finds its counters at zero
    assert np.array_equal(s.dplan.cpu().numpy(), s.plan)


def test_two_streams_at_once(native):
    """Two engines on streams of their own, each with its layer, plan and workspace, queued without a wait."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    engines = [native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None, st.cuda_stream)
               for st in streams]
    cases, outs = [], []
    for i, (e, st) in enumerate(zip(engines, streams)):
        with torch.cuda.stream(st):
            cases.append(Case(native, e, 24 + i, "bf16", 8, 128, [(1, 3000), (7, 1500), (40, 200), (1, 17)]))
            outs.append(torch.zeros((len(cases[i].qkv), 8 * 128), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, e, o in zip(cases, engines, outs):
            s.append(sync=False)
            e.op_kv4_attention(s.dqkv.data_ptr(), s.dev.data_ptr(), s.plan, s.dplan.data_ptr(), s.work.data_ptr(),
                               o.data_ptr(), sync=False)
    for s, e, o in zip(cases, engines, outs):
        e.sync()
        s.append_oracle()
        s.check(o, rounded_operands=True)
        e.close()


@pytest.mark.parametrize("heads", [1, 37])
@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("reqs", [[(1, 0)] * 5, [(1, 0), (1, 2), (2, 0), (2, 2), (1, 1), (4, 0)], [(5, 0), (1, 0)]])
def test_read_of_short_ranges(native, eng, dtype, d, heads, reqs):
    s = Case(native, eng, 26, dtype, heads, d, reqs)
    s.append()
    s.append_oracle()
    total = sum(s.n) + sum(s.c)
    out = torch.full((2 * heads * total + 8, d), float("nan"), dtype=TD[dtype], device="cuda")
    eng.op_kv4_read(s.dev.data_ptr(), s.plan, s.dplan.data_ptr(), out.data_ptr())
    assert out[-8:].isnan().all()
    out, at = out[:-8].view(2, heads, total, d), 0
    for n, c, o in zip(s.n, s.c, s.off):
        for got, want in zip(out[:, :, at:at + n + c], s.layer.read(o, n + c)):
            assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(TD[dtype]))
        at += n + c


def prompt_case(native, eng, seed, d, **kw):
    """A batch whose rows are many enough for the prefill kernel (its fp16 operands are in the workspace)."""
    s = Case(native, eng, seed, "bf16", 40, d, [(600, 40), (140, 500), (1, 60), (5, 900)], **kw)
    assert eng.kv4_workspace_bytes(s.plan) > 2 * len(s.qkv) * s.heads * d
    return s


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("std", [1.0, 1e-20, 1e15])
def test_prompts_of_many_heads(native, eng, d, std):
    s = prompt_case(native, eng, 27, d, std=std)
    s.qkv[:, 0] = rounded(s.qkv[:, 0] / np.float32(std), "bf16").float().numpy()
    s.upload()
    s.append()
    s.append_oracle()
    s.check(s.attention(), rounded_operands=True)


@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_prompts_of_many_heads(native, eng, d):
    s = prompt_case(native, eng, 28, d)
    s.qkv[250, 2, 7, 3] = np.nan   # of the first request: a value of head 7 from row 250 on
    s.qkv[300, 1, 9, 5] = np.inf   # a key of head 9 from row 300 on
    s.upload()
    s.append()
    out = s.attention().float().reshape(len(s.qkv), 40, d)
    bad = out.isnan()
    assert bad[250:600, 7, :32].all() and bad[300:600, 9].all()
    bad[250:600, 7], bad[300:600, 9] = False, False
    assert not bad.any() and out[:250].isfinite().all()


def test_prompts_behind_the_last_row(native, eng):
    s = prompt_case(native, eng, 29, 128)
    need, rows = eng.kv4_workspace_bytes(s.plan), len(s.qkv)
    s.work = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    s.append()
    out = torch.full((rows + 200, s.heads * s.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    eng.op_kv4_attention(s.dqkv.data_ptr(), s.dev.data_ptr(), s.plan, s.dplan.data_ptr(), s.work.data_ptr(),
                         out.data_ptr())
    assert out[rows:].isnan().all() and out[:rows].isfinite().all() and (s.work[need:] == 0xA5).all()
    assert np.array_equal(s.dplan.cpu().numpy(), s.plan)


@pytest.mark.parametrize("dtype,d", TYPES)
def test_single_rows_beside_groups(native, eng, dtype, d):
    """Single rows in the launch of the groups (few keys), and in their own (many)."""
    for heads, reqs in ((3, [(1, 0), (2, 100), (1, 700), (7, 33), (1, 5)]), (40, [(1, 3000), (3, 20), (1, 2500)])):
        s = Case(native, eng, 30, dtype, heads, d, reqs)
        s.append()
        s.append_oracle()
        s.check(s.attention())
