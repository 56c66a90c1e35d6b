"""Token sampling on the GPU against the float64 oracle (oracle/sampling.py).  Tokens are equal: the kernel sums
weights of 42 fraction bits exactly, so a token differs from the oracle's only where u times the total, or a filter's
border, lies within about V 2^-42 of a border between two tokens; the inputs are seeded and none does."""

import numpy as np
import pytest
import torch

from oracle.sampling import sample

pytestmark = pytest.mark.gpu

INF = float("inf")


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


def draw(native, eng, x, u, t=None, k=None, p=None, m=None, ld=0, sync=True):
    """x: torch tensor [rows, ld] on the CPU; parameters: lists or None."""
    x = x.cuda()
    V = x.shape[1] if not ld else ld[0]
    keep = [torch.tensor(a, dtype=torch.int32 if i == 1 else torch.float32, device="cuda") if a is not None else None
            for i, a in enumerate((t, k, p, m))]
    ptr = [a.data_ptr() if a is not None else 0 for a in keep]
    out = torch.full((x.shape[0],), -7, dtype=torch.int32, device="cuda")
    du = torch.tensor(u, dtype=torch.float32, device="cuda")
    eng.op_sample(native.DTYPE_BF16 if x.dtype == torch.bfloat16 else native.DTYPE_FP32, x.data_ptr(), x.shape[0], V,
                  out.data_ptr(), du.data_ptr(), *ptr, ld=x.shape[1], sync=sync)
    torch.cuda.synchronize()
    return out.cpu().tolist()


def want(x, u, t=None, k=None, p=None, m=None):
    rows = len(u)
    x = x.float().numpy()
    return [sample(x[i], u[i], *(a[i] if a is not None else z for a, z in ((t, 1.0), (k, 0), (p, 1.0), (m, 0.0))))
            for i in range(rows)]


def logits(seed, rows, V, dtype, std=3.0):
    g = np.random.default_rng(seed)
    return torch.from_numpy((g.standard_normal((rows, V)) * std).astype(np.float32)).to(dtype), g


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 512, 1000, 1023, 1025, 4097, 50257, 131071, 300001])
def test_every_filter(native, eng, V, dtype):
    rows = 24
    x, g = logits(V, rows, V, dtype)
    u = g.random(rows, dtype=np.float32).tolist()
    t = [float(a) for a in np.float32(g.choice([0.0, 0.2, 0.7, 1.0, 1.5, 10.0, 1000.0], rows))]
    k = [int(a) for a in g.choice([-1, 0, 1, 2, 5, 50, 1000, 3000, V, V + 1], rows)]
    p = [float(a) for a in np.float32(g.choice([0.0, 0.1, 0.5, 0.9, 0.95, 0.999, 1.0], rows))]
    m = [float(a) for a in np.float32(g.choice([0.0, 0.0, 1e-4, 0.05, 0.5, 1.0], rows))]
    none = [None] * 4
    assert draw(native, eng, x, u) == want(x, u)
    for i, a in enumerate((t, k, p, m)):
        only = list(none)
        only[i] = a
        assert draw(native, eng, x, u, *only) == want(x, u, *only), i
    assert draw(native, eng, x, u, t, k, p, m) == want(x, u, t, k, p, m)


def test_ends_of_the_uniform(native, eng):
    x, g = logits(3, 4, 777, torch.float32)
    for u in (0.0, 2.0 ** -149, 2.0 ** -41, 0.5, 1 - 2.0 ** -24):
        assert draw(native, eng, x, [u] * 4, p=[1.0, 0.9, 0.3, 0.0]) == want(x, [u] * 4, p=[1.0, 0.9, 0.3, 0.0])


@pytest.mark.parametrize("V", [64, 1024, 50257])
def test_ties(native, eng, V):
    """Equal logits: filters keep the lowest ids; u on a border between two tokens takes the upper one."""
    x = torch.full((8, V), -2.5)
    u = [0.0, 0.25, 0.5, 0.75, 0.5, 0.99, 0.999, 1 - 2.0 ** -24]
    k = [0, 0, 0, 7, 32, 33, V - 1, 1]
    p = [1.0, 1.0, 0.5, 1.0, 0.5, 0.25, 0.75, 1.0]
    assert draw(native, eng, x, u, k=k, p=p) == want(x, u, k=k, p=p)
    x = torch.round(logits(4, 8, V, torch.float32)[0])  # a few distinct values
    k = [1, 2, 10, 100, 5, 37, 0, 0]
    assert draw(native, eng, x, u, k=k, p=p) == want(x, u, k=k, p=p)


def test_zeros_of_both_signs_are_one_value(native, eng):
    x = torch.zeros((3, 100))
    x[:, ::2] = -0.0
    assert draw(native, eng, x, [0.0, 0.5, 0.9], k=[3, 4, 7]) == [0, 2, 6]
    assert draw(native, eng, x, [0.5] * 3, t=[0.0] * 3) == [0, 0, 0]


def test_masked_and_special_logits(native, eng):
    V = 1000
    x, g = logits(5, 12, V, torch.float32)
    lowest = torch.finfo(torch.float32).min
    x[0, 10:] = -INF
    x[1] = -INF                      # nothing left
    x[2] = float("nan")
    x[3, ::2] = float("nan")
    x[4, 100:] = lowest              # masks of the type's lowest value
    x[5] = lowest                    # every token at it: equally likely
    x[6, [5, 7, 800]] = INF          # three certain ones
    x[7] = -INF
    x[7, 999] = lowest               # one token
    x[8, 0] = torch.finfo(torch.float32).max
    x[9] = -INF
    x[9, 3:5] = torch.tensor([-1e30, -2e30])
    u = [0.3, 0.3, 0.3, 0.7, 0.99, 0.5, 0.5, 0.9, 0.9, 0.99, 0.1, 0.2]
    for kw in (dict(), dict(k=[50] * 12), dict(p=[0.9] * 12), dict(k=[600] * 12, p=[0.99] * 12, m=[0.01] * 12),
               dict(t=[0.0] * 12), dict(t=[1e-6] * 12), dict(t=[1e6] * 12)):
        got = draw(native, eng, x, u, **kw)
        assert got[1] == -1 and got[2] == -1
        assert got == want(x, u, **kw), kw


def test_temperature_near_zero_and_subnormal(native, eng):
    x, g = logits(6, 4, 500, torch.float32)
    t = [1e-45, 1e-30, 1e-3, 0.0]
    assert draw(native, eng, x, [0.9] * 4, t=t) == [int(a) for a in x.argmax(1)]


def test_stride_and_rows_behind(native, eng):
    """ld > vocab, odd: what lies between the rows is not read; unused outputs stay."""
    x, g = logits(7, 5, 1237, torch.float32)
    x[:, 1000:] = 1e9
    u = [0.1, 0.3, 0.5, 0.7, 0.9]
    assert draw(native, eng, x, u, p=[0.9] * 5, ld=(1000,)) == want(x[:, :1000], u, p=[0.9] * 5)
    out = torch.full((8,), -7, dtype=torch.int32, device="cuda")
    xd, ud = x.cuda(), torch.tensor(u, device="cuda")
    eng.op_sample(native.DTYPE_FP32, xd.data_ptr(), 5, 1000, out.data_ptr(), ud.data_ptr(), ld=1237)
    assert out[5:].tolist() == [-7] * 3


def test_largest_vocabulary(native, eng):
    V = 1 << 20
    x, g = logits(8, 3, V, torch.float32, std=0.5)
    u = [0.2, 0.6, 0.97]
    for kw in (dict(), dict(k=[100000, 5, 0], p=[0.9, 0.8, 0.95])):
        assert draw(native, eng, x, u, **kw) == want(x, u, **kw)


def test_many_rows(native, eng):
    x, g = logits(9, 700, 3001, torch.float32)
    u = g.random(700, dtype=np.float32).tolist()
    k, p = [40] * 700, [float(np.float32(0.92))] * 700
    assert draw(native, eng, x, u, k=k, p=p) == want(x, u, k=k, p=p)


@pytest.mark.parametrize("rows,V", [(320, 20011), (1024, 700), (1025, 700), (513, 33000)])
def test_rows_of_every_kind_in_one_batch(native, eng, rows, V):
    """More rows than run at once, which are taken by their work: greedy, unfiltered, short and long top-k and nuclei."""
    x, g = logits(rows, rows, V, torch.float32, std=2.0)
    u = g.random(rows, dtype=np.float32).tolist()
    t = [float(a) for a in np.float32(g.choice([0.0, 0.7, 1.0, 1.5], rows))]
    k = [int(a) for a in g.choice([0, 0, 5, 40, 1024, 1025, 5000], rows)]
    p = [float(a) for a in np.float32(g.choice([0.3, 0.9, 0.99, 1.0], rows))]
    assert draw(native, eng, x, u, t, k, p) == want(x, u, t, k, p)
    assert draw(native, eng, x, u, k=k) == want(x, u, k=k)


@pytest.mark.parametrize("name,value", [("t", -1.0), ("t", float("nan")), ("t", INF), ("t", 1.1e6), ("p", -0.1),
                                        ("p", 1.5), ("p", float("nan")), ("m", 2.0), ("m", float("nan")), ("u", 1.0),
                                        ("u", -0.5), ("u", float("nan"))])
def test_parameters_out_of_range(native, eng, name, value):
    """The row gives -1 and the engine reports a device error once; the other rows are sampled."""
    x, g = logits(10, 3, 200, torch.float32)
    kw = dict(u=[0.5] * 3, t=[1.0] * 3, p=[0.9] * 3, m=[0.0] * 3)
    good = want(x, **kw)
    kw[name] = [kw[name][0], value, kw[name][2]]
    got = draw(native, eng, x, **kw, sync=False)
    assert got[1] == -1 and got[0] == good[0] and got[2] == good[2]
    with pytest.raises(native.OrcaError) as e:
        eng.sync()
    assert e.value.code == native.ERR_DEVICE_FLAG
    eng.sync()


def test_refusals(native, eng):
    L, E, h = native.lib, native.ERR_INVALID, eng.handle
    x, o = torch.zeros(100, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    a, b = x.data_ptr(), o.data_ptr()
    for args in ((0, 0, 1, 10, 10, None, None, None, None, a, b), (0, a, 1, 10, 10, None, None, None, None, 0, b),
                 (0, a, 1, 10, 10, None, None, None, None, a, 0), (0, a, -1, 10, 10, None, None, None, None, a, b),
                 (0, a, 1, 0, 10, None, None, None, None, a, b), (0, a, 1, 10, 9, None, None, None, None, a, b),
                 (2, a, 1, 10, 10, None, None, None, None, a, b), (0, a + 2, 1, 10, 10, None, None, None, None, a, b),
                 (1, a + 1, 1, 10, 10, None, None, None, None, a, b), (0, a, 1, 10, 10, a + 1, None, None, None, a, b),
                 (0, a, 1, 10, 10, None, None, None, None, a, b + 2),
                 (0, a, 1, (1 << 20) + 1, 1 << 21, None, None, None, None, a, b)):
        assert L.orca_op_sample(h, *args) == E
    assert L.orca_op_sample(h, 0, a, 0, 10, 10, None, None, None, None, a, b) == 0
    eng.sync()


def test_captured(native):
    st = torch.cuda.Stream()
    e = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None, st.cuda_stream)
    try:
        x, g = logits(11, 6, 2000, torch.float32)
        with torch.cuda.stream(st):
            xd, u = x.cuda(), torch.full((6,), 0.3, device="cuda")
            p, out = torch.full((6,), 0.5, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=st):
                e.op_sample(native.DTYPE_FP32, xd.data_ptr(), 6, 2000, out.data_ptr(), u.data_ptr(),
                            top_p=p.data_ptr(), sync=False)
            for v in (0.1, 0.8):
                u.fill_(v)
                gr.replay()
                e.sync()
                assert out.tolist() == want(x, [v] * 6, p=[0.5] * 6)
    finally:
        e.close()
