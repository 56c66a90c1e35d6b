"""Host side of the 4-bit K/V cache and of sampling: sizes, plans and refusals.  No GPU."""

import ctypes as C

import numpy as np
import pytest

from iteration_level_scheduling_gb300 import build
from oracle import kv4


@pytest.fixture(scope="module")
def native():
    build.build()
    from iteration_level_scheduling_gb300 import native as n
    return n


def words(native, dtype=1, heads=4, d=64, slots=100, n=(1,), c=(10,), o=(3,), eng=None):
    n, c, o = np.array(n, np.int32), np.array(c, np.int32), np.array(o, np.int64)
    return native.lib.orca_kv4_plan_words(eng, dtype, heads, d, slots, len(n), n.ctypes.data, c.ctypes.data,
                                          o.ctypes.data)


def plan(native, dtype=1, heads=4, d=64, slots=100, n=(1,), c=(10,), o=(3,)):
    w = words(native, dtype, heads, d, slots, n, c, o)
    assert w > 0
    buf = np.zeros(w, np.int32)
    n, c, o = np.array(n, np.int32), np.array(c, np.int32), np.array(o, np.int64)
    assert native.lib.orca_kv4_plan_build(None, dtype, heads, d, slots, len(n), n.ctypes.data, c.ctypes.data,
                                          o.ctypes.data, buf.ctypes.data, w) == 0
    return buf


@pytest.mark.parametrize("heads,d,slots", [(1, 16, 1), (3, 32, 17), (40, 128, 4096), (7, 64, 15)])
def test_layer_bytes(native, heads, d, slots):
    S, G = (slots + 15) // 16 * 16, max(1, d // 32)
    want = 2 * heads * S * (d // 2 + 4 * G)
    assert native.kv4_layer_bytes(heads, d, slots) == want
    kv4.Layer(heads, d, slots, np.zeros(want, np.uint8))


@pytest.mark.parametrize("bad", [(0, 64, 10), (1025, 64, 10), (4, 48, 10), (4, 256, 10), (4, 64, 0),
                                 (4, 64, 2 ** 31 - 1)])
def test_layer_bytes_refusals(native, bad):
    with pytest.raises(native.OrcaError) as e:
        native.kv4_layer_bytes(*bad)
    assert e.value.code == native.ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(heads=0), dict(d=20), dict(slots=0),
    dict(n=(0,)), dict(c=(-1,)), dict(o=(-1,)), dict(slots=13), dict(o=(2 ** 40,)),
    dict(n=(1, 2 ** 31 - 1), c=(0, 0), o=(0, 1), slots=2 ** 31 - 16),  # tables beyond 32-bit offsets
])
def test_plan_refusals(native, kw):
    assert words(native, **kw) == native.ERR_INVALID


def test_plan_null_arrays_and_short_buffer(native):
    a = np.array([1], np.int32)
    o = np.array([0], np.int64)
    args = [None, 1, 4, 64, 100, 1, a.ctypes.data, a.ctypes.data, o.ctypes.data]
    w = native.lib.orca_kv4_plan_words(*args)
    buf = np.zeros(w, np.int32)
    assert native.lib.orca_kv4_plan_build(*args, buf.ctypes.data, w - 1) == native.ERR_INVALID
    assert not buf.any()
    assert native.lib.orca_kv4_plan_build(*args, None, w) == native.ERR_INVALID
    for i in (6, 7, 8):
        bad = list(args)
        bad[i] = None
        assert native.lib.orca_kv4_plan_words(*bad) == native.ERR_INVALID
    args[5] = 0
    assert native.lib.orca_kv4_plan_words(*args) == native.ERR_INVALID


def test_workspace_of_something_else(native):
    junk = np.zeros(64, np.int32)
    assert native.lib.orca_kv4_workspace_bytes(junk.ctypes.data) == native.ERR_INVALID
    assert native.lib.orca_kv4_workspace_bytes(None) == native.ERR_INVALID


def test_operators_need_an_engine(native):
    p = plan(native)
    assert native.lib.orca_op_kv4_append(None, 16, 16, p.ctypes.data, 16) == native.ERR_INVALID
    assert native.lib.orca_op_kv4_read(None, 16, p.ctypes.data, 16, 16) == native.ERR_INVALID
    assert native.lib.orca_op_kv4_attention(None, 16, 16, p.ctypes.data, 16, 16, 16) == native.ERR_INVALID
    assert native.lib.orca_op_sample(None, 0, 16, 1, 10, 10, None, None, None, None, 16, 16) == native.ERR_INVALID
    assert native.lib.orca_sample_last(None, None, None, None, None, 16, None) == native.ERR_INVALID


def test_oracle_quantise_ties_and_edges():
    """Worked by hand: scale 1, minimum 0; halves go to the even code; -0, constants, non-finite groups."""
    x = np.zeros((1, 32), np.float32)
    x[0, :6] = [0, 15, 0.5, 1.5, 2.5, 14.5]
    c, s, m = kv4.quantise(x)
    assert s[0, 0] == 1 and m[0, 0] == 0
    assert c[0, :6].tolist() == [0, 15, 0, 2, 2, 14]
    c, s, m = kv4.quantise(np.full((1, 32), -3.5, np.float32))
    assert s[0, 0] == 0 and m[0, 0] == -3.5 and not c.any()
    for bad in (np.inf, -np.inf, np.nan):
        x[0, 7] = bad
        assert np.isnan(kv4.stands_for(*kv4.quantise(x))).all()


def test_addresses_of_arrays(native):
    """Arrays of every kind that a caller may pass: writable, read-only (a plan kept unchanged), empty, a view."""
    plan = np.arange(12, dtype=np.int32)
    fixed = plan.copy()
    fixed.setflags(write=False)
    for a in (plan, fixed, plan[:0], plan[3:], plan[::2], plan.reshape(3, 4).T):
        assert native._ptr(a) == a.__array_interface__["data"][0] or a.size == 0


@pytest.mark.parametrize("dtype,d,reqs", [
    (0, 128, [(8192, 24576)]), (0, 128, [(2048, 30000)]), (0, 64, [(4096, 0), (512, 60000), (1, 900)]),
    (1, 32, [(8192, 24576)]), (1, 16, [(3000, 100000)] * 2), (0, 128, [(20, 500000)]), (0, 16, [(16, 2000000)]),
])
def test_workspace_of_long_prompts_in_groups(native, dtype, d, reqs):
    """Prompts that run in groups of rows: the partial outputs of their chunks stay below half of the K/V in
    fp32 (32 heads, every key of the batch), or below 64 MiB."""
    n, c = zip(*reqs)
    o = np.cumsum([0] + [a + b for a, b in reqs])
    p = plan(native, dtype, 32, d, int(o[-1]), n, c, o[:-1])
    keys = int(o[-1])
    assert native.lib.orca_kv4_workspace_bytes(p.ctypes.data) <= max(64 << 20, 2 * 32 * keys * d * 4 // 2)


def test_quantisation_error():
    """Between the ends of what is held a component is off by half a step at most.  At the ends by what s and m lost to
    bf16 (2^-8 each): 2^-8 of the range and 2^-8 of the minimum, which is more than half a step once the minimum is
    some seven times the range or more."""
    g = np.random.default_rng(1)
    for offset in (0.0, 1.0, 10.0, 100.0):
        x = (g.standard_normal((2000, 32)) + offset).astype(np.float32)
        c, s, m = kv4.quantise(x)
        off = np.abs(kv4.stands_for(c, s, m) - x).max(1)
        lo, hi = x.min(1).astype(np.float64), x.max(1).astype(np.float64)
        half, ends = s[:, 0] / 2.0, 2.0 ** -8 * (hi - lo + np.abs(lo))
        assert (off <= np.maximum(half, ends) * (1 + 2.0 ** -20)).all()
        assert (off <= half * (1 + 2.0 ** -6)).all() or offset > 1


def test_attention_before_and_after_quantisation():
    """Attention over what the cache stands for against attention over the rows as they were.  Of independent errors a
    key's s / sqrt(12) moves a score by as much (|q| = sqrt(d)) and its weight by that share, a value's moves the output
    like the values themselves: together sqrt(2) s / sqrt(12) of the output's root mean square (values of variance one),
    taken half as large again."""
    g = np.random.default_rng(2)
    for d in (64, 128):
        q, k, v = g.standard_normal((20, 4, d)), g.standard_normal((4, 500, d)), g.standard_normal((4, 500, d))
        kc, vc = kv4.quantise(k), kv4.quantise(v)
        out, ref = kv4.attention(q, kv4.stands_for(*kc), kv4.stands_for(*vc), 480), kv4.attention(q, k, v, 480)
        step = np.sqrt((kc[1].astype(np.float64) ** 2).mean())
        assert np.sqrt(((out - ref) ** 2).mean()) <= 1.5 * np.sqrt(2 / 12) * step * np.sqrt((ref ** 2).mean())
