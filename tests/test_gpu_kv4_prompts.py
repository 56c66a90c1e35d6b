"""Prompts over the 4-bit K/V cache that run on the prefill kernel, whose operands are fp16: where fp16's range, and not
its precision, would decide the result.  Batches are built so that the plan chooses that kernel, which each test
asserts from the plan's header."""

import math

import numpy as np
import pytest
import torch

from test_gpu_kv4 import Case, eng, native, rounded  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

Q_PRE = 18  # word of a plan's header: requests on the prefill kernel


def on_prefill_kernel(plan, n):
    assert plan[Q_PRE] == n


@pytest.mark.parametrize("d,heads,lead", [(128, 2, 1.5625), (64, 16, 2.1875)])
def test_many_small_weights_count(native, eng, d, heads, lead):  # noqa: F811
    """A key far ahead of 20000 others, each of about 2^-25.4 of its weight: together they weigh 2^-11, and since the
    leading key's value is 0 and the others' is 1, the output is what they weigh.

    The inputs are exact in 4 bits and in fp16 (each group constant).  Errors: bf16 rounding of the output 2^-9 (taken
    as a whole step, 2^-8), fp16 weights 2^-11, the exponential's and the sums' fp32 2^-18; and for weights below fp16's
    normal range 2^-25 of what 1 stands for, 2^-11 of the largest weight or less: keys 2^-36."""
    keys, rows = 20000, 512
    H, slots = heads * d, keys + rows
    layer = torch.full((native.kv4_layer_bytes(heads, d, slots),), 0xFF, dtype=torch.uint8, device="cuda")

    def qkv(n, first_ahead):
        x = torch.zeros((n, 3, H), dtype=torch.bfloat16, device="cuda")
        x[:, 0], x[:, 2] = 1, 1
        if first_ahead:
            x[0, 1], x[0, 2] = lead, 0
        return x.view(n, 3 * H)

    for n, c in ((keys, 0), (rows, keys)):
        x = qkv(n, c == 0)
        plan = eng.kv4_plan(native.DTYPE_BF16, heads, d, slots, [n], [c], [0])
        dplan = torch.from_numpy(plan).cuda()
        eng.op_kv4_append(x.data_ptr(), layer.data_ptr(), plan, dplan.data_ptr())
    on_prefill_kernel(plan, 1)
    work = torch.full((eng.kv4_workspace_bytes(plan),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((rows, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    eng.op_kv4_attention(x.data_ptr(), layer.data_ptr(), plan, dplan.data_ptr(), work.data_ptr(), out.data_ptr())
    others = (keys + np.arange(rows)) * math.exp(-lead * math.sqrt(d))
    ref = (others / (1 + others))[:, None]
    got = out.float().cpu().numpy().astype(np.float64)
    assert (np.abs(got - ref) <= ref * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) + (keys + rows) * 2.0 ** -36).all()


def prompt_bound(s, req, r0):
    """Reference and bound of a prompt's rows: [n, heads, d] each.  A score sum q k / sqrt(d) is off by 2^-11 of
    sum |q k| / sqrt(d) (k in fp16; q has bf16's 8 bits) and by fp32's (d + 16) 2^-23 of it, by which its weight's
    logarithm is off; the weight and the value are rounded to fp16, 2^-11 each; weights below fp16's normal range are
    off by 2^-36 of the largest, and values of a group more than 2^28 below the largest are not left to fp16.  With
    a(k) the first of these, the output, a mean of the values, moves by at most
    sum_k p_k (e^a(k) - 1) (|v_k| + |out|), and so on; products of two errors are covered by 1 %."""
    n, c, o = s.n[req], s.c[req], s.off[req]
    k, v = s.layer.read(o, c + n)
    q = s.qkv[r0:r0 + n, 0].astype(np.float64)
    sees = np.arange(c + n)[None, :] <= c + np.arange(n)[:, None]
    ref, lim = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(s.heads):
        # what a row does not see takes no part: also not through 0 times a large number
        x = q[:, h] @ k[h].T / math.sqrt(s.d)
        a = np.abs(q[:, h]) @ np.abs(k[h]).T / math.sqrt(s.d) * (2.0 ** -11 + (s.d + 16) * 2.0 ** -23)
        x, a = np.where(sees, x, -np.inf), np.where(sees, a, 0.0)
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out = p @ v[h]
        w = np.where(p > 0, p * np.expm1(np.where(p > 0, a, 0.0)), 0.0)
        top = np.abs(v[h]).max(1)
        top = np.where(sees, top[None, :], 0.0).max(1, keepdims=True)
        err = w @ np.abs(v[h]) + w.sum(1, keepdims=True) * np.abs(out) + 2 * 2.0 ** -11 * (p @ np.abs(v[h]))
        err = 1.01 * err + (c + n) * 2.0 ** -36 * top
        ref[:, h], lim[:, h] = out, err + 2.0 ** -8 * (np.abs(out) + err)
    return ref, lim


def attend(s):
    s.append()
    s.append_oracle()
    return s.attention().float().cpu().numpy().reshape(len(s.qkv), s.heads, s.d).astype(np.float64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", [1, 2])  # a key, a value
@pytest.mark.parametrize("at,size", [(300, 2.0 ** 45), (290, 2.0 ** 33), (120, 2.0 ** -60)])
def test_one_row_of_another_size(native, eng, d, which, at, size):  # noqa: F811
    """The K or V of one row of one head many orders of magnitude above (or below) the others': the rows before it do
    not see it and are what they are without it, the rows behind it have it among their keys."""
    s = Case(native, eng, 40, "bf16", 40, d, [(300, 150), (200, 10)])
    on_prefill_kernel(s.plan, 2)
    at -= 1
    s.qkv[at, which, 7] *= np.float32(size)
    if which == 1 and size > 1:
        s.qkv[at, 1, 7] = -np.abs(s.qkv[at, 1, 7])
        s.qkv[at:300, 0, 7] = np.abs(s.qkv[at:300, 0, 7])  # (a score of no weight, whatever fp32 makes of its size)
    s.qkv = rounded(s.qkv, "bf16").float().numpy()
    s.upload()
    got = attend(s)
    for req, r0 in ((0, 0), (1, 300)):
        ref, lim = prompt_bound(s, req, r0)
        d_ = np.abs(got[r0:r0 + s.n[req]] - ref)
        assert np.isfinite(d_).all() and (d_ <= lim).all(), float((d_ / np.maximum(lim, 1e-300)).max())
