"""Attention over the 4-bit K/V cache by the form that a plan gives each request -- single rows (whole or split), groups
of rows (whole or split), prompts on the prefill kernel -- and by several of them in one call.  Every test asserts from
the plan's header that the forms it is about are there, and every request is held to the bound of its own form."""

import math

import numpy as np
import pytest
import torch

from oracle import kv4
from test_gpu_kv4 import Case, eng, native, rounded  # noqa: F401 (fixtures)
from test_gpu_kv4_prompts import prompt_bound

pytestmark = pytest.mark.gpu

# words of a plan's header
ITEMS, SPLITS, PRE, O_PRE, RITEMS, RJOINS = 6, 7, 18, 23, 28, 30


def forms(s, **want):
    p = s.plan
    got = dict(singles=p[ITEMS] > 0, split_singles=p[SPLITS] > 0, groups=p[RITEMS] > 0, split_groups=p[RJOINS] > 0,
               prompts=p[PRE])
    assert all(got[k] == v for k, v in want.items()), got
    return s


def check(s, out, rms=True):
    """Rows on the codes themselves: scores to (d + 16) 2^-24 of sum |q k| (natural logarithm; the doubled term is
    numerator and denominator), weights as two bf16 (2^-16), fp32 sums 2^-24 per key; the output's rounding is eps / 2.
    Prompts: prompt_bound, and since that is a worst case, their root mean square error over request and head, which
    random roundings make about 2^-9.7 of the output's (bf16's 2^-9 / sqrt(3), fp16's thrice 2^-11 / sqrt(3) in
    quadrature): 2^-8 at most."""
    got = out.float().cpu().numpy().reshape(len(s.qkv), s.heads, s.d).astype(np.float64)
    eps = torch.finfo(out.dtype).eps / 2
    prompts = {int(s.plan[s.plan[O_PRE] + 4 * i]) for i in range(s.plan[PRE])}
    r = 0
    for i, (n, c, o) in enumerate(zip(s.n, s.c, s.off)):
        if i in prompts:
            ref, lim = prompt_bound(s, i, r)
        else:
            k, v = s.layer.read(o, c + n)
            q = s.qkv[r:r + n, 0].astype(np.float64)
            ref = kv4.attention(q, k, v, c)
            size = np.abs(q).transpose(1, 0, 2) @ np.abs(k).transpose(0, 2, 1) / math.sqrt(s.d)  # [heads, n, keys]
            tol = 4 * (s.d + 16) * 2.0 ** -24 * size.max(2) + 2.0 ** -15 + (c + n) * 2.0 ** -24
            lim = eps * np.abs(ref) + (tol * np.abs(v).max((1, 2))[:, None]).T[:, :, None]
        d = np.abs(got[r:r + n] - ref)
        assert np.isfinite(d).all() and (d <= lim).all(), (i, n, c, float((d / lim).max()))
        if i in prompts and rms:
            e, a = np.sqrt((d ** 2).mean((0, 2))), np.sqrt((ref ** 2).mean((0, 2)))
            assert (e <= 2.0 ** -8 * a).all(), (i, float((e / a).max()))
        r += n


def run(s, **kw):
    s.append()
    s.append_oracle()
    out = s.attention()
    check(s, out, **kw)
    return out


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_groups_and_single_rows_in_one_call(native, eng, d):  # noqa: F811
    """Each request in the form that is cheaper for it: prompts beside groups (split) and single rows (split and not)."""
    s = Case(native, eng, 50, "bf16", 40, d, [(500, 0), (2, 1200), (1, 5200), (2, 1200), (1, 40), (3, 1200), (2, 1200)])
    run(forms(s, prompts=1, groups=True, split_groups=True, singles=True, split_singles=True))


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_tiles_of_one_row(native, eng, d):  # noqa: F811
    """129 and 257 rows: the last tile of the prefill kernel has one; a split single row beside them."""
    s = Case(native, eng, 51, "bf16", 40, d, [(129, 300), (257, 100), (1, 900)])
    run(forms(s, prompts=2, groups=False, split_singles=True))


@pytest.mark.parametrize("dtype,d", [("bf16", 32), ("bf16", 16), ("fp32", 128), ("fp32", 64), ("fp32", 32), ("fp32", 16)])
def test_prompts_in_groups(native, eng, dtype, d):  # noqa: F811
    """What the prefill kernel does not take, by the bound of exact codes."""
    s = Case(native, eng, 52, dtype, 3, d, [(130, 0), (127, 200), (257, 65), (1, 300), (33, 1)])
    run(forms(s, prompts=0, groups=True))


SEVERAL = [(500, 0), (2, 1200), (1, 5200), (2, 1200), (1, 40)]  # at 40 heads of 128 in all forms


def test_a_wide_head_beside_other_forms(native, eng):  # noqa: F811
    """A prompt that is neither the first request nor alone, with one head whose values fp16 does not hold (attended on
    the codes), beside groups and single rows."""
    s = forms(Case(native, eng, 57, "bf16", 40, 128, SEVERAL[1:3] + SEVERAL[:1] + SEVERAL[3:]), prompts=1, groups=True,
              split_groups=True, split_singles=True)
    first = sum(s.n[:2])
    s.qkv[first + 480, 2, 11] *= np.float32(2.0 ** 50)
    s.qkv = rounded(s.qkv, "bf16").float().numpy()
    s.upload()
    run(s, rms=False)


def test_all_forms_captured(native):  # noqa: F811
    """Append and attention captured with prompts, groups and split single rows in the call, and replayed over changed
    inputs: the arrival counters in the plan's device copy are found at zero by every replay."""
    st = torch.cuda.Stream()
    e = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None, st.cuda_stream)
    try:
        with torch.cuda.stream(st):
            s = Case(native, e, 53, "bf16", 40, 128, SEVERAL)
            forms(s, prompts=1, groups=True, split_groups=True, split_singles=True)
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
                step()
            for i in range(2):
                s.qkv = s.qkv[::-1].copy()
                s.dqkv.copy_(rounded(s.qkv.reshape(len(s.qkv), -1), "bf16").cuda())
                gr.replay()
                e.sync()
                s.append_oracle()
                check(s, out)
            assert np.array_equal(s.dplan.cpu().numpy(), s.plan)
            want = out.clone()
            for i in range(10):
                gr.replay()
            e.sync()
            assert torch.equal(out, want)
    finally:
        e.close()


def test_all_forms_on_two_streams(native):  # noqa: F811
    """Two engines on streams of their own, each with its layer, plan and workspace, queued without a wait: every
    output has the bits of the same call alone."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    engines = [native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None, st.cuda_stream)
               for st in streams]
    cases, outs, alone = [], [], []
    for i, (e, st) in enumerate(zip(engines, streams)):
        with torch.cuda.stream(st):
            s = Case(native, e, 54 + i, "bf16", 40, 128, SEVERAL[i:] + SEVERAL[:i])
            forms(s, prompts=1, groups=True, split_groups=True, split_singles=True)
            s.append()
            s.append_oracle()
            alone.append(s.attention())
            check(s, alone[i])
            cases.append(s)
            outs.append([torch.zeros_like(alone[i]) for _ in range(20)])
    torch.cuda.synchronize()
    for k in range(20):
        for s, e, o in zip(cases, engines, outs):
            s.append(sync=False)
            e.op_kv4_attention(s.dqkv.data_ptr(), s.dev.data_ptr(), s.plan, s.dplan.data_ptr(), s.work.data_ptr(),
                               o[k].data_ptr(), sync=False)
    for e, o, a in zip(engines, outs, alone):
        e.sync()
        assert all(torch.equal(x, a) for x in o)
        e.close()


def test_a_row_alone_and_in_company(native, eng):  # noqa: F811
    """A row's output has the same bits alone and beside others where the plan splits its keys alike, in every form; and
    call after call whatever the plan."""
    def part(s, r, n):
        """The requests of s from r on, n of them, on s's own layer and rows, by a plan of their own."""
        first = sum(s.n[:r])
        t = Case.__new__(Case)
        t.__dict__.update(s.__dict__)
        t.n, t.c, t.off = s.n[r:r + n], s.c[r:r + n], s.off[r:r + n]
        t.qkv, t.dqkv = s.qkv[first:first + sum(t.n)], s.dqkv[first:first + sum(t.n)].contiguous()
        t.plan = eng.kv4_plan(native.DTYPE_BF16, s.heads, s.d, s.slots, t.n, t.c, t.off)
        t.dplan = torch.from_numpy(t.plan).cuda()
        t.work = torch.full((max(1, eng.kv4_workspace_bytes(t.plan)),), 0xFF, dtype=torch.uint8, device="cuda")
        return t, slice(first, first + sum(t.n))

    for heads, reqs in ((40, [(1, 300), (1, 390), (1, 7)]), (40, [(1, 900), (1, 1300)]), (2, [(3, 90), (2, 20), (7, 60)]),
                        (40, [(300, 300), (350, 150)])):
        s = Case(native, eng, 56, "bf16", heads, 128, reqs)
        s.append()
        whole = s.attention()
        for _ in range(3):
            assert torch.equal(s.attention(), whole)
        for r in range(len(reqs)):
            t, rows = part(s, r, 1)
            splits = lambda p: sorted(p[p[15] + 8 * i + 3] for i in range(p[ITEMS]))  # noqa: E731 (chunks of a row)
            assert set(splits(t.plan)) <= set(splits(s.plan)) and t.plan[RJOINS] == 0 and s.plan[RJOINS] == 0
            assert bool(t.plan[PRE]) == bool(s.plan[PRE])
            assert torch.equal(t.attention(), whole[rows]), (reqs, r)
