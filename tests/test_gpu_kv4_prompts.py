"""Prompts over the 4-bit K/V cache that run on the prefill kernel, whose operands are fp16: where fp16's range, and not
its precision, would decide the result.  Batches are built so that the plan chooses that kernel, which each test
asserts from the plan's header."""

import math

import numpy as np
import pytest
import torch

from test_gpu_kv4 import eng, native  # noqa: F401 (fixtures)

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
