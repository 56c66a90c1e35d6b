"""What programmatic launches guarantee, by a model over the order of `pdl_trigger` and `pdl_wait` in the kernels' source
(no GPU).

A kernel launched behind another may start once every block of that one has triggered or ended.  `pdl_wait` returns when
the kernel in front has ended, and with it every kernel in front of that.  So at the start of kernel i, before its own
wait, the kernels that have ended for certain are all of those in front of kernel i - 1 if i - 1 triggers behind its
wait, and otherwise only those that had ended for certain when i - 1 itself started.  A chain of kernels that trigger
first lets the last of them start while the first still runs.

Three kernels load data ahead of their wait: tensor-core decode attention (keys in front of the iteration's own), the
tcgen05 GEMM (weights) and the row groups behind 4-bit prompts (the marks of heads that fp16 does not hold)."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "iteration_level_scheduling_gb300",
                    "csrc")


def body(file, kernel):
    text = open(os.path.join(CSRC, file)).read()
    at = re.search(r"\b" + kernel + r"\s*\(", text).start()
    end = text.find("__global__", at)
    return re.sub(r"//[^\n]*", "", text[at:end if end >= 0 else len(text)])


def triggers_behind_wait(file, kernel):
    """Of the first of each in the source (a kernel without a trigger triggers when it ends)."""
    b = body(file, kernel)
    wait, trigger = b.find("pdl_wait()"), b.find("pdl_trigger()")
    assert wait >= 0, kernel
    return trigger < 0 or wait < trigger


def ended_at_start(chain):
    """For every kernel of the chain, how many kernels of it have ended for certain when it starts."""
    ended = [0]
    for i in range(1, len(chain)):
        never = chain[i - 1] is None  # no trigger at all: ends first
        ended.append(i if never else i - 1 if chain[i - 1] else ended[i - 1])
    return ended


def kind(file, kernel):
    return None if "pdl_trigger()" not in body(file, kernel) else triggers_behind_wait(file, kernel)


def test_the_model():
    assert ended_at_start([False, False, False, False]) == [0, 0, 0, 0]
    assert ended_at_start([False, True, False, False]) == [0, 0, 1, 1]
    assert ended_at_start([None, False, False]) == [0, 1, 1]


def test_decode_starts_behind_what_wrote_its_pool_before_the_iteration():
    """An iteration, planned beforehand, straight behind a 4-bit read-back into the pool, or behind the iteration
    before: decode attention's early loads must find all that was written in front of the iteration."""
    layer = [("k_misc.cu", "layernorm_kernel"), ("k_gemm_tc.cu", "gemm_tc_kernel")]
    for first in (("k_kv4.cu", "kv4_read_kernel"), ("k_kv4.cu", "kv4_read_few_kernel"), ("k_misc.cu", "argmax_kernel"),
                  ("k_sample.cu", "sample_kernel")):
        chain = [kind(*k) for k in [first, ("k_misc.cu", "embed_kernel")] + layer]
        assert ended_at_start(chain + [False])[-1] >= 1, first


def test_the_gemm_starts_behind_what_packed_its_weights():
    """A linear layer straight behind the packing of its weights, which it loads ahead of its wait."""
    for gemm in ("gemm_tc_kernel", "gemm_sk_kernel"):
        assert body("k_gemm_tc.cu", gemm).find("pdl_trigger()") >= 0
        assert ended_at_start([kind("k_gemm_tc.cu", "pack_weight_kernel"), False])[-1] == 1


def test_row_groups_behind_prompts_start_behind_what_marked_their_heads():
    """prep, read, prefill on fp16 operands, row groups: the marks are prep's."""
    b = body("k_attn.cu", "attn_prefill_tc_kernel").replace("if constexpr (!F16) pdl_trigger();", "")
    late = 0 <= b.find("pdl_wait()") < b.find("pdl_trigger()")
    chain = [kind("k_kv4.cu", "kv4_prep_kernel"), kind("k_kv4.cu", "kv4_read_kernel"), late]
    wide = body("k_kv4.cu", "kv4_rows_wide_kernel")
    assert wide.find("a.wide + i") < wide.find("pdl_wait()")
    assert ended_at_start(chain + [False])[-1] >= 1
