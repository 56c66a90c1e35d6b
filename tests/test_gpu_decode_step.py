"""The operators of a decode step together, as a serving program runs them: the K/V of the rows written to a 4-bit
cache layer, attention over it, the output projection and the LM head, a token sampled per request -- several steps in
a row, each step's token choosing the next one's input -- and sampling inside the engine's own iterations."""

import numpy as np
import pytest
import torch

from iteration_level_scheduling_gb300 import synth
from oracle import kv4
from oracle.sampling import sample

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def native():
    from iteration_level_scheduling_gb300 import build
    build.build()
    from iteration_level_scheduling_gb300 import native as n
    return n


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_one_layer(native, captured):
    """One attention layer between an embedding and an LM head, three requests, a prompt and three increments.  Every
    operator reads what the one before wrote on the device; nothing waits in between.  Each operator is compared with
    float64 on the inputs that it was given on the device (the tolerances are then its own)."""
    heads, d, V, slots = 4, 64, 1000, 400
    H = heads * d
    g = np.random.default_rng(3)
    st = torch.cuda.Stream()
    eng = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None, st.cuda_stream)
    with torch.cuda.stream(st):
        emb = bf16(g.standard_normal((V, H))).cuda()
        wq = bf16(g.standard_normal((3 * H, H)) / 16).cuda()
        wo = bf16(g.standard_normal((H, H)) / 16).cuda()
        layer = torch.full((native.kv4_layer_bytes(heads, d, slots),), 0xFF, dtype=torch.uint8, device="cuda")
        host = np.full(layer.numel(), 0xFF, np.uint8)
        oracle = kv4.Layer(heads, d, slots, host)
        off, n, ctx = [1, 140, 250], [70, 5, 1], [0, 0, 0]
        tokens = torch.from_numpy(g.integers(0, V, sum(n))).cuda()
        t, k = torch.tensor([0.7, 1.0, 0.0], device="cuda"), torch.tensor([40, 0, 0], dtype=torch.int32, device="cuda")
        p, m = torch.tensor([0.9, 0.95, 1.0], device="cuda"), torch.tensor([0.0, 0.02, 0.0], device="cuda")
        for it in range(4):
            rows = sum(n)
            x = emb[tokens].contiguous()
            qkv = torch.zeros((rows, 3 * H), dtype=torch.bfloat16, device="cuda")
            att, y = torch.zeros_like(x), torch.zeros_like(x)
            logits = torch.zeros((3, V), device="cuda")
            last = torch.cumsum(torch.tensor(n), 0).cuda() - 1
            lasts = torch.zeros((3, H), dtype=torch.bfloat16, device="cuda")
            u = torch.from_numpy(g.random(3, dtype=np.float32)).cuda()
            out = torch.zeros(3, dtype=torch.int32, device="cuda")
            plan = eng.kv4_plan(native.DTYPE_BF16, heads, d, slots, n, ctx, off)
            dplan = torch.from_numpy(plan).cuda()
            work = torch.zeros(max(16, eng.kv4_workspace_bytes(plan)), dtype=torch.uint8, device="cuda")

            def step():
                B = native.DTYPE_BF16
                eng.op_linear(B, x.data_ptr(), wq.data_ptr(), rows, 3 * H, H, out_bf16=qkv.data_ptr(), sync=False)
                eng.op_kv4_append(qkv.data_ptr(), layer.data_ptr(), plan, dplan.data_ptr(), sync=False)
                eng.op_kv4_attention(qkv.data_ptr(), layer.data_ptr(), plan, dplan.data_ptr(), work.data_ptr(),
                                     att.data_ptr(), sync=False)
                eng.op_linear(B, att.data_ptr(), wo.data_ptr(), rows, H, H, out_bf16=y.data_ptr(), sync=False)
                torch.index_select(y, 0, last, out=lasts)
                eng.op_linear(B, lasts.data_ptr(), emb.data_ptr(), 3, V, H, out_f32=logits.data_ptr(), sync=False)
                eng.op_sample(native.DTYPE_FP32, logits.data_ptr(), 3, V, out.data_ptr(), u.data_ptr(),
                              temperature=t.data_ptr(), top_k=k.data_ptr(), top_p=p.data_ptr(), min_p=m.data_ptr(),
                              sync=False)

            if captured:  # a step twice over the same slots writes the same bytes
                step()
                eng.sync()
                gr = torch.cuda.CUDAGraph()
                with torch.cuda.graph(gr, stream=st):
                    step()
                att.zero_(), out.zero_(), logits.zero_()
                gr.replay()
            else:
                step()
            eng.sync()
            f = qkv.float().cpu().numpy().reshape(rows, 3, heads, d)
            r = 0
            for ni, c, o in zip(n, ctx, off):
                for j in range(ni):
                    oracle.write(o + c + j, f[r + j, 1], f[r + j, 2])
                kk, vv = oracle.read(o, c + ni)
                ref = kv4.attention(f[r:r + ni, 0].astype(np.float64), kk, vv, c)
                err = np.abs(att[r:r + ni].float().cpu().numpy().reshape(ni, heads, d) - ref)
                # the last rounding, and 2^-9 of the largest value for what prompts round to fp16 (2^-11 on the weight,
                # the value and, times the score's size of at most 2, the score)
                assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * np.abs(vv).max()).all()
                r += ni
            z = logits.cpu().numpy()
            want = [sample(z[i], u[i].item(), t[i].item(), k[i].item(), p[i].item(), m[i].item()) for i in range(3)]
            assert out.tolist() == want
            ctx = [a + b for a, b in zip(ctx, n)]
            n = [1, 1, 1]
            tokens = out.long()
    eng.close()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sampling_in_the_engines_iterations(native, dtype):
    """orca_sample_last: the tokens are those of the iteration's logits, and the next iteration's references mean them."""
    from gpu_util import make_engine
    cfg = synth.ModelConfig(n_layers=2, hidden=128, n_heads=2, ffn=256, vocab=700, max_pos=64, dtype=dtype)
    w = synth.make_weights(cfg, 5, random_affine=True, std=0.2)
    prompts = [[3, 1, 4, 1, 5], [9, 2], [6, 5, 3, 5, 8, 9, 7]]
    g = np.random.default_rng(1)
    t, p = torch.tensor([2.0, 1.0, 0.0], device="cuda"), torch.tensor([0.9, 1.0, 1.0], device="cuda")

    def first(eng):
        offs = [eng.kv_alloc(i, 64) for i in range(3)]
        eng.run_iteration(native.BatchDesc([0, 1, 2], [0, 0, 0], [len(a) for a in prompts], [0, 0, 0], offs,
                                           sum(prompts, [])))
        return offs

    a, b = make_engine(cfg, w, 64, 4, 256), make_engine(cfg, w, 64, 4, 256)
    try:
        with pytest.raises(native.OrcaError) as e:
            a.sample_last(t.data_ptr())
        assert e.value.code == native.ERR_INVALID  # nothing has run
        offs = first(a)
        first(b)
        ctx = [len(x) for x in prompts]
        for it in range(3):
            u = torch.from_numpy(g.random(3, dtype=np.float32)).cuda()
            out = torch.zeros(3, dtype=torch.int32, device="cuda")
            z = a.last_logits(3)
            a.sample_last(u.data_ptr(), temperature=t.data_ptr(), top_p=p.data_ptr(), out_tokens=out.data_ptr())
            tok = out.tolist()
            assert tok == [sample(z[i], u[i].item(), t[i].item(), 0, p[i].item()) for i in range(3)]
            assert tok[2] == int(z[2].argmax())
            # by reference in one engine, by value in the other
            a.run_iteration(native.BatchDesc([0, 1, 2], [1] * 3, [1] * 3, ctx, offs, [-1, -2, -3]))
            b.run_iteration(native.BatchDesc([0, 1, 2], [1] * 3, [1] * 3, ctx, offs, tok))
            assert np.array_equal(a.last_logits(3), b.last_logits(3))
            ctx = [c + 1 for c in ctx]
    finally:
        a.close()
        b.close()


def test_sampling_between_planned_iterations(native):
    """Planned iterations and sampling queued one behind the other, tokens passed on by reference, nothing read back in
    between: the tokens of a run that waits for every step and passes them by value."""
    from gpu_util import make_engine
    cfg = synth.ModelConfig(n_layers=2, hidden=128, n_heads=2, ffn=256, vocab=700, max_pos=64, dtype="bf16")
    w = synth.make_weights(cfg, 6, random_affine=True, std=0.2)
    prompts, steps = [[3, 1, 4, 1, 5], [9, 2], [6, 5, 3, 5, 8, 9, 7]], 6
    lens = [len(x) for x in prompts]
    u = torch.from_numpy(np.random.default_rng(2).random((steps, 3), dtype=np.float32)).cuda()
    t, p = torch.tensor([2.0, 1.0, 0.0], device="cuda"), torch.tensor([0.9, 1.0, 1.0], device="cuda")

    def batch(it, offs, tokens):
        if it == 0:
            return native.BatchDesc([0, 1, 2], [0] * 3, lens, [0] * 3, offs, sum(prompts, []))
        return native.BatchDesc([0, 1, 2], [1] * 3, [1] * 3, [n + it - 1 for n in lens], offs, tokens)

    a, b = make_engine(cfg, w, 64, 4, 256), make_engine(cfg, w, 64, 4, 256)
    try:
        offs = [a.kv_alloc(i, 64) for i in range(3)]
        assert offs == [b.kv_alloc(i, 64) for i in range(3)]
        want, tok = [], None
        for it in range(steps):
            a.run_iteration(batch(it, offs, tok))
            out = torch.zeros(3, dtype=torch.int32, device="cuda")
            a.sample_last(u[it].data_ptr(), temperature=t.data_ptr(), top_p=p.data_ptr(), out_tokens=out.data_ptr())
            tok = out.tolist()
            want.append(tok)
        plans, got = [], torch.zeros((steps, 3), dtype=torch.int32, device="cuda")
        for it in range(steps):
            d = batch(it, offs, [-1, -2, -3])
            plans.append(np.zeros(b.plan_words(d), np.int32))
            b.plan_build(d, plans[it])
        dev = [torch.from_numpy(x).cuda() for x in plans]
        torch.cuda.synchronize()
        for it in range(steps):
            b.run_planned(plans[it], dev[it].data_ptr())
            b.sample_last(u[it].data_ptr(), temperature=t.data_ptr(), top_p=p.data_ptr(),
                          out_tokens=got[it].data_ptr(), sync=False)
        b.sync()
        assert got.tolist() == want
    finally:
        a.close()
        b.close()
