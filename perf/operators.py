"""Workloads of the 4-bit K/V cache (write and read back, attention) and of token sampling.

Each case is one call that a serving program makes.  ``run`` computes it with
elementary torch operations, or, where ``own`` is true, through the engine's
operator entry points on the same buffers.

A 4-bit layer (``layer``: one uint8 buffer, S = slots rounded up to 16, G = groups
of 32 components, at least one) holds, in this order

    K codes   [heads][S][head_dim / 2]   component 2b in the low, 2b + 1 in the high bits of byte b
    V codes   [heads][S / 2][head_dim / 4] 32-bit words: four components of the even slot in the
              low half, of the odd slot in the high half, four bits each
    K params  [heads][S][G]              bf16 scale (low half), bf16 minimum (high half)
    V params  [heads][S / 2][G][2]       the same, the pair's even slot first

and a component stands for minimum + scale * code.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # one request's increment at a small width: the smallest write, where latency counts
        dict(name="cache-one-token", op="cache", dtype="bf16", heads=20, head_dim=64, requests=1, rows=1, ctx=300),
        # the increments of a full decode batch at the 13B width
        dict(name="cache-decode-batch", op="cache", dtype="bf16", heads=40, head_dim=128, requests=64, rows=1, ctx=1000),
        # ragged prompts at the 13B width, as an initiation iteration writes them
        dict(name="cache-prompts", op="cache", dtype="bf16", heads=40, head_dim=128, requests=8, rows=2047, ctx=0),
        # an fp32 model's chunk of odd length behind a cached context
        dict(name="cache-fp32-chunk", op="cache", dtype="fp32", heads=12, head_dim=32, requests=5, rows=333, ctx=77),
        # one request's increment over a short context
        dict(name="attn-one-token", op="attn", dtype="bf16", heads=20, head_dim=64, requests=1, rows=1, ctx=300),
        # a decode batch of the 13B continuous-batching traffic: ragged contexts
        dict(name="attn-decode-batch", op="attn", dtype="bf16", heads=40, head_dim=128, requests=64, rows=1, ctx=4000),
        # few requests far into long contexts: the keys have to be split
        dict(name="attn-decode-long", op="attn", dtype="bf16", heads=32, head_dim=128, requests=3, rows=1, ctx=100001),
        # a few rows per request behind cached contexts (the ends of chunked prompts)
        dict(name="attn-few-rows", op="attn", dtype="bf16", heads=32, head_dim=128, requests=9, rows=7, ctx=1500),
        # ragged prompt chunks over cached contexts
        dict(name="attn-prompt-chunks", op="attn", dtype="bf16", heads=40, head_dim=128, requests=4, rows=1024, ctx=1000),
        # an fp32 model's decode batch
        dict(name="attn-fp32-decode", op="attn", dtype="fp32", heads=12, head_dim=64, requests=17, rows=1, ctx=900),
        # one request's next token, the usual filters on
        dict(name="sample-one-row", op="sample", dtype="fp32", rows=1, vocab=50257, kind="usual"),
        # a large batch, every row with parameters of its own
        dict(name="sample-batch", op="sample", dtype="fp32", rows=192, vocab=50257, kind="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "attn", "attn", "sample"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "sample":
        vocab = _log(rng, 500, 131072)
        return dict(op=op, dtype=dtype, rows=min(_log(rng, 1, 192), max(1, 9_000_000 // vocab)), vocab=vocab,
                    kind=rng.choice(["usual", "mixed", "top_p", "plain"]))
    heads, head_dim = _log(rng, 1, 40), rng.choice([16, 32, 64, 128, 128])
    if op == "cache":
        rows = 1 if rng.random() < 0.4 else _log(rng, 2, 1500)
        return dict(op=op, dtype=dtype, heads=heads, head_dim=head_dim, requests=_log(rng, 1, 64 if rows == 1 else 8),
                    rows=rows, ctx=rng.choice([0, _log(rng, 1, 2000)]) if rows > 1 else _log(rng, 1, 2000))
    form = rng.choice(["decode", "decode", "long", "few", "chunk"])
    if form == "decode":
        return dict(op=op, dtype=dtype, heads=heads, head_dim=head_dim, requests=_log(rng, 1, 64), rows=1,
                    ctx=_log(rng, 1, 4000))
    if form == "long":
        return dict(op=op, dtype=dtype, heads=heads, head_dim=head_dim, requests=rng.randint(1, 3), rows=1,
                    ctx=_log(rng, 4000, 100000))
    if form == "few":
        return dict(op=op, dtype=dtype, heads=heads, head_dim=head_dim, requests=_log(rng, 1, 9),
                    rows=rng.randint(2, 24), ctx=_log(rng, 1, 1500))
    # chunks of prompts: an fp32 model's are kept shorter (it has no tensor cores to run on)
    return dict(op=op, dtype=dtype, heads=heads, head_dim=head_dim, requests=rng.randint(1, 4),
                rows=_log(rng, 25, 1024 if dtype == "bf16" else 200), ctx=rng.choice([0, _log(rng, 1, 1000)]))


def _batch(case):
    """(n_input, ctx_len, kv_offset, slots) of a case's requests: ragged, in gaps, one of them at an odd slot."""
    n, c, off, at = [], [], [], 1
    for i in range(case["requests"]):
        f = 1.0 if i == 0 else 0.25 + 0.75 * ((i * 37 % 64) / 64.0)
        n.append(max(1, round(case["rows"] * f)) if case["rows"] > 1 else 1)
        c.append(round(case["ctx"] * (f if i % 2 else 1.25 - f)) if i else case["ctx"])
        off.append(at)
        at += c[-1] + n[-1] + i % 3
    return n, c, off, at + 2


# --------------------------------------------------------------------------- #
# the 4-bit layer in elementary operations
# --------------------------------------------------------------------------- #
def _views(layer, heads, head_dim, slots):
    """(K codes, V codes as bytes [h, S/2, d/4, slot of the pair, 2], K params, V params as bf16 [..., 2])."""
    S, G = (slots + 15) // 16 * 16, max(1, head_dim // 32)
    codes, params = heads * S * head_dim // 2, heads * S * G * 4
    kc = layer[:codes].view(heads, S, head_dim // 2)
    vc = layer[codes:2 * codes].view(heads, S // 2, head_dim // 4, 2, 2)
    kp = layer[2 * codes:2 * codes + params].view(torch.bfloat16).view(heads, S, G, 2)
    vp = layer[2 * codes + params:].view(torch.bfloat16).view(heads, S // 2, G, 2, 2)
    return kc, vc, kp, vp


def _layer_bytes(heads, head_dim, slots):
    S, G = (slots + 15) // 16 * 16, max(1, head_dim // 32)
    return heads * S * (head_dim + 8 * G)


def _quantise(x):
    """x [..., d] fp32 -> codes [..., d] uint8, scale and minimum [..., G] bf16."""
    d = x.shape[-1]
    g = x.unflatten(-1, (max(1, d // 32), min(32, d)))
    lo, hi = g.amin(-1), g.amax(-1)
    fifteen = torch.full((), 15.0, device=x.device)
    scale, low = ((hi - lo) / fifteen).bfloat16(), lo.bfloat16()
    s, m = scale.double()[..., None], low.double()[..., None]
    at = torch.where(s > 0, (g.double() - m) / torch.where(s > 0, s, 1.0), 0.0)  # in 64 bits: values next to a border
    return torch.round(at).clamp(0, 15).to(torch.uint8).flatten(-2), scale, low


def _nibbles(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _write(layer, heads, head_dim, slots, slot, k, v):
    """k, v [rows, heads, head_dim] fp32 into slots `slot` [rows]."""
    kc, vc, kp, vp = _views(layer, heads, head_dim, slots)
    c, s, m = _quantise(k)
    kc[:, slot] = _nibbles(c).transpose(0, 1)
    kp[:, slot] = torch.stack([s, m], -1).transpose(0, 1)
    c, s, m = _quantise(v)
    vc[:, slot // 2, :, slot % 2] = _nibbles(c).unflatten(-1, (head_dim // 4, 2))
    vp[:, slot // 2, :, slot % 2] = torch.stack([s, m], -1)


def _unpack(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _read(layer, heads, head_dim, slots, slot):
    """The values that slots `slot` [n] hold: k, v [heads, n, head_dim] fp32."""
    kc, vc, kp, vp = _views(layer, heads, head_dim, slots)
    width = min(32, head_dim)

    def values(codes, p):
        g = codes.float().unflatten(-1, (head_dim // width, width))
        return (g * p[..., 0, None].float() + p[..., 1, None].float()).flatten(-2)

    k = values(_unpack(kc[:, slot]), kp[:, slot])
    v = values(_unpack(vc[:, slot // 2, :, slot % 2].flatten(-2)).transpose(0, 1),
               vp[:, slot // 2, :, slot % 2].transpose(0, 1))
    return k, v


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _like_kv(shape, g):
    """K/V rows: normal, with a few channels several times larger than the others."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., 3::29] *= 4.0
    return x


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "sample":
        return _prepare_sample(case, g)
    heads, d, dtype = case["heads"], case["head_dim"], DTYPES[case["dtype"]]
    n, c, off, slots = _batch(case)
    H, rows = heads * d, sum(n)
    qkv = _like_kv((rows, 3, heads, d), g)
    qkv[:, 0] = torch.randn((rows, heads, d), generator=g, device="cuda")
    layer = torch.zeros(_layer_bytes(heads, d, slots), dtype=torch.uint8, device="cuda")
    at = torch.cat([torch.arange(b, b + x + y) for x, y, b in zip(n, c, off)]).cuda()
    st = dict(case=case, n=n, c=c, off=off, slots=slots, layer=layer, qkv=qkv.reshape(rows, 3 * H).to(dtype))
    if case["op"] == "attn":
        for part in at.split(max(1, (1 << 24) // H)):  # the cache as earlier iterations have written it
            x = _like_kv((part.numel(), 2, heads, d), g).to(dtype).float()
            _write(layer, heads, d, slots, part, x[:, 0], x[:, 1])
        st["out"] = torch.empty((rows, H), dtype=dtype, device="cuda")
        # per row: its request and its last key; per request and key: the slot (clamped to the request's own)
        st["req"] = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n)).cuda()
        st["row"] = torch.cat([torch.arange(x) for x in n]).cuda()
        keys = torch.tensor([x + y for x, y in zip(n, c)]).cuda()
        st["keys"], st["ctx"] = keys, torch.tensor(c).cuda()
        pos = torch.arange(int(keys.max()), device="cuda")
        st["slot_of"] = torch.tensor(off).cuda()[:, None] + torch.minimum(pos[None], keys[:, None] - 1)
    else:
        st["slot"] = torch.cat([torch.arange(b + y, b + x + y) for x, y, b in zip(n, c, off)]).cuda()
        st["out"] = torch.empty((2, heads, rows, d), dtype=dtype, device="cuda")
    if own:
        from iteration_level_scheduling_gb300 import native
        eng = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None,
                            torch.cuda.current_stream().cuda_stream)
        dt = native.DTYPE_BF16 if case["dtype"] == "bf16" else native.DTYPE_FP32
        plan = eng.kv4_plan(dt, heads, d, slots, n, c, off)
        st.update(eng=eng, plan=plan, dev_plan=torch.from_numpy(plan).cuda())
        if case["op"] == "attn":
            st["work"] = torch.empty(max(16, eng.kv4_workspace_bytes(plan)), dtype=torch.uint8, device="cuda")
        else:  # the rows just written, as ranges of their own
            back = eng.kv4_plan(dt, heads, d, slots, n, [0] * len(n), [b + y for b, y in zip(off, c)])
            st.update(back=back, dev_back=torch.from_numpy(back).cuda())
    return st


def _prepare_sample(case, g):
    rows, vocab, dtype = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    ld = (vocab + 7) // 8 * 8  # the row stride of a padded logits matrix
    logits = torch.full((rows, ld), 9e9, device="cuda")
    x = torch.randn((rows, vocab), generator=g, device="cuda") * 2.0 - 4.0
    tail = -torch.log(torch.rand((rows, vocab), generator=g, device="cuda").clamp_min(1e-12))
    x += tail * (tail > 4) * 0.9  # some tokens stand out, as a trained model's do
    x = torch.where(torch.rand((rows, vocab), generator=g, device="cuda") < 0.02, torch.tensor(-math.inf).cuda(), x)
    logits[:, :vocab] = x
    u = torch.rand(rows, generator=g, device="cuda")
    r = torch.rand((4, rows), generator=g, device="cuda")
    t, k, p, m = torch.ones(rows, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda"), \
        torch.ones(rows, device="cuda"), torch.zeros(rows, device="cuda")
    if case["kind"] == "usual":
        t, k, p = t * 0.8, k + 50, p * 0.95
    elif case["kind"] == "top_p":
        p = p * 0.9
    elif case["kind"] == "mixed":  # greedy rows, rows without filters, small and large top-k, nuclei of every size
        t = torch.where(r[0] < 0.1, 0.0, 0.5 + r[0])
        k = torch.where(r[1] < 0.4, 0, torch.exp(r[1] * 8.0)).to(torch.int32)
        p = torch.where(r[2] < 0.4, 1.0, 0.3 + 0.69 * r[2])
        m = torch.where(r[3] < 0.6, 0.0, 0.1 * r[3])
    st = dict(case=case, logits=logits.to(dtype), ld=ld, vocab=vocab, t=t, k=k, p=p, m=m, u=u,
              out=torch.empty(rows, dtype=torch.int32, device="cuda"))
    if own:
        from iteration_level_scheduling_gb300 import native
        st["eng"] = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None,
                                  torch.cuda.current_stream().cuda_stream)
        st["dt"] = native.DTYPE_BF16 if case["dtype"] == "bf16" else native.DTYPE_FP32
    return st


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def run(st):
    op = st["case"]["op"]
    if op == "cache":
        return {"kv": _run_cache(st)}
    if op == "attn":
        return {"out": _run_attn(st)}
    return {"token": _run_sample(st)}


def _run_cache(st):
    """Write the rows' keys and values, read the written slots back: [K|V][heads][rows][head_dim]."""
    if own:
        st["eng"].op_kv4_append(st["qkv"].data_ptr(), st["layer"].data_ptr(), st["plan"], st["dev_plan"].data_ptr(),
                                sync=False)
        st["eng"].op_kv4_read(st["layer"].data_ptr(), st["back"], st["dev_back"].data_ptr(), st["out"].data_ptr(),
                              sync=False)
        return st["out"]
    heads, d = st["case"]["heads"], st["case"]["head_dim"]
    x = st["qkv"].float().unflatten(-1, (3, heads, d))
    _write(st["layer"], heads, d, st["slots"], st["slot"], x[:, 1], x[:, 2])
    return torch.stack(_read(st["layer"], heads, d, st["slots"], st["slot"])).to(st["qkv"].dtype)


def _run_attn(st):
    """Row j of request i sees the keys 0 .. ctx + j of its request: softmax(q k / sqrt(d)) v per head."""
    if own:
        st["eng"].op_kv4_attention(st["qkv"].data_ptr(), st["layer"].data_ptr(), st["plan"], st["dev_plan"].data_ptr(),
                                   st["work"].data_ptr(), st["out"].data_ptr(), sync=False)
        return st["out"]
    heads, d = st["case"]["heads"], st["case"]["head_dim"]
    B, T = st["slot_of"].shape
    k, v = (x.unflatten(1, (B, T)).transpose(0, 1) for x in _read(st["layer"], heads, d, st["slots"],
                                                                  st["slot_of"].reshape(-1)))
    q = torch.zeros((B, max(st["n"]), heads, d), device="cuda")
    q[st["req"], st["row"]] = st["qkv"][:, :heads * d].float().unflatten(-1, (heads, d))
    s = torch.matmul(q.transpose(1, 2), k.transpose(-1, -2)) / math.sqrt(d)
    last = st["ctx"][:, None] + torch.arange(max(st["n"]), device="cuda")
    s = s.masked_fill(torch.arange(T, device="cuda") > last[:, None, :, None], -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True))
    out = torch.matmul(s, v) / s.sum(-1, keepdim=True)
    return out.transpose(1, 2)[st["req"], st["row"]].flatten(-2).to(st["qkv"].dtype)


def _run_sample(st):
    """Temperature, top-k, top-p of what top-k left, min-p relative to the largest probability; then the first token
    whose cumulative probability, in the order of the ids, exceeds u.  Temperature 0: the largest logit."""
    if own:
        st["eng"].op_sample(st["dt"], st["logits"].data_ptr(), st["case"]["rows"], st["vocab"], st["out"].data_ptr(),
                            st["u"].data_ptr(), temperature=st["t"].data_ptr(), top_k=st["k"].data_ptr(),
                            top_p=st["p"].data_ptr(), min_p=st["m"].data_ptr(), ld=st["ld"], sync=False)
        return st["out"]
    x = st["logits"][:, :st["vocab"]].double()
    t = st["t"].double()[:, None]
    x, order = torch.sort(x, dim=-1, descending=True, stable=True)  # ties: the lowest id first
    w = torch.exp((x - x[:, :1]) / torch.where(t > 0, t, 1.0))  # in 64 bits: sums that are compared with a border
    k = torch.where((st["k"] <= 0) | (t[:, 0] == 0), st["vocab"], st["k"])
    k = torch.where(t[:, 0] == 0, 1, k)
    w = w * (torch.arange(st["vocab"], device="cuda") < k[:, None])
    before = torch.cumsum(w, -1) - w
    p = st["p"].double()[:, None]
    keep = ((before < p * w.sum(-1, keepdim=True)) | (p >= 1)) & (w >= st["m"].double()[:, None])
    keep[:, 0] = True
    w = torch.zeros_like(w).scatter_(1, order, w * keep)
    c = torch.cumsum(w, -1)
    hit = (c > st["u"].double()[:, None] * c[:, -1:]) & (w > 0)
    return hit.to(torch.uint8).argmax(-1).to(torch.int32)


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        return {"bytes": case["rows"] * (case["vocab"] * es + 24), "flops": 4 * case["rows"] * case["vocab"]}
    heads, d = case["heads"], case["head_dim"]
    n, c, _, _ = _batch(case)
    H, held = heads * d, 2 * heads * (d // 2 + 4 * max(1, d // 32))  # bytes of one slot, K and V
    if case["op"] == "cache":
        return {"bytes": sum(n) * (2 * H * es + 2 * held + 2 * H * es), "flops": sum(n) * 2 * H * 8}
    pairs = sum(x * y + x * (x + 1) // 2 for x, y in zip(n, c))
    return {"bytes": sum(x + y for x, y in zip(n, c)) * held + 2 * sum(n) * H * es, "flops": 4 * pairs * H}


# --------------------------------------------------------------------------- #
# the definitions in 64 bits, request by request and row by row
# --------------------------------------------------------------------------- #
def _held(layer, heads, d, slots, first, count):
    """What slots first .. first + count - 1 hold, from the bytes: k, v [heads, count, d] in 64 bits."""
    S, G = (slots + 15) // 16 * 16, max(1, d // 32)
    words = layer.view(torch.int32)
    kc, vc, kp, vp = words.split([heads * S * d // 8, heads * S * d // 8, heads * S * G, heads * S * G])
    comp = torch.arange(d, device=layer.device)
    odd = torch.arange(first, first + count, device=layer.device) % 2
    pairs = slice(first // 2, (first + count + 1) // 2)  # those that hold the slots: cut to them below

    def cut(x):
        return x.flatten(1, 2)[:, first % 2:first % 2 + count]

    kc = (kc.view(heads, S, d // 8)[:, first:first + count, comp // 8] >> (4 * (comp % 8)).int()) & 15
    vc = vc.view(heads, S // 2, d // 4)[:, pairs, comp // 4]
    vc = (cut(vc[:, :, None].expand(-1, -1, 2, -1)) >> (16 * odd[:, None] + 4 * (comp % 4)).int()) & 15
    kp = kp.view(heads, S, G)[:, first:first + count]
    vp = cut(vp.view(heads, S // 2, G, 2)[:, pairs].transpose(2, 3))

    def real(codes, p):
        scale, low = (p << 16).view(torch.float32).double(), (p & -65536).view(torch.float32).double()
        return low[..., comp // 32] + scale[..., comp // 32] * codes

    return real(kc, kp), real(vc, vp)


def _stands_for(x):
    """x [..., d] fp32 -> the values that its 4-bit form stands for, in 64 bits."""
    d = x.shape[-1]
    g = x.reshape(x.shape[:-1] + (max(1, d // 32), min(32, d)))

    def bf16(a):  # to the nearest, ties to even
        u = a.contiguous().view(torch.int32).long()
        u = (u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16
        return u.int().view(torch.float32).double()

    lo, hi = g.min(-1).values, g.max(-1).values
    scale, low = bf16((hi - lo) / torch.tensor([15.0], device=x.device))[..., None], bf16(lo)[..., None]
    code = ((g.double() - low) / scale).nan_to_num(0.0).round().clip(0, 15)
    return (low + scale * code).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "sample":
        return {"token": _exact_sample(st)}
    heads, d = case["heads"], case["head_dim"]
    H = heads * d
    if case["op"] == "cache":
        x = st["qkv"].float().reshape(-1, 3, heads, d)
        return {"kv": torch.stack([_stands_for(x[:, i].transpose(0, 1)) for i in (1, 2)])}
    q = st["qkv"][:, :H].double().unflatten(-1, (heads, d)).transpose(0, 1)
    rows = []
    at = 0
    for n, c, off in zip(st["n"], st["c"], st["off"]):
        k, v = _held(st["layer"], heads, d, st["slots"], off, n + c)
        s = q[:, at:at + n] @ k.transpose(1, 2) / math.sqrt(d)
        s += torch.triu(torch.full((n, n + c), -math.inf, dtype=torch.float64, device="cuda"), c + 1)
        rows.append((torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, H))
        at += n
    return {"out": torch.cat(rows)}


def _exact_sample(st):
    x = st["logits"][:, :st["vocab"]].double().cpu().numpy()
    t, k, p, m, u = (st[a].double().cpu().numpy() for a in ("t", "k", "p", "m", "u"))
    got = np.zeros(len(x), np.int32)
    for i, row in enumerate(x):
        if t[i] == 0:
            got[i] = int(np.argmax(row))
            continue
        w = np.exp((row - row.max()) / t[i])
        order = np.lexsort((np.arange(len(row)), -row))
        if k[i] > 0:
            order = order[:int(k[i])]
        if p[i] < 1:
            mass = np.cumsum(w[order])
            order = order[:int(np.searchsorted(mass, p[i] * mass[-1])) + 1]
        order = np.sort(order[w[order] >= m[i]])
        mass = np.cumsum(w[order])
        got[i] = order[min(int(np.searchsorted(mass, u[i] * mass[-1], side="right")), len(order) - 1)]
    return got
