"""Workloads of the paged K/V cache: append with the rotation of positions, and attention over the pages.

Each case is one call that a serving program makes.  ``run`` computes it with
elementary torch operations, or, where ``own`` is true, through the engine's
operator entry points on the same buffers.

A layer of the cache is [K|V][kv_heads][pages * page][head_dim], the layout of the
engine's pool; position t of request i is held in slot table[i][t // page] * page +
t % page.  Query head h reads the keys and values of head h // (heads // kv_heads).
A row of q, k and v side by side has (heads + 2 kv_heads) * head_dim components, a
row of queries heads * head_dim, and either may be padded to a longer stride.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def _append(name, dtype, heads, kv_heads, head_dim, page, requests, rows, ctx, rot, pairs="halves", pad=0):
    return dict(name=name, op="append", dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
                requests=requests, rows=rows, ctx=ctx, rot=rot, pairs=pairs, pad=pad)


def _attn(name, dtype, heads, kv_heads, head_dim, page, requests, rows, ctx, pad=0):
    return dict(name=name, op="attn", dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
                requests=requests, rows=rows, ctx=ctx, pad=pad)


def listed():
    return [
        # one request's increment at a small width: the smallest write, where latency counts
        _append("append-one-token", "bf16", 20, 20, 64, 16, 1, 1, 300, rot=64),
        # the increments of a full decode batch at the 13B width, keys and values shared by five query heads
        _append("append-decode-batch", "bf16", 40, 8, 128, 16, 64, 1, 500, rot=128),
        # ragged prompts at the 13B width, as an initiation iteration writes them
        _append("append-prompts", "bf16", 40, 8, 128, 64, 8, 2047, 0, rot=128),
        # an fp32 model's chunk of odd length: a part of each head rotated, neighbours paired, padded rows
        _append("append-fp32-chunk", "fp32", 12, 3, 64, 32, 5, 333, 77, rot=24, pairs="neighbours", pad=8),
        # one request's increment over a short context
        _attn("attn-one-token", "bf16", 20, 20, 64, 16, 1, 1, 300),
        # a decode batch of the 13B width with shared key/value heads: ragged contexts
        _attn("attn-decode-batch", "bf16", 40, 8, 128, 16, 64, 1, 4000),
        # the same where every query head has keys and values of its own
        _attn("attn-decode-heads", "bf16", 40, 40, 128, 32, 64, 1, 1000),
        # few requests far into long contexts: the keys have to be split
        _attn("attn-decode-long", "bf16", 32, 4, 128, 64, 3, 1, 100001),
        # an fp32 model's decode batch
        _attn("attn-fp32-decode", "fp32", 12, 4, 64, 16, 17, 1, 900, pad=8),
        # a few rows per request behind cached contexts (the ends of chunked prompts, drafts to be verified)
        _attn("attn-few-rows", "bf16", 32, 8, 128, 16, 9, 7, 1500),
        # ragged prompt chunks over cached contexts
        _attn("attn-prompt-chunks", "bf16", 40, 8, 128, 16, 4, 1024, 1000),
        # whole prompts of a narrow model, large pages
        _attn("attn-prompts", "bf16", 16, 2, 64, 128, 8, 2047, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    head_dim = rng.choice([16, 32, 64, 128, 128])
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, _log(rng, 1, 40)])
    kv_heads = _log(rng, 1, max(1, 40 // group))
    shape = dict(dtype=dtype, heads=group * kv_heads, kv_heads=kv_heads, head_dim=head_dim,
                 page=rng.choice([16, 16, 32, 48, 64, 128, 256]), pad=rng.choice([0, 0, 8, 64]))
    if op == "append":
        rows = 1 if rng.random() < 0.4 else _log(rng, 2, 1500)
        return dict(op=op, **shape, requests=_log(rng, 1, 64 if rows == 1 else 8), rows=rows,
                    ctx=rng.choice([0, _log(rng, 1, 2000)]) if rows > 1 else _log(rng, 1, 500),
                    rot=rng.choice([0, head_dim, head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)]),
                    pairs=rng.choice(["halves", "halves", "neighbours"]))
    form = rng.choice(["decode", "decode", "long", "few", "chunk"])
    if form == "decode":  # at most some 0.8 GB of keys and values
        ctx = _log(rng, 1, 4000)
        most = max(1, int(8e8 / (ctx * 2 * kv_heads * head_dim * (2 if dtype == "bf16" else 4))))
        return dict(op=op, **shape, requests=min(_log(rng, 1, 64), most), rows=1, ctx=ctx)
    if form == "long":
        ctx = _log(rng, 4000, 100000)
        most = max(1, int(6e8 / (ctx * 2 * kv_heads * head_dim * (2 if dtype == "bf16" else 4))))
        return dict(op=op, **shape, requests=min(rng.randint(1, 3), most),
                    rows=1, ctx=min(ctx, int(6e8 / (2 * kv_heads * head_dim * (2 if dtype == "bf16" else 4)))))
    if form == "few":
        return dict(op=op, **shape, requests=_log(rng, 1, 9), rows=rng.randint(2, 24), ctx=_log(rng, 1, 1500))
    # chunks of prompts: an fp32 model's are kept shorter
    return dict(op=op, **shape, requests=rng.randint(1, 4), rows=_log(rng, 25, 1024 if dtype == "bf16" else 200),
                ctx=rng.choice([0, _log(rng, 1, 1000)]))


def _batch(case):
    """(n_input, ctx_len) of a case's requests: ragged, the first of full length."""
    n, c = [], []
    for i in range(case["requests"]):
        f = 1.0 if i == 0 else 0.25 + 0.75 * ((i * 37 % 64) / 64.0)
        n.append(max(1, round(case["rows"] * f)) if case["rows"] > 1 else 1)
        c.append(round(case["ctx"] * (f if i % 2 else 1.25 - f)) if i else case["ctx"])
    return n, c


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _like_kv(shape, g):
    """K/V rows: normal, with a few channels several times larger than the others."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., 3::29] *= 4.0
    return x


def _padded(x, pad):
    """The rows of x with `pad` elements behind each."""
    return torch.nn.functional.pad(x, (0, pad), value=7.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    heads, kv_heads, d, page, dtype = (case[k] for k in ("heads", "kv_heads", "head_dim", "page", "dtype"))
    dtype = DTYPES[dtype]
    n, c = _batch(case)
    rows = sum(n)
    # pages as a pool hands them out after a while: in no order, a few of them free
    need = [(x + y + page - 1) // page for x, y in zip(n, c)]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.zeros((len(n), max(need)), dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    layer = torch.empty((2, kv_heads, n_pages * page, d), dtype=dtype, device="cuda")
    for part in layer.view(-1, d).split(1 << 22):  # free slots hold what earlier requests left in them
        part.copy_(_like_kv(part.shape, g))
    st = dict(case=case, n=n, c=c, table=table, n_pages=n_pages, layer=layer)
    # slot of every request's positions, clamped to its own last one
    keys = torch.tensor([x + y for x, y in zip(n, c)])
    pos = torch.minimum(torch.arange(int(keys.max()))[None], keys[:, None] - 1)
    slot = (torch.gather(table.long(), 1, pos // page) * page + pos % page).cuda()
    req = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n)).cuda()
    row = torch.cat([torch.arange(x) for x in n]).cuda()
    ctx = torch.tensor(c).cuda()
    st.update(keys=keys.cuda(), slot_of=slot, req=req, row=row, ctx=ctx)
    if case["op"] == "append":
        x = _like_kv((rows, heads + 2 * kv_heads, d), g)
        x[:, :heads] = torch.randn((rows, heads, d), generator=g, device="cuda")
        st["qkv"] = _padded(x.flatten(1), case["pad"]).to(dtype)
        st["q_out"] = _padded(torch.zeros((rows, heads * d), device="cuda"), case["pad"]).to(dtype)
        st["at"] = ctx[req] + row  # positions of the rows
        # the table that a model keeps: cosines, then sines, of every position and pair
        angle = torch.arange(int(keys.max()), dtype=torch.float64, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda") / max(1, case["rot"] // 2))
        st["rope"] = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float().contiguous()
    else:
        st["q"] = _padded(torch.randn((rows, heads * d), generator=g, device="cuda"), case["pad"]).to(dtype)
        st["out"] = _padded(torch.zeros((rows, heads * d), device="cuda"), case["pad"]).to(dtype)
    if own:
        from iteration_level_scheduling_gb300 import native
        eng = native.Engine(1, 64, 1, 64, 64, 64, native.DTYPE_BF16, 64, 64, 64, None,
                            torch.cuda.current_stream().cuda_stream)
        dt = native.DTYPE_BF16 if case["dtype"] == "bf16" else native.DTYPE_FP32
        plan = eng.paged_plan(dt, heads, kv_heads, d, page, n_pages, n, c, table.numpy())
        st.update(eng=eng, plan=plan, dev_plan=torch.from_numpy(plan).cuda(),
                  work=torch.empty(max(16, eng.paged_workspace_bytes(plan)), dtype=torch.uint8, device="cuda"))
    return st


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def run(st):
    return _run_append(st) if st["case"]["op"] == "append" else {"out": _run_attn(st)}


def _run_append(st):
    """Rotate the rows' queries and keys, write queries out and keys and values to their pages."""
    case = st["case"]
    heads, kv_heads, d, rot = case["heads"], case["kv_heads"], case["head_dim"], case["rot"]
    if own:
        st["eng"].op_paged_append(st["qkv"].data_ptr(), st["layer"].data_ptr(), st["plan"], st["dev_plan"].data_ptr(),
                                  q_out=st["q_out"].data_ptr(), rope=st["rope"].data_ptr() if rot else 0,
                                  rope_len=st["rope"].shape[0] if rot else 0, rot_dim=rot,
                                  neighbours=case["pairs"] == "neighbours", ld_qkv=st["qkv"].shape[1],
                                  ld_q=st["q_out"].shape[1], sync=False)
        return {"q": st["q_out"], "kv": st["layer"]}
    x = st["qkv"][:, :(heads + 2 * kv_heads) * d].float().unflatten(-1, (heads + 2 * kv_heads, d))
    qk, v = x[:, :heads + kv_heads], x[:, heads + kv_heads:]
    if rot:
        cos, sin = st["rope"][st["at"]][:, None].split(rot // 2, -1)
        if case["pairs"] == "halves":
            a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        qk = torch.cat([turned, qk[..., rot:]], -1)
    dtype, slot = st["layer"].dtype, st["slot_of"][st["req"], st["at"]]
    st["q_out"][:, :heads * d] = qk[:, :heads].flatten(1).to(dtype)
    st["layer"][0][:, slot] = qk[:, heads:].transpose(0, 1).to(dtype)
    st["layer"][1][:, slot] = v.transpose(0, 1).to(dtype)
    return {"q": st["q_out"], "kv": st["layer"]}


def _run_attn(st):
    """Row j of request i sees the keys 0 .. ctx + j of its request: softmax(q k / sqrt(d)) v per head."""
    case = st["case"]
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["head_dim"]
    if own:
        st["eng"].op_paged_attention(st["q"].data_ptr(), st["layer"].data_ptr(), st["plan"], st["dev_plan"].data_ptr(),
                                     st["work"].data_ptr(), st["out"].data_ptr(), ld_q=st["q"].shape[1],
                                     ld_out=st["out"].shape[1], sync=False)
        return st["out"]
    B, T = st["slot_of"].shape
    rows = max(st["n"])
    k, v = (x[:, st["slot_of"]].float().transpose(0, 1) for x in st["layer"])  # [B, kv_heads, T, d]
    q = torch.zeros((B, rows, heads, d), device="cuda")
    q[st["req"], st["row"]] = st["q"][:, :heads * d].float().unflatten(-1, (heads, d))
    q = q.unflatten(2, (kv_heads, heads // kv_heads)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, kv_heads, group * rows, d]
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    last = (st["ctx"][:, None] + torch.arange(rows, device="cuda")).repeat(1, heads // kv_heads)
    s = s.masked_fill(torch.arange(T, device="cuda") > last[:, None, :, None], -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(s, v) / s.sum(-1, keepdim=True)
    o = o.unflatten(2, (heads // kv_heads, rows)).permute(0, 3, 1, 2, 4)  # [B, rows, kv_heads, group, d]
    st["out"][:, :heads * d] = o[st["req"], st["row"]].flatten(1).to(st["out"].dtype)
    return st["out"]


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["head_dim"]
    n, c = _batch(case)
    if case["op"] == "append":
        width = (heads + 2 * kv_heads) * d
        return {"bytes": 2 * sum(n) * width * es + max(n) * case["rot"] * 4,
                "flops": 3 * sum(n) * (heads + kv_heads) * case["rot"]}
    pairs = sum(x * y + x * (x + 1) // 2 for x, y in zip(n, c))
    return {"bytes": sum(x + y for x, y in zip(n, c)) * 2 * kv_heads * d * es + 2 * sum(n) * heads * d * es,
            "flops": 4 * pairs * heads * d}


# --------------------------------------------------------------------------- #
# the definitions in 64 bits, request by request
# --------------------------------------------------------------------------- #
def _slots(st, i, first, count):
    """Slots of positions first .. first + count - 1 of request i."""
    page = st["case"]["page"]
    return torch.tensor([int(st["table"][i, t // page]) * page + t % page for t in range(first, first + count)],
                        device="cuda")


def exact(case, seed):
    st = prepare(case, seed)
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["head_dim"]
    group, H = heads // kv_heads, heads * d
    if case["op"] == "append":
        q_out, layer = st["q_out"].double(), st["layer"].double()
        at = 0
        for i, (n, c) in enumerate(zip(st["n"], st["c"])):
            x = st["qkv"][at:at + n].double()
            y, slots = x.clone(), _slots(st, i, c, n)
            for p in range(case["rot"] // 2):  # the pair (a, b) as a + b i, turned by the angle
                turn = torch.complex(*(st["rope"][c:c + n, p + z * (case["rot"] // 2)].double() for z in (0, 1)))
                ia, ib = (p, p + case["rot"] // 2) if case["pairs"] == "halves" else (2 * p, 2 * p + 1)
                cols = torch.arange(heads + kv_heads, device="cuda") * d
                z = torch.complex(x[:, cols + ia], x[:, cols + ib]) * turn[:, None]
                y[:, cols + ia], y[:, cols + ib] = z.real, z.imag
            q_out[at:at + n, :H] = y[:, :H]
            for h in range(kv_heads):
                layer[0, h, slots] = y[:, H + h * d:H + (h + 1) * d]
                layer[1, h, slots] = y[:, H + (kv_heads + h) * d:H + (kv_heads + h + 1) * d]
            at += n
        return {"q": q_out, "kv": layer}
    out = st["out"].double()
    at = 0
    for i, (n, c) in enumerate(zip(st["n"], st["c"])):
        slots = _slots(st, i, 0, n + c)
        hidden = torch.triu(torch.full((n, n + c), -math.inf, dtype=torch.float64, device="cuda"), c + 1)
        for h in range(kv_heads):
            k, v = st["layer"][0, h, slots].double(), st["layer"][1, h, slots].double()
            for j in range(h * group, (h + 1) * group):
                w = torch.softmax(st["q"][at:at + n, j * d:(j + 1) * d].double() @ k.T * d ** -0.5 + hidden, -1)
                out[at:at + n, j * d:(j + 1) * d] = w @ v
        at += n
    return {"out": out}
