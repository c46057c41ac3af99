"""Timed cases of the operators that fill and read the cache around a resolve: appending rows (with the key norm and the
position rotation on the way) and the attention of a batch over a prefix that all of its requests share.

Each case is a dict of plain values. ``prepare`` makes a case's inputs on the GPU from a seed, ``run`` makes one pass:
through the library where ``own`` is true, else in elementary torch operations with 32-bit arithmetic (64-bit for the
angles of far positions). ``exact`` computes the same outputs in 64 bits, written separately.
"""
import math

import torch

own = False

LATENT, ROPE, HEADS = 512, 64, 128
WIDTH = LATENT + ROPE
SCALE = 1.0 / math.sqrt(192.0)  # the query-key head dimension of the unabsorbed heads, 128 + 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROW_BYTES = {"bf16": 1152, "fp8": 656}


def listed():
    return [
        # one token of one request, the smallest decode step: latency only; its queries rotate in the same call
        dict(name="append_decode_1", op="append", tokens=1, requests=1, start=4095, row="bf16", type="bf16", heads=128,
             norm=True, interleaved=True, page=64, to="pages", padded=0),
        # a decode step of 32 requests, two of the batch's entries padding
        dict(name="append_decode_32", op="append", tokens=32, requests=32, start=8000, row="bf16", type="bf16",
             heads=128, norm=True, interleaved=True, page=64, to="pages", padded=2),
        # a decode step of 8 requests whose 656-byte rows go straight to the host history
        dict(name="append_history_8", op="append", tokens=8, requests=8, start=700, row="fp8", type="bf16", heads=0,
             norm=True, interleaved=True, page=0, to="history", padded=0),
        # a prefill chunk over three requests with its queries, ragged, fp32 projections, half-split rotation
        dict(name="append_chunk_2047", op="append", tokens=2047, requests=3, start=129, row="bf16", type="f32",
             heads=128, norm=False, interleaved=False, page=16, to="pages", padded=5),
        # a long prompt's keys into fp8 rows (queries are rotated elsewhere during prefill)
        dict(name="append_prompt_131071", op="append", tokens=131071, requests=1, start=0, row="fp8", type="bf16",
             heads=0, norm=True, interleaved=True, page=64, to="pages", padded=0),
        # a short system prompt under one request
        dict(name="prefix_1x257", op="prefix", batch=1, length=257, page=16, holes=0.0, device_length=False, join=False),
        # a few requests over a prompt of a few thousand tokens, joined with each request's own rows
        dict(name="prefix_8x4096", op="prefix", batch=8, length=4096, page=64, holes=0.0, device_length=False,
             join=True),
        # one request over a long document: the rows' bytes bound it
        dict(name="prefix_1x131072", op="prefix", batch=1, length=131072, page=64, holes=0.0, device_length=False,
             join=False),
        # rows listed one by one, as a resident map lists them, some of them gone
        dict(name="prefix_5x8191_rows", op="prefix", batch=5, length=8191, page=1, holes=0.1, device_length=False,
             join=True),
        # a large batch over a medium prefix whose length is read on the device (a replayed graph)
        dict(name="prefix_100x2047", op="prefix", batch=100, length=2047, page=32, holes=0.0, device_length=True,
             join=True),
        # the whole decode batch over a long shared document: the tensor cores bound it
        dict(name="prefix_32x65537", op="prefix", batch=32, length=65537, page=64, holes=0.02, device_length=False,
             join=True),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.5:
        row = rng.choice(("bf16", "fp8"))
        to = rng.choice(("pages", "pages", "history"))
        tokens = _spread(rng, 1, 255 if to == "history" else 65535)
        heads = rng.choice((0, 16, 128)) if tokens <= 2048 else 0
        return dict(op="append", tokens=tokens, requests=_spread(rng, 1, min(tokens, 8)), start=rng.randrange(0, 512 if to == "history" else 8192),
                    row=row, type=rng.choice(("bf16", "f16", "f32")), heads=heads, norm=rng.random() < 0.6,
                    interleaved=rng.random() < 0.5, page=rng.choice((1, 16, 32, 64)) if to == "pages" else 0, to=to,
                    padded=rng.randrange(0, tokens) // 4)
    batch = _spread(rng, 1, 128)
    length = _spread(rng, 1, min(131072, 32 * 65536 // batch))
    return dict(op="prefix", batch=batch, length=length, page=rng.choice((1, 8, 16, 32, 64, 128)),
                holes=rng.choice((0.0, 0.0, 0.05)), device_length=rng.random() < 0.4, join=rng.random() < 0.6)


def _tokens_of(case, g):
    """Host plan of an append: per token its request and position (-1: padding), and the pages of each request."""
    n, reqs, start = case["tokens"], case["requests"], case["start"]
    dead = torch.zeros(n, dtype=torch.bool)
    if case["padded"]:
        dead[torch.randperm(n, generator=g)[: case["padded"]]] = True
    cut = [0] + sorted((torch.randperm(n - 1, generator=g)[: reqs - 1] + 1).tolist()) + [n]
    req = torch.repeat_interleave(torch.arange(reqs), torch.tensor([b - a for a, b in zip(cut, cut[1:])]))
    first = torch.tensor(cut[:-1])[req]
    pos = start + req + (torch.arange(n) - first)
    ctx = start + reqs + n
    return req.int(), torch.where(dead, -1, pos).int(), ctx, [b - a for a, b in zip(cut, cut[1:])]


def _append_state(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    t, n, dev = TYPES[case["type"]], case["tokens"], "cuda"
    req, pos, ctx, runs = _tokens_of(case, g)
    rb = ROW_BYTES[case["row"]]
    s = dict(case=case, n=n, ctx=ctx, rb=rb, runs=runs)
    # the projections' outputs: latents of a varied scale, some of them large, then the rotary key
    s["kv"] = (torch.randn(n, WIDTH, generator=gd, device=dev) * torch.exp(torch.randn(n, 1, generator=gd, device=dev))).to(t)
    s["weight"] = 1 + 0.2 * torch.randn(LATENT, generator=gd, device=dev) if case["norm"] else None
    s["inv_freq"] = 10000.0 ** (-torch.arange(0, ROPE, 2, device=dev, dtype=torch.float32) / ROPE)
    s["req"], s["pos"] = req.to(dev), pos.to(dev)
    s["live"] = torch.nonzero(pos >= 0).flatten().to(dev)
    s["q_rope"] = s["q"] = None
    if case["heads"]:
        s["q_rope"] = torch.randn(n, case["heads"], ROPE, generator=gd, device=dev).to(t)
        s["q"] = torch.randn(n, case["heads"], WIDTH, generator=gd, device=dev, dtype=torch.bfloat16)
    if case["to"] == "pages":
        # pages wholly before the first new token have left the pool; a few pages belong to somebody else
        page, per = case["page"], -(-ctx // case["page"])
        need = torch.zeros(case["requests"], per, dtype=torch.bool)
        alive = pos >= 0
        need[req.long()[alive], torch.div(pos.long(), page, rounding_mode="floor")[alive]] = True
        count = n // page + 2 * case["requests"]
        table = torch.full((case["requests"], per), -1, dtype=torch.int32)
        table[need] = torch.randperm(count + 3, generator=g)[:int(need.sum())].int()
        s["pages"], s["page"] = table.to(dev), page
        s["rows"] = torch.randint(0, 64, ((count + 3) * page, rb), generator=gd, device=dev, dtype=torch.uint8)
    else:
        s["host"] = torch.zeros(case["requests"], ctx, rb, dtype=torch.uint8, pin_memory=True)
        # (token index, request, position, how many) of each run of the batch without padding between
        p, spans = pos.tolist(), []
        for i in range(n):
            if p[i] < 0:
                continue
            if spans and spans[-1][0] + spans[-1][3] == i and spans[-1][1] == int(req[i]):
                spans[-1][3] += 1
            else:
                spans.append([i, int(req[i]), p[i], 1])
        s["spans"] = spans
    if own:
        _append_plan(s)
    return s


def _library():
    import hierarchical_sparse_attention_hs_gb300 as hs

    return hs


def _pool_of(hs, s, requests, ctx, rb, host=None):
    """A pool of one layer; without a host history its rows come from a device copy."""
    s["hot"] = torch.zeros(requests * 16 * rb, dtype=torch.uint8, device="cuda")
    src = None if host is not None else torch.empty(requests * ctx * rb, dtype=torch.uint8, device="cuda")
    d = hs.hs_pool_desc(1, requests, ctx, 16, 16, rb, None if host is None else host.data_ptr(), 0, 0,
                        s["hot"].data_ptr(), None, None if src is None else src.data_ptr())
    s["meta"] = torch.empty(hs.hs_meta_bytes(d), dtype=torch.uint8, device="cuda")
    d.meta = s["meta"].data_ptr()
    s["src"] = src
    s["hs"], s["pool"] = hs, hs.hs_pool_create(d)


def _append_plan(s):
    hs, c = _library(), s["case"]
    _pool_of(hs, s, c["requests"], s["ctx"], s["rb"], s.get("host"))
    s["desc"] = hs.append_desc(s["kv"], s["inv_freq"], s["pos"], req_ids=s["req"], norm_weight=s["weight"], norm_eps=1e-6,
                               interleaved=c["interleaved"], q_rope=s["q_rope"], q=s["q"])
    s["paged"] = hs.paged_rows(s["rows"], s["pages"], s["page"]) if c["to"] == "pages" else None


def _prefix_state(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    dev, batch, length, page = "cuda", case["batch"], case["length"], case["page"]
    room = length + (2 * page + 37 if case["device_length"] else 0)  # the list may be longer than today's prefix
    npages = -(-room // page)
    table = torch.randperm(npages + 5, generator=g)[:npages].int()
    if case["holes"]:
        table[torch.rand(npages, generator=g) < case["holes"]] = -1
    s = dict(case=case, page=page, length=length, room=npages * page if case["device_length"] else length)
    s["pages"] = table.to(dev)
    s["rows"] = torch.randn((npages + 5) * page, WIDTH, generator=gd, device=dev, dtype=torch.bfloat16)
    s["q"] = torch.randn(batch, HEADS, WIDTH, generator=gd, device=dev, dtype=torch.bfloat16)
    s["length_d"] = torch.tensor([length], dtype=torch.int32, device=dev) if case["device_length"] else None
    s["own_out"] = s["own_lse"] = None
    if case["join"]:  # what each request's attention over its own selected rows left (2048 rows: lse near 9)
        s["own_out"] = 0.05 * torch.randn(batch, HEADS, LATENT, generator=gd, device=dev)
        s["own_lse"] = 9 + torch.randn(batch, HEADS, generator=gd, device=dev)
    s["out"] = torch.empty(batch, HEADS, LATENT, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.empty(batch, HEADS, device=dev)
    if own:
        hs = _library()
        _pool_of(hs, s, 1, 16, 1152)
        s["paged"] = hs.paged_rows(s["rows"], s["pages"], page)
        n = hs.hs_mla_prefix_workspace(s["pool"], batch, s["room"])
        s["work"] = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    return s


def prepare(case, seed):
    return _append_state(case, seed) if case["op"] == "append" else _prefix_state(case, seed)


def _rotated(x, cos, sin, interleaved):
    """x [..., 64] in 32 bits, cos and sin [..., 32]."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _append_outputs(s):
    """What an append leaves, as views of the caller's buffers."""
    buf = s["rows"] if s["case"]["to"] == "pages" else s["host"]
    if s["case"]["row"] == "bf16":
        got = [buf.view(torch.bfloat16)]
    else:
        got = [buf[..., :LATENT].view(torch.float8_e4m3fn), buf[..., LATENT:LATENT + 16].view(torch.float32),
               buf[..., LATENT + 16:].view(torch.bfloat16)]
    return got + ([s["q"]] if s["q"] is not None else [])


def _run_append(s):
    c = s["case"]
    if own:
        s["hs"].hs_append(s["pool"], 0, s["n"], s["desc"], s["paged"], c["to"] == "history")
        return _append_outputs(s)
    x = s["kv"].float()
    z = x[:, :LATENT]
    if c["norm"]:
        z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * s["weight"]
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    k = _rotated(x[:, LATENT:], cos, sin, c["interleaved"])
    if c["row"] == "bf16":
        row = torch.cat((z, k), -1).to(torch.bfloat16).view(torch.uint8)
    else:
        z = z.view(-1, 4, 128)
        amax = z.abs().amax(-1, keepdim=True)
        scale = torch.where(amax > 0, amax / 448.0, 1.0)
        e = (z * (1.0 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1, LATENT)
        row = torch.cat((e.view(torch.uint8), scale.view(-1, 4).view(torch.uint8), k.to(torch.bfloat16).view(torch.uint8)), -1)
    live = s["live"]
    if c["to"] == "pages":
        pos, page = s["pos"][live].long(), s["page"]
        at = s["pages"][s["req"][live].long(), pos // page].long() * page + pos % page
        s["rows"][at] = row[live]
    else:  # one asynchronous copy for each run of tokens, as a program without the operator does it
        for i, r, p, m in s["spans"]:
            s["host"][r, p:p + m].copy_(row[i:i + m], non_blocking=True)
    if s["q"] is not None:
        qr = _rotated(s["q_rope"].float(), cos[:, None], sin[:, None], c["interleaved"])
        s["q"][live, :, LATENT:] = qr[live].to(torch.bfloat16)
    return _append_outputs(s)


def _run_prefix(s):
    c = s["case"]
    if own:
        hs = s["hs"]
        hs.hs_mla_prefix(s["pool"], c["batch"], s["q"], s["paged"], s["room"], s["length_d"], SCALE, s["own_out"],
                         s["own_lse"], s["out"], hs.HS_TYPE_BF16, s["lse"], s["work"])
        return [s["out"], s["lse"]]
    t = torch.arange(s["room"], device="cuda")
    page = s["pages"][t // s["page"]].long()
    valid = page >= 0
    if s["length_d"] is not None:
        valid &= t < s["length_d"]
    rows = torch.where(valid[:, None], s["rows"][page.clamp(min=0) * s["page"] + t % s["page"]], 0).float()
    score = torch.matmul(s["q"].view(-1, WIDTH).float(), rows.t())
    score.mul_(SCALE).masked_fill_(~valid, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows[:, :LATENT]) / total.clamp(min=1e-30)
    lse = (top + total.log()).view(c["batch"], HEADS)
    out = out.view(c["batch"], HEADS, LATENT)
    if c["join"]:
        m = torch.maximum(lse, s["own_lse"])
        a, b = (lse - m).exp()[..., None], (s["own_lse"] - m).exp()[..., None]
        out = (a * out + b * s["own_out"]) / (a + b)
        lse = m + (a + b).log()[..., 0]
    return [out.to(torch.bfloat16), lse]


def run(state):
    return _run_append(state) if state["case"]["op"] == "append" else _run_prefix(state)


def work(case):
    if case["op"] == "append":
        n, size = case["tokens"] - case["padded"], {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
        b = n * (WIDTH * size + ROW_BYTES[case["row"]] + 8) + n * case["heads"] * ROPE * (size + 2)
        b += 4 * LATENT if case["norm"] else 0
        f = n * ((5 * LATENT if case["norm"] else LATENT) + 6 * 32 * (1 + case["heads"]))
        return {"bytes": b, "flops": f}
    batch, n = case["batch"], case["length"] * (1 - case["holes"])
    b = n * 1152 + batch * HEADS * (WIDTH * 2 + LATENT * 2 + 4) + (batch * HEADS * (LATENT + 1) * 4 if case["join"] else 0)
    return {"bytes": b, "flops": 2.0 * batch * HEADS * n * (WIDTH + LATENT)}


def _exact_append(case, seed):
    s = _append_state(case, seed)
    d = torch.float64
    x = s["kv"].to(d)
    z, k = x[:, :LATENT], x[:, LATENT:]
    if case["norm"]:
        z = z * s["weight"].to(d) / (z.pow(2).sum(-1, keepdim=True) / LATENT + 1e-6).sqrt()
    turn = torch.polar(torch.ones((), dtype=d, device="cuda"), s["pos"].to(d)[:, None] * s["inv_freq"].to(d))

    def rotate(v, w):  # as complex numbers
        pair = v.unflatten(-1, (32, 2)) if case["interleaved"] else torch.stack((v[..., :32], v[..., 32:]), -1)
        r = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * w)
        return r.flatten(-2) if case["interleaved"] else torch.cat((r[..., 0], r[..., 1]), -1)

    live, k = s["live"], rotate(k, turn)
    req, pos = s["req"][live].long(), s["pos"][live].long()
    if case["row"] == "bf16":
        parts = [torch.cat((z, k), -1)]
    else:
        amax = z.view(-1, 4, 128).abs().amax(-1)
        scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        parts = [z / scale.repeat_interleave(128, -1), scale, k]
    got = []
    for before, new in zip(_append_outputs(s), parts):
        was = before.to(device="cuda", dtype=d)
        if case["to"] == "pages":
            was[s["pages"][req, pos // case["page"]].long() * case["page"] + pos % case["page"]] = new[live]
        else:
            was[req, pos] = new[live]
        got.append(was)
    if s["q"] is not None:
        q = s["q"].to(d)
        q[live, :, LATENT:] = rotate(s["q_rope"].to(d), turn[:, None])[live]
        got.append(q)
    return got


def _exact_prefix(case, seed):
    s = _prefix_state(case, seed)
    d = torch.float64
    at = torch.arange(case["length"])
    page = s["pages"].cpu().long()[at // case["page"]]
    at = (page * case["page"] + at % case["page"])[page >= 0].cuda()
    rows, outs, lses = s["rows"][at].to(d), [], []
    for b in range(case["batch"]):
        e = SCALE * torch.einsum("hd,td->ht", s["q"][b].to(d), rows)
        lse = torch.logsumexp(e, -1)
        out = torch.einsum("ht,tv->hv", (e - lse[:, None]).exp(), rows[:, :LATENT]) if len(at) else \
            torch.zeros(HEADS, LATENT, dtype=d, device="cuda")
        if case["join"]:
            both = torch.logaddexp(lse, s["own_lse"][b].to(d))
            out = (lse - both).exp()[:, None] * out + (s["own_lse"][b].to(d) - both).exp()[:, None] * s["own_out"][b].to(d)
            lse = both
        outs.append(out)
        lses.append(lse)
    return [torch.stack(outs), torch.stack(lses)]


def exact(case, seed):
    return _exact_append(case, seed) if case["op"] == "append" else _exact_prefix(case, seed)
