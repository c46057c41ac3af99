"""Timed cases of the operators around a cache whose rows hold their latents in 4 bits: writing rows, reading rows back as
numbers, and the sparse decode attention over them.

A row of 416 bytes holds 512 latents as whole numbers from -7 to 7 in 4 bits each, 32 scales, one for each 16 latents
(8 bits: 5 of exponent, 3 of fraction, no sign, which are the upper bits of a half), and the rotary key's 64 bf16 values; a
latent is its number times its scale. The 32-bit word i holds latents 8 i to 8 i + 7, each plus 8: the even ones at bits 0,
4, 8, 12, the odd ones at bits 16, 20, 24, 28. Rows of 656 bytes (e4m3 latents, a 32-bit scale for each 128) are read back
as well.

Each case is a dict of plain values. ``prepare`` makes a case's inputs on the GPU from a seed, ``run`` makes one pass:
through the library where ``own`` is true, else in elementary torch operations with 32-bit arithmetic (64-bit for the
angles of far positions and for values next to a border between two codes). ``exact`` computes the same outputs in 64 bits, written
separately.
"""
import math

import torch

own = False

LATENT, ROPE, HEADS = 512, 64, 128
WIDTH = LATENT + ROPE
BLOCK = 16  # latents of one scale of a 4-bit row
SCALE = 1.0 / math.sqrt(192.0)  # the query-key head dimension of the unabsorbed heads, 128 + 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROW_BYTES = {"int4": 416, "fp8": 656}
SLOTS_MOST = 8192  # slots of a request's hot buffer that every pool takes


def listed():
    return [
        # a decode step of one request: its row and its queries, then the row as attention will see it; latency only
        dict(name="write_decode_1", op="write", tokens=1, requests=1, start=4095, type="bf16", heads=128, norm=True,
             interleaved=True, page=64, padded=0),
        # a decode step of 33 requests, two of the batch's entries padding, half-split rotation
        dict(name="write_decode_33", op="write", tokens=33, requests=33, start=8000, type="f16", heads=128, norm=True,
             interleaved=False, page=16, padded=2),
        # a long prompt's rows (normed by the projection's own epilogue), read back for the attention of its next chunk
        dict(name="write_prompt_131071", op="write", tokens=131071, requests=1, start=0, type="bf16", heads=0, norm=False,
             interleaved=True, page=64, padded=0),
        # the rows a few requests selected, for a consumer that takes bf16 rows: some in the hot buffer, some in the paged rows
        dict(name="read_tiered_3x257", op="read", row="int4", source="tiered", batch=3, k=257, slots=512, type="bf16",
             padded=0.05),
        # a decode batch's selections out of the hot buffer, fp8 rows, as 32-bit numbers
        dict(name="read_slots_32x2048_fp8", op="read", row="fp8", source="slots", batch=32, k=2048, slots=4096, type="f32",
             padded=0.0),
        # a whole long history in token order, for a prefill chunk that attends to all of it
        dict(name="read_history_131072", op="read", row="int4", source="history", batch=1, k=131072, slots=512,
             type="bf16", padded=0.0),
        # one request whose selection is short: the smallest call
        dict(name="decode_1x65", op="decode", source="slots", batch=1, k=65, slots=512, padded=0.0),
        # one request, the usual selection
        dict(name="decode_1x2048", op="decode", source="slots", batch=1, k=2048, slots=4096, padded=0.0),
        # a few requests, some of their rows still in the ordinary paged pool, some entries padding
        dict(name="decode_7x2047", op="decode", source="tiered", batch=7, k=2047, slots=4096, padded=0.1),
        # the decode batch of the sparse-attention workload
        dict(name="decode_32x2048", op="decode", source="slots", batch=32, k=2048, slots=4096, padded=0.0),
        # a large batch with an odd selection, straight from the full history
        dict(name="decode_100x1111", op="decode", source="history", batch=100, k=1111, slots=2048, padded=0.0),
        # few requests that select much: a long list over a large hot buffer
        dict(name="decode_5x16384", op="decode", source="slots", batch=5, k=16384, slots=20000, padded=0.0),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "decode"))
    if op == "write":
        # decode steps come with their norm and queries, prompts with latents that are normed already
        step = rng.random() < 0.5
        tokens = _spread(rng, 1, 64) if step else _spread(rng, 65, 65535)
        return dict(op="write", tokens=tokens, requests=_spread(rng, 1, min(tokens, 8)), start=rng.randrange(0, 8192),
                    type=rng.choice(("bf16", "f16", "f32") if step else ("bf16", "f16")),
                    heads=rng.choice((0, 16, 128)) if tokens <= 2048 else 0, norm=step,
                    interleaved=rng.random() < 0.5, page=rng.choice((1, 16, 32, 64)), padded=rng.randrange(0, tokens) // 4)
    source = rng.choice(("slots", "slots", "tiered", "history"))
    batch = _spread(rng, 1, 128)
    if op == "read":
        k = _spread(rng, 1, min(65535, 131072 // batch))
        return dict(op="read", row=rng.choice(("int4", "int4", "fp8")), source=source, batch=batch, k=k, slots=k + 1 + k // 3,
                    type=rng.choice(("bf16", "bf16", "f16", "f32")), padded=rng.choice((0.0, 0.0, 0.1)))
    k = _spread(rng, 1, min(16384, 98304 // batch))
    return dict(op="decode", source=source, batch=batch, k=k, slots=k + 1 + k // 3, padded=rng.choice((0.0, 0.0, 0.1)))


# ---- the 4-bit format, in 64 bits

def _scale_of(z):
    """The scale of each 16 latents [...][32]: their largest magnitude / 7, to 4 significant bits, within its range."""
    a = z.double().unflatten(-1, (-1, BLOCK)).abs().amax(-1) / torch.full((), 7.0, dtype=torch.float64, device=z.device)
    step = torch.exp2(torch.frexp(a).exponent.clamp(min=-13).double() - 4)
    return (torch.round(a / step) * step).clamp(2.0 ** -17, 3840.0)


def _pack(z, key):
    """Rows of 416 bytes from latents [n][512] and rotary keys [n][64]."""
    scale = _scale_of(z)
    code = (torch.round(z.double() / scale.repeat_interleave(BLOCK, -1)).clamp(-7, 7) + 8).byte().unflatten(-1, (-1, 8))
    pair = code[..., [0, 4, 1, 5]] | code[..., [2, 6, 3, 7]] << 4
    return torch.cat((pair.flatten(-2), (scale.half().view(torch.int16) >> 7).byte(), key.to(torch.bfloat16).view(torch.uint8)), -1)


def _values(rows):
    """What rows [...][416 or 656] stand for, in 32 bits [...][576]."""
    if rows.shape[-1] == 416:
        pair = rows[..., :LATENT // 2].unflatten(-1, (-1, 4))
        code = torch.cat((pair & 15, pair >> 4), -1)[..., [0, 2, 4, 6, 1, 3, 5, 7]]  # they are latents 0 4 1 5 2 6 3 7
        scale = (rows[..., LATENT // 2:LATENT // 2 + 32].short() << 7).view(torch.float16).float()
        z = (code.flatten(-2).float() - 8) * scale.repeat_interleave(BLOCK, -1)
    else:
        scale = rows[..., LATENT:LATENT + 16].contiguous().view(torch.float32)
        z = rows[..., :LATENT].contiguous().view(torch.float8_e4m3fn).float() * scale.repeat_interleave(128, -1)
    return torch.cat((z, rows[..., -2 * ROPE:].contiguous().view(torch.bfloat16).float()), -1)


def _random_rows(n, kind, gd):
    """Rows as a model leaves them: latents of unit size with a few large channels."""
    out = torch.empty(n, ROW_BYTES[kind], dtype=torch.uint8, device="cuda")
    channel = torch.exp(0.4 * torch.randn(LATENT, generator=gd, device="cuda"))
    for i in range(0, n, 32768):
        m = min(32768, n - i)
        z = torch.randn(m, LATENT, generator=gd, device="cuda") * channel
        key = torch.randn(m, ROPE, generator=gd, device="cuda")
        if kind == "int4":
            out[i:i + m] = _pack(z, key)
        else:
            scale = z.view(m, 4, 128).abs().amax(-1) / 448
            e = (z.view(m, 4, 128) / scale[..., None]).to(torch.float8_e4m3fn).view(m, LATENT)
            out[i:i + m] = torch.cat((e.view(torch.uint8), scale.view(torch.uint8),
                                      key.to(torch.bfloat16).view(torch.uint8)), -1)
    return out


# ---- states

def _library():
    import hierarchical_sparse_attention_hs_gb300 as hs

    return hs


def _pool(s, requests, ctx, slots, row_bytes, hot, history=None):
    """A pool of one layer over these hot rows; its history is a device copy."""
    hs = _library()
    d = hs.hs_pool_desc(1, requests, ctx, slots, min(slots, 2048), row_bytes, None, 0, 0, hot.data_ptr(), None, None)
    s["source"] = history if history is not None else torch.empty(requests * ctx * row_bytes, dtype=torch.uint8, device="cuda")
    d.noio_src = s["source"].data_ptr()
    s["meta"] = torch.empty(hs.hs_meta_bytes(d), dtype=torch.uint8, device="cuda")
    d.meta = s["meta"].data_ptr()
    s["hs"], s["pool"] = hs, hs.hs_pool_create(d)


def _write_state(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    t, n, reqs, page, dev = TYPES[case["type"]], case["tokens"], case["requests"], case["page"], "cuda"
    dead = torch.zeros(n, dtype=torch.bool)
    if case["padded"]:
        dead[torch.randperm(n, generator=g)[: case["padded"]]] = True
    cut = [0] + sorted((torch.randperm(n - 1, generator=g)[: reqs - 1] + 1).tolist()) + [n]
    req = torch.repeat_interleave(torch.arange(reqs), torch.tensor([b - a for a, b in zip(cut, cut[1:])]))
    pos = torch.where(dead, -1, case["start"] + req + torch.arange(n) - torch.tensor(cut[:-1])[req])
    ctx = case["start"] + reqs + n
    # pages wholly before the first new token have left the pool; a few pages belong to somebody else
    alive, per = pos >= 0, -(-ctx // page)
    need = torch.zeros(reqs, per, dtype=torch.bool)
    need[req[alive], torch.div(pos[alive], page, rounding_mode="floor")] = True
    count = n // page + 2 * reqs + 3
    table = torch.full((reqs, per), -1, dtype=torch.int32)
    table[need] = torch.randperm(count, generator=g)[:int(need.sum())].int()
    row = torch.full((n,), -1, dtype=torch.int64)
    row[alive] = table[req[alive], torch.div(pos[alive], page, rounding_mode="floor")].long() * page + pos[alive] % page
    s = dict(case=case, n=n, req=req.int().to(dev), pos=pos.int().to(dev), pages=table.to(dev), page=page)
    s["live"] = torch.nonzero(alive).flatten().to(dev)
    s["at"] = row[alive].to(dev)
    # the list through which the rows are read back, as a resolve names rows of the paged pool
    s["entries"] = torch.where(row >= 0, -2 - row, -1).int().to(dev)
    s["rows"] = torch.zeros(count * page, ROW_BYTES["int4"], dtype=torch.uint8, device=dev)
    # the projections' outputs: latents of a varied scale where a norm follows, else of a normed size; the rotary key
    size = torch.exp(torch.randn(n, 1, generator=gd, device=dev)) if case["norm"] else 1.0
    s["kv"] = (torch.randn(n, WIDTH, generator=gd, device=dev) * size).to(t)
    s["weight"] = 1 + 0.2 * torch.randn(LATENT, generator=gd, device=dev) if case["norm"] else None
    s["inv_freq"] = 10000.0 ** (-torch.arange(0, ROPE, 2, device=dev, dtype=torch.float32) / ROPE)
    s["q_rope"] = s["q"] = None
    if case["heads"]:
        s["q_rope"] = torch.randn(n, case["heads"], ROPE, generator=gd, device=dev).to(t)
        s["q"] = torch.randn(n, case["heads"], WIDTH, generator=gd, device=dev, dtype=torch.bfloat16)
    s["values"] = torch.empty(n, WIDTH, dtype=torch.bfloat16, device=dev)
    if own:
        s["hot"] = torch.zeros(reqs * 16 * ROW_BYTES["int4"], dtype=torch.uint8, device=dev)
        _pool(s, reqs, ctx, 16, ROW_BYTES["int4"], s["hot"])
        hs = s["hs"]
        s["desc"] = hs.append_desc(s["kv"], s["inv_freq"], s["pos"], req_ids=s["req"], norm_weight=s["weight"], norm_eps=1e-6,
                                   interleaved=case["interleaved"], q_rope=s["q_rope"], q=s["q"])
        s["paged"] = hs.paged_rows(s["rows"], s["pages"], page)
    return s


def _list_state(case, seed):
    """A hot buffer or a history, paged rows beside it, and every request's list of entries."""
    gd = torch.Generator(device="cuda").manual_seed(seed)
    batch, k, slots, dev = case["batch"], case["k"], case["slots"], "cuda"
    kind = case.get("row", "int4")
    history = case["source"] == "history"
    s = dict(case=case, ctx=slots if not history else max(slots, k + 5))
    per = s["ctx"] if history else slots
    s["rows"] = _random_rows(batch * per, kind, gd).view(batch, per, -1)
    if history and batch == 1 and k > 65536:
        e = torch.arange(k, device=dev).view(1, k)  # a whole history is read in order
    else:
        e = torch.rand(batch, per, generator=gd, device=dev).argsort(-1)[:, :k]
    s["resident"] = None
    if case["source"] == "tiered":
        s["resident"] = _random_rows(max(64, batch * k // 4), kind, gd)
        there = torch.rand(batch, k, generator=gd, device=dev) < 0.25
        e = torch.where(there, -2 - torch.randint(0, s["resident"].shape[0], (batch, k), generator=gd, device=dev), e)
    if case["padded"]:
        e = torch.where(torch.rand(batch, k, generator=gd, device=dev) < case["padded"], -1, e)
        if batch > 2 and case["op"] == "decode":
            e[1] = -1  # a request with nothing selected
    s["entries"] = e.int().contiguous()
    if case["op"] == "read":
        s["out"] = torch.empty(batch, k, WIDTH, dtype=TYPES[case["type"]], device=dev)
    else:
        s["q"] = torch.randn(batch, HEADS, WIDTH, generator=gd, device=dev, dtype=torch.bfloat16)
        s["out"] = torch.empty(batch, HEADS, LATENT, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(batch, HEADS, device=dev)
    if own:
        s["list"], s["paged"] = s["entries"], s["resident"]
        s["by_token"] = history
        if not history and slots > SLOTS_MOST:
            # more rows than a hot buffer has slots: the history's, or, beside rows of the paged pool, all in that pool
            s["by_token"] = s["resident"] is None
            if not s["by_token"]:
                first = slots * torch.arange(batch, device=dev)[:, None]
                s["list"] = torch.where(e >= 0, -2 - (e + first), torch.where(e <= -2, e - batch * slots, e)).int()
                s["paged"] = torch.cat((s["rows"].flatten(0, 1), s["resident"]))
        if s["by_token"] or slots > SLOTS_MOST:
            s["hot"] = torch.zeros(batch * 16 * ROW_BYTES[kind], dtype=torch.uint8, device=dev)
            _pool(s, batch, per, 16, ROW_BYTES[kind], s["hot"], s["rows"])
        else:
            _pool(s, batch, 64, slots, ROW_BYTES[kind], s["rows"])
    return s


def prepare(case, seed):
    return _write_state(case, seed) if case["op"] == "write" else _list_state(case, seed)


# ---- one pass

def _rotated(x, cos, sin, interleaved):
    """x [..., 64], cos and sin [..., 32]."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _run_write(s):
    c = s["case"]
    got = [s["values"]] + ([s["q"]] if s["q"] is not None else [])
    if own:
        hs = s["hs"]
        hs.hs_append(s["pool"], 0, s["n"], s["desc"], s["paged"], False)
        hs.hs_gather_values(s["pool"], 0, 1, s["entries"], s["n"], s["rows"], s["rows"].shape[0], s["values"], hs.HS_TYPE_BF16)
        return got
    live = s["live"]
    z = s["kv"][:, :LATENT].double()
    if c["norm"]:
        z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * s["weight"].double()
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    key = _rotated(s["kv"][:, LATENT:].float(), cos, sin, c["interleaved"])
    s["rows"][s["at"]] = _pack(z, key)[live]
    s["values"].zero_()
    s["values"][live] = _values(s["rows"][s["at"]]).to(torch.bfloat16)
    if s["q"] is not None:
        qr = _rotated(s["q_rope"].float(), cos[:, None], sin[:, None], c["interleaved"])
        s["q"][live, :, LATENT:] = qr[live].to(torch.bfloat16)
    return got


def _selected(s):
    """The values of the listed rows in 32 bits [batch][k][576], zeros for padding, and which entries are rows."""
    e = s["entries"].long()
    rows = s["rows"]
    raw = torch.gather(rows, 1, e.clamp(min=0)[..., None].expand(-1, -1, rows.shape[-1]))
    valid = e >= 0
    if s["resident"] is not None:
        raw = torch.where((e <= -2)[..., None], s["resident"][(-2 - e).clamp(min=0)], raw)
        valid = valid | (e <= -2)
    return torch.where(valid[..., None], _values(raw), 0.0), valid


def _run_read(s):
    c = s["case"]
    if own:
        hs = s["hs"]
        out_type = {"bf16": hs.HS_TYPE_BF16, "f16": hs.HS_TYPE_F16, "f32": hs.HS_TYPE_F32}[c["type"]]
        if s["by_token"]:
            hs.hs_gather_values_history(s["pool"], 0, c["batch"], s["list"], c["k"], s["out"], out_type)
        else:
            r = s["paged"]
            hs.hs_gather_values(s["pool"], 0, c["batch"], s["list"], c["k"], r, 0 if r is None else r.shape[0], s["out"],
                                out_type)
        return [s["out"]]
    return [_selected(s)[0].to(s["out"].dtype)]


def _run_decode(s):
    c = s["case"]
    if own:
        hs = s["hs"]
        if s["by_token"]:
            hs.hs_mla_decode_int4_history(s["pool"], 0, c["batch"], s["q"], s["list"], c["k"], SCALE, s["out"],
                                          hs.HS_TYPE_BF16, s["lse"])
        else:
            r = s["paged"]
            hs.hs_mla_decode_int4(s["pool"], 0, c["batch"], s["q"], s["list"], c["k"], r, 0 if r is None else r.shape[0],
                                  SCALE, s["out"], hs.HS_TYPE_BF16, s["lse"])
        return [s["out"], s["lse"]]
    rows, valid = _selected(s)
    score = torch.matmul(s["q"].float(), rows.transpose(1, 2))
    score.mul_(SCALE).masked_fill_(~valid[:, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows[..., :LATENT]) / total.clamp(min=1e-30)
    return [out.to(torch.bfloat16), (top + total.log())[..., 0]]


def run(state):
    return {"write": _run_write, "read": _run_read, "decode": _run_decode}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "write":
        n, size = case["tokens"] - case["padded"], {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
        # the projections in, the rows out, and their values
        b = n * (WIDTH * size + ROW_BYTES["int4"] + 12 + WIDTH * 2) + n * case["heads"] * ROPE * (size + 2)
        b += 4 * LATENT if case["norm"] else 0
        return {"bytes": b, "flops": n * ((7 if case["norm"] else 4) * LATENT + 6 * 32 * (1 + case["heads"]))}
    n = case["batch"] * case["k"] * (1 - case["padded"])
    if case["op"] == "read":
        size = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
        return {"bytes": n * ROW_BYTES[case["row"]] + case["batch"] * case["k"] * (4 + WIDTH * size), "flops": n * LATENT}
    b = n * ROW_BYTES["int4"] + case["batch"] * (4 * case["k"] + HEADS * (WIDTH * 2 + LATENT * 2 + 4))
    return {"bytes": b, "flops": 2.0 * HEADS * n * (WIDTH + LATENT)}


# ---- the same from the definitions, in 64 bits

def _exact_row(rows):
    """What 4-bit or fp8 rows stand for, in 64 bits, from the fields of their bits."""
    d = torch.float64
    b = rows.to(torch.int64)
    if rows.shape[-1] == 416:
        word = sum(b[..., i:256:4] << 8 * i for i in range(4))  # [...][64]
        z = torch.stack([(word >> at) % 16 for at in (0, 16, 4, 20, 8, 24, 12, 28)], -1).flatten(-2).to(d) - 8
        f = b[..., 256:288]
        ex, m = f // 8, (f % 8).to(d)
        scale = torch.where(ex == 0, m / 8 * 2.0 ** -14, (1 + m / 8) * torch.exp2(ex.to(d) - 15))
        z = (z.unflatten(-1, (32, 16)) * scale[..., None]).flatten(-2)
    else:
        scale = rows[..., 512:528].contiguous().view(torch.float32).to(d)
        z = (rows[..., :512].contiguous().view(torch.float8_e4m3fn).to(d).unflatten(-1, (4, 128)) * scale[..., None]).flatten(-2)
    return z, rows[..., -128:].contiguous().view(torch.bfloat16).to(d)


def _exact_write(case, seed):
    s = _write_state(case, seed)
    d = torch.float64
    x = s["kv"].to(d)
    z = x[:, :LATENT]
    if case["norm"]:
        z = z * s["weight"].to(d) / (z.pow(2).sum(-1, keepdim=True) / LATENT + 1e-6).sqrt()
    turn = torch.polar(torch.ones((), dtype=d, device="cuda"), s["pos"].to(d)[:, None] * s["inv_freq"].to(d))

    def rotate(v, w):  # as complex numbers
        pair = v.unflatten(-1, (32, 2)) if case["interleaved"] else torch.stack((v[..., :32], v[..., 32:]), -1)
        r = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * w)
        return r.flatten(-2) if case["interleaved"] else torch.cat((r[..., 0], r[..., 1]), -1)

    # every scale that the format has: the nearest is looked up
    f = torch.arange(1, 256, device="cuda")
    every = torch.where(f < 8, f / 8 * 2.0 ** -14, (1 + f % 8 / 8) * torch.exp2(f.to(d) // 8 - 15))
    every = every[every <= 3840]
    want = z.unflatten(-1, (32, 16)).abs().amax(-1) / 7
    hi = torch.searchsorted(every, want.contiguous()).clamp(1, len(every) - 1)
    lo, up = every[hi - 1], every[hi]
    odd = (hi + 1) % 2 == 1  # the code of `up` is hi + 1
    scale = torch.where((up - want < want - lo) | ((up - want == want - lo) & ~odd), up, lo)
    near = (z.unflatten(-1, (32, 16)) / scale[..., None]).round().clamp(-7, 7)
    values = torch.zeros(case["tokens"], WIDTH, dtype=d, device="cuda")
    live = s["live"]
    values[live] = torch.cat(((near * scale[..., None]).flatten(-2), rotate(x[:, LATENT:], turn)), -1)[live]
    got = [values]
    if s["q"] is not None:
        q = s["q"].to(d)
        q[live, :, LATENT:] = rotate(s["q_rope"].to(d), turn[:, None])[live]
        got.append(q)
    return got


def _exact_list(case, seed):
    s = _list_state(case, seed)
    d = torch.float64
    outs, lses = [], []
    for b in range(case["batch"]):
        e = s["entries"][b].long()
        hot, away = torch.nonzero(e >= 0).flatten(), torch.nonzero(e <= -2).flatten()
        raw = torch.zeros(case["k"], s["rows"].shape[-1], dtype=torch.uint8, device="cuda")
        raw[hot] = s["rows"][b][e[hot]]
        if len(away):
            raw[away] = s["resident"][-2 - e[away]]
        if case["op"] == "read":
            z, key = _exact_row(raw)
            row = torch.cat((z, key), -1)
            row[e == -1] = 0
            outs.append(row)
            continue
        z, key = _exact_row(raw[e != -1])
        q = s["q"][b].to(d)
        score = SCALE * (torch.einsum("hd,td->ht", q[:, :LATENT], z) + torch.einsum("hd,td->ht", q[:, LATENT:], key))
        lse = torch.logsumexp(score, -1) if len(z) else torch.full((HEADS,), -math.inf, dtype=d, device="cuda")
        outs.append(torch.einsum("ht,tv->hv", (score - lse[:, None]).exp(), z) if len(z) else
                    torch.zeros(HEADS, LATENT, dtype=d, device="cuda"))
        lses.append(lse)
    return [torch.stack(outs)] + ([torch.stack(lses)] if lses else [])


def exact(case, seed):
    return _exact_write(case, seed) if case["op"] == "write" else _exact_list(case, seed)
