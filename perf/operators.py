"""The operators between the packed linear layers, as cases to measure: the plan of a paged
cache from request lengths, the write into a cache held in 4 bits, attention over it, and the
norms around a block with its gate and residual scale.

``run`` computes each in its plain form (elementary torch operations in 32 bits) or, with
``own`` set, through the framework's entry points.  ``exact`` is the definition in 64 bits.

The cache (uint8 [pages, heads, page * dim * 9 / 8]) holds, for one page and key/value head,
the key codes, the value codes, the key parameters and the value parameters.  64 channels of
one token share a scale s and a minimum m (fp16): x = m + s c with a code c of 4 bits.

* key codes: token t, quarter c of 0..3, step s of 0..dim/32-1: one dword with channels
  32 s + 8 c + j in nibble j, dwords in the order [t][c][s];
* value codes: token t, column n of 0..15: dim/16 nibbles, channel 16 j + n in nibble j,
  words in the order [t / 4][n][t % 4];
* parameters: per token the scales of its groups, then their minima.
"""
import math

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # the first steps of one short chat on the 8B shape: all latency
        dict(name="attend-one-short", op="attend", b=1, rows=1, length=77, hq=32, hkv=8, dim=128, page=16,
             window=0, dtype="fp16"),
        # an ordinary decode batch, ragged lengths, 8B shape
        dict(name="attend-decode-32", op="attend", b=32, rows=1, length=4001, hq=32, hkv=8, dim=128, page=64,
             window=0, dtype="fp16"),
        # one request with a very long context, 70B shape: few rows, the long axis has to be split
        dict(name="attend-decode-long", op="attend", b=1, rows=1, length=131071, hq=64, hkv=8, dim=128, page=64,
             window=0, dtype="bf16"),
        # a full decode batch, 70B shape: the largest read of the cache
        dict(name="attend-decode-wide", op="attend", b=128, rows=1, length=8192, hq=64, hkv=8, dim=128, page=64,
             window=0, dtype="bf16"),
        # a few drafted tokens per request checked at once, small heads, a sliding window
        dict(name="attend-draft-window", op="attend", b=8, rows=5, length=2003, hq=16, hkv=4, dim=64, page=32,
             window=1024, dtype="bf16"),
        # chunks of two prompts over what is cached of them, 8B shape: bound by the products
        dict(name="attend-prompt", op="attend", b=2, rows=1024, length=4096, hq=32, hkv=8, dim=128, page=64,
             window=0, dtype="fp16"),
        # the new keys and values of a decode batch, padded to a captured size, and read back
        dict(name="append-decode", op="append", tokens=48, pad=16, hkv=8, dim=128, page=64, dtype="fp16"),
        # those of a long prompt
        dict(name="append-prompt", op="append", tokens=8191, pad=0, hkv=8, dim=128, page=64, dtype="bf16"),
        # slots and pages of a decode step, some requests ended
        dict(name="plan-decode", op="plan", b=256, length=4000, prompt=0, page=16, width=512),
        # slots and pages of a step that mixes prompts with decoding requests
        dict(name="plan-prompts", op="plan", b=1000, length=2000, prompt=4096, page=16, width=512),
        # a decode step's post norm, gate, residual and next norm, 16-bit output
        dict(name="norm-decode", op="norm", m=4, n=4096, post=True, gate="channel", alpha=1.0, beta=0.5,
             dtype="fp16", res="same", out="16"),
        # a prompt's, residual in 32 bits, quantized to int8 for the next packed layer
        dict(name="norm-prompt-int8", op="norm", m=2047, n=8192, post=True, gate="channel", alpha=1.0, beta=0.22,
             dtype="fp16", res="fp32", out="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "plan", "norm", "norm"])
    dtype = rng.choice(["fp16", "bf16"])
    page = rng.choice([16, 32, 64, 128])
    if op == "attend":
        hq, hkv, dim = rng.choice([(32, 8, 128), (64, 8, 128), (16, 4, 64), (8, 8, 128), (24, 2, 128), (16, 2, 256)])
        kind = rng.choice(["decode", "decode", "prompt"])
        if kind == "decode":
            rows = rng.choice([1, 1, 1, 2, 7])
            length = max(rows, _log(rng, 1, 100000))
            b = max(1, min(128, _log(rng, 1, 128), 600000 // length))
        else:
            rows = _log(rng, 9, 1500)
            length = rows + _log(rng, 1, 4000)
            b = max(1, min(4, _log(rng, 1, 4), 2500 // rows))
        window = rng.choice([0, 0, 0, max(1, length // 3)])
        return dict(op=op, b=b, rows=rows, length=length, hq=hq, hkv=hkv, dim=dim, page=page, window=window,
                    dtype=dtype)
    if op == "append":
        hkv, dim = rng.choice([(8, 128), (4, 64), (2, 256), (1, 128)])
        return dict(op=op, tokens=_log(rng, 1, 8000), pad=rng.choice([0, 0, 5, 32]), hkv=hkv, dim=dim, page=page,
                    dtype=dtype)
    if op == "plan":
        return dict(op=op, b=_log(rng, 1, 1500), length=_log(rng, 1, 4000), prompt=rng.choice([0, 0, _log(rng, 10, 3000)]),
                    page=page, width=512)
    out = rng.choice(["16", "16", "int8"])
    n = 128 * _log(rng, 1, 100) if out == "int8" else _log(rng, 64, 12000)
    return dict(op=op, m=_log(rng, 1, 3000), n=n, post=rng.random() < 0.7,
                gate=rng.choice(["none", "channel", "token"]), alpha=rng.choice([1.0, 1.41]),
                beta=rng.choice([1.0, 0.22]), dtype=dtype, res=rng.choice(["same", "fp32"]), out=out)


def _lengths(case):
    """Tokens cached and rows asked for, per request: ragged, from the case alone."""
    b, r, top = case["b"], case["rows"], case["length"]
    rows = [max(1, r - (i % 3) * (r // 5)) for i in range(b)]
    lens = [max(rows[i], top - (i * 37) % (top // 2 + 1)) for i in range(b)]
    return lens, rows


def _requests(case):
    """(tokens held, tokens added) of each request of a plan; -1 added: the request ended."""
    b, top, cap = case["b"], case["length"], case["width"] * case["page"]
    held = [min(cap // 2, (top * (1 + (i * 29) % 64)) // 64) for i in range(b)]
    fresh = [-1 if i % 17 == 5 else 1 for i in range(b)]
    if case["prompt"]:
        for i in range(0, b, 50):
            held[i], fresh[i] = 0, min(cap, max(1, case["prompt"] - 13 * i % 97))
    return held, fresh


def work(case):
    op = case["op"]
    if op == "attend":
        lens, rows = _lengths(case)
        w, keys, read = case["window"], 0, 0
        for n, r in zip(lens, rows):
            first = n - r
            seen = [(p + 1 if not w else min(w, p + 1)) for p in range(first, n)]
            keys += sum(seen)
            read += n - (max(0, first - w + 1) if w else 0)
        t = sum(rows)
        return {"bytes": read * case["hkv"] * case["dim"] * 9 // 8 + t * case["hq"] * (4 * case["dim"] + 4),
                "flops": 4 * case["dim"] * case["hq"] * keys}
    if op == "append":
        t, c = case["tokens"], case["hkv"] * case["dim"]
        return {"bytes": t * c * (4 + 9 / 8 + 9 / 8 + 4) + 4 * (t + case["pad"]), "flops": 8 * t * c}
    if op == "plan":
        held, fresh = _requests(case)
        t = sum(max(f, 0) for f in fresh)
        p = case["page"]
        pages = sum(-(-h // p) if f < 0 else -(-(h + f) // p) - -(-h // p) for h, f in zip(held, fresh))
        return {"bytes": 20 * case["b"] + 8 * t + 8 * pages, "flops": 0}
    m, n = case["m"], case["n"]
    res = 4 if case["res"] == "fp32" else 2
    out = m * n * 2 if case["out"] == "16" else m * n + m * n // 128 * (4 + 4 + 32)
    gate = m * n * 2 if case["gate"] == "token" else n * 2 if case["gate"] == "channel" else 0
    return {"bytes": m * n * (2 + 2 * res) + out + gate + n * 2 * (2 if case["post"] else 1), "flops": 14 * m * n}


# ----------------------------------------------------------------------------- the inputs

def _keys_values(gen, t, h, d, dtype):
    """Keys with a few strong channels and an offset per channel, as after a projection; plain values."""
    dev = "cuda"
    k = torch.randn(t, h, d, generator=gen, device=dev)
    gain = torch.ones(h, d, device=dev)
    gain[:, torch.randint(0, d, (max(1, d // 48),), generator=gen, device=dev)] = 6.0
    k = k * gain + 0.5 * torch.randn(1, h, d, generator=gen, device=dev)
    v = torch.randn(t, h, d, generator=gen, device=dev) * 0.7
    return k.to(dtype), v.to(dtype)


def _codes(x):
    """(code, scale, minimum) of each group of 64 channels, every step in 32 bits."""
    x = x.float()
    x = torch.where(x.isnan(), torch.zeros_like(x), x).clamp(-65504.0, 65504.0)
    g = x.view(*x.shape[:-1], x.shape[-1] // 64, 64)
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    m = lo.half()
    s = ((hi - lo) / torch.full_like(lo, 15.0)).half()
    s = torch.where((s == 0) & (hi > lo), torch.full_like(s, 2.0 ** -24), s)
    sf = s.float()
    c = torch.round((g - m.float()) / torch.where(sf == 0, torch.ones_like(sf), sf)).clamp(0.0, 15.0)
    c = torch.where(sf == 0, torch.zeros_like(c), c)
    return c, s, m


def _store(cache, page, slots, k, v):
    """Writes tokens into the cache's documented layout."""
    pages, h, d = cache.shape[0], cache.shape[1], k.shape[2]
    pg, tok = torch.div(slots, page, rounding_mode="floor").long(), (slots % page).long()
    half, t, g = page * d // 2, k.shape[0], d // 64
    c, s, m = _codes(k)
    c = c.view(t, h, d // 32, 4, 4, 2).to(torch.uint8)
    by = (c[..., 0] | (c[..., 1] << 4)).permute(0, 1, 3, 2, 4).reshape(t, h, d // 2)
    cache[:, :, :half].view(pages, h, page, d // 2)[pg, :, tok] = by
    par = torch.cat([s.view(t, h, g), m.view(t, h, g)], -1)
    words = cache.view(torch.float16)
    words[:, :, half: half + page * 2 * g].view(pages, h, page, 2 * g)[pg, :, tok] = par
    c, s, m = _codes(v)
    c = c.view(t, h, d // 32, 2, 16).to(torch.uint8)
    by = (c[:, :, :, 0] | (c[:, :, :, 1] << 4)).transpose(2, 3)
    cache[:, :, half: 2 * half].view(pages, h, page // 4, 16, 4, d // 32)[pg, :, tok // 4, :, tok % 4, :] = by
    par = torch.cat([s.view(t, h, g), m.view(t, h, g)], -1)
    words[:, :, half + page * 2 * g:].view(pages, h, page, 2 * g)[pg, :, tok] = par


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    return {"attend": _prepare_attend, "append": _prepare_append, "plan": _prepare_plan,
            "norm": _prepare_norm}[case["op"]](case, gen)


def _prepare_attend(case, gen):
    lens, rows = _lengths(case)
    b, h, d, page, dt = case["b"], case["hkv"], case["dim"], case["page"], DT[case["dtype"]]
    held = [-(-n // page) for n in lens]
    width = max(held)
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    grid = torch.arange(width, device="cuda")[None] < torch.tensor(held, device="cuda")[:, None]
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    table[grid] = order[: sum(held)]
    # what no request has written yet is whatever the memory held
    cache = torch.full((pages, h, page * d * 9 // 8), 255, dtype=torch.uint8, device="cuda")
    total = sum(lens)
    ln = torch.tensor(lens, device="cuda")
    start = torch.cumsum(ln, 0) - ln
    for at in range(0, total, 65536):
        idx = torch.arange(at, min(total, at + 65536), device="cuda")
        seq = torch.searchsorted(start, idx, right=True) - 1
        pos = idx - start[seq]
        slots = table[seq, torch.div(pos, page, rounding_mode="floor")].long() * page + pos % page
        _store(cache, page, slots, *_keys_values(gen, idx.numel(), h, d, dt))
    t = sum(rows)
    cu = torch.tensor([0] + rows, device="cuda").cumsum(0).to(torch.int32)
    q = torch.randn(t, case["hq"], d, generator=gen, device="cuda").to(dt)
    return dict(op="attend", q=q, cache=cache, table=table, lens=ln.to(torch.int32), cu=cu, rows=max(rows),
                length=max(lens), page=page, window=case["window"], scale=1.0 / math.sqrt(d),
                out=torch.empty_like(q), lse=torch.empty(t, case["hq"], device="cuda"))


def _prepare_append(case, gen):
    t, pad, h, d, page = (case[x] for x in ("tokens", "pad", "hkv", "dim", "page"))
    dt = DT[case["dtype"]]
    pages = -(-t // page) + 5
    k, v = _keys_values(gen, t + pad, h, d, dt)
    # runs of consecutive tokens on pages in any order, as a plan hands them out
    order = torch.randperm(pages, generator=gen, device="cuda")
    i = torch.arange(t, device="cuda") + 3
    slots = torch.full((t + pad,), -1, dtype=torch.int32, device="cuda")
    slots[:t] = (order[torch.div(i, page, rounding_mode="floor")] * page + i % page).to(torch.int32)
    cache = torch.full((pages, h, page * d * 9 // 8), 255, dtype=torch.uint8, device="cuda")
    return dict(op="append", k=k, v=v, slots=slots, cache=cache, page=page, ko=torch.zeros_like(k),
                vo=torch.zeros_like(v))


def _prepare_plan(case, gen):
    held, fresh = _requests(case)
    b, page, width = case["b"], case["page"], case["width"]
    have = [-(-n // page) for n in held]
    more = sum(-(-(n + max(f, 0)) // page) - p for n, f, p in zip(held, fresh, have) if f >= 0)
    pages = sum(have) + more + 7
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    grid = torch.arange(width, device="cuda")[None] < torch.tensor(have, device="cuda")[:, None]
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    table[grid] = order[: sum(have)]
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    count = pages - sum(have)
    free[:count] = order[sum(have):]
    t = sum(max(f, 0) for f in fresh)
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(op="plan", fresh=torch.tensor(fresh, dtype=torch.int32, device="cuda"),
                lens=torch.tensor(held, dtype=torch.int32, device="cuda"), table=table, free=free,
                count=torch.tensor([count], dtype=torch.int32, device="cuda"), page=page, pages=pages,
                tokens=t + 8, lens_out=e(b), count_out=e(2), cu=e(b + 1), slots=e(t + 8), pos=e(t + 8))


def _prepare_norm(case, gen):
    m, n, dt = case["m"], case["n"], DT[case["dtype"]]
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    rt = torch.float32 if case["res"] == "fp32" else dt
    h = rand(m, n) * 2.0
    h[:, torch.randint(0, n, (max(1, n // 200),), generator=gen, device="cuda")] *= 12.0
    s = dict(op="norm", x=(rand(m, n) * 1.5).to(dt), h=h.to(rt), pre=(1 + 0.2 * rand(n)).to(dt),
             post=(1 + 0.2 * rand(n)).to(dt) if case["post"] else None, gate=None, alpha=case["alpha"],
             beta=case["beta"], eps=1e-5, out=case["out"], h_out=torch.empty(m, n, dtype=rt, device="cuda"))
    if case["gate"] != "none":
        s["gate"] = (rand(n) if case["gate"] == "channel" else rand(m, n)).to(dt)
    if case["out"] == "16":
        s["y"] = torch.empty(m, n, dtype=dt, device="cuda")
    else:
        g = n // 128
        s["aq"] = torch.empty(m, n, dtype=torch.int8, device="cuda")
        s["sa"] = torch.empty(g, m, device="cuda")
        s["asum"] = torch.empty(g, m, dtype=torch.int32, device="cuda")
        s["rowop"] = torch.empty(g, m, 8, dtype=torch.int32, device="cuda")
        s["y"] = torch.empty(m, g, 128, dtype=torch.float16, device="cuda")
    return s


# -------------------------------------------------------------------------------- a pass

def run(state):
    if own:
        return {"attend": _own_attend, "append": _own_append, "plan": _own_plan, "norm": _own_norm}[state["op"]](state)
    return {"attend": _plain_attend, "append": _plain_append, "plan": _plain_plan,
            "norm": _plain_norm}[state["op"]](state)


def _own_attend(s):
    from weight_activation_quantized_amd import mixllm as L
    if "ws" not in s:
        size = L.mixllm_kv4_attention_workspace_bytes(s["q"].shape[0], s["lens"].shape[0], s["q"].shape[1],
                                                      s["cache"].shape[1], s["q"].shape[2], s["rows"], s["length"],
                                                      s["window"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    L.mixllm_kv4_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu"], s["out"], s["page"], s["rows"],
                           s["length"], scale=s["scale"], window=s["window"], lse=s["lse"], workspace=s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_append(s):
    from weight_activation_quantized_amd import mixllm as L
    L.mixllm_kv4_append(s["k"], s["v"], s["slots"], s["cache"], s["page"])
    L.mixllm_kv4_read(s["cache"], s["slots"], s["ko"], s["vo"], s["page"])
    return {"k": s["ko"], "v": s["vo"]}


def _own_plan(s):
    from weight_activation_quantized_amd import mixllm as L
    L.mixllm_kv_plan(s["fresh"], s["lens"], s["table"], s["free"], s["count"], s["page"], s["pages"], s["lens_out"],
                     s["count_out"], s["cu"], s["slots"], s["pos"])
    return {x: s[x] for x in ("lens_out", "count_out", "cu", "slots", "pos", "table", "free")}


def _own_norm(s):
    from weight_activation_quantized_amd import mixllm as L
    if s["out"] == "16":
        L.mixllm_residual_norm(s["x"], s["h"], s["pre"], s["h_out"], y=s["y"], post_weight=s["post"], gate=s["gate"],
                               alpha=s["alpha"], beta=s["beta"], eps=s["eps"])
        return {"h": s["h_out"], "y": s["y"]}
    L.mixllm_residual_norm(s["x"], s["h"], s["pre"], s["h_out"], aq=s["aq"], sa=s["sa"], asum=s["asum"],
                           rowop=s["rowop"], post_weight=s["post"], gate=s["gate"], alpha=s["alpha"], beta=s["beta"],
                           eps=s["eps"])
    m, n = s["aq"].shape
    torch.mul(s["aq"].view(m, n // 128, 128), s["sa"].t().unsqueeze(2), out=s["y"])
    return {"h": s["h_out"], "y": s["y"]}


# The plain forms.

def _unpacked(cache, pages, page, d):
    """Keys and values [B, heads, tokens, dim] in 32 bits of the given pages [B, width]."""
    b, width = pages.shape
    h, g, half = cache.shape[1], d // 64, page * d // 2
    blk = cache[pages.reshape(-1).long().clamp(min=0)]
    par = blk[:, :, 2 * half:].contiguous().view(torch.float16).view(b * width, h, 2, page, 2, g).float()

    def values(codes, p):
        x = codes.view(b * width, h, page, g, 64).float() * p[:, :, :, 0, :, None] + p[:, :, :, 1, :, None]
        return x.view(b, width, h, page, d).transpose(1, 2).reshape(b, h, width * page, d)

    kb = blk[:, :, :half].reshape(b * width, h, page, 4, d // 32, 4).transpose(3, 4)
    k = values(torch.stack((kb & 15, kb >> 4), -1), par[:, :, 0])
    vb = blk[:, :, half: 2 * half].reshape(b * width, h, page // 4, 16, 4, d // 32).permute(0, 1, 2, 4, 5, 3)
    v = values(torch.stack((vb & 15, vb >> 4), -2).contiguous(), par[:, :, 1])
    return k, v


def _plain_attend(s):
    q, cu, lens, w = s["q"], s["cu"].long(), s["lens"].long(), s["window"]
    (t, hq, d), page, r = q.shape, s["page"], s["rows"]
    b, hkv = lens.shape[0], s["cache"].shape[1]
    k, v = _unpacked(s["cache"], s["table"][:, : -(-s["length"] // page)], page, d)
    n = k.shape[2]
    nq = cu[1:] - cu[:-1]
    i = torch.arange(r, device=q.device)
    qp = q.float()[(cu[:-1, None] + i).clamp(max=t - 1)]                       # [B, R, Hq, D]
    qp = qp.view(b, r, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, (hq // hkv) * r, d)
    at = torch.arange(n, device=q.device)
    known = at < lens[:, None]                                                 # [B, N]
    k = torch.where(known[:, None, :, None], k, torch.zeros_like(k))
    v = torch.where(known[:, None, :, None], v, torch.zeros_like(v))
    sc = torch.matmul(qp, k.transpose(2, 3).contiguous()).view(b, hq, r, n) * s["scale"]
    pos = (lens - nq)[:, None] + i                                             # [B, R]
    seen = known[:, None] & (at <= pos[..., None])
    if w:
        seen = seen & (at > pos[..., None] - w)
    sc = sc.masked_fill(~seen[:, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top.isinf(), torch.zeros_like(top), top))
    den = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hkv, -1, n), v).view(b, hq, r, d) / torch.where(den == 0, torch.ones_like(den), den)
    lse = (top + torch.log(den)).squeeze(-1)
    row = torch.arange(t, device=q.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    at = row - cu[seq]
    return {"out": o[seq, :, at].to(q.dtype), "lse": lse[seq, :, at]}


def _plain_append(s):
    live = (s["slots"] >= 0)[:, None, None]

    def back(x):
        c, sc, m = _codes(x)
        y = (m.float() + sc.float() * c).view(x.shape)
        return torch.where(live, y, torch.zeros_like(y)).to(x.dtype)

    return {"k": back(s["k"]), "v": back(s["v"])}


def _plain_plan(s):
    page, cap, dev = s["page"], s["tokens"], s["fresh"].device
    fresh, table, free = s["fresh"].long(), s["table"].clone(), s["free"].clone()
    width, pool = table.shape[1], free.shape[0]
    held = s["lens"].long().clamp(0, width * page)
    ended, add = fresh < 0, fresh.clamp(min=0)
    have = torch.div(held + page - 1, page, rounding_mode="floor")
    col = torch.arange(width, device=dev)
    # pages of ended requests go back on top of the free ones
    back = torch.where(ended, have, torch.zeros_like(have))
    first = torch.cumsum(back, 0) - back
    gone = ended[:, None] & (col < have[:, None])
    place = s["count"].long() + first[:, None] + col
    at = torch.where(gone & (place < pool), place, torch.full_like(place, pool))
    free = torch.cat([free, free[:1]]).scatter(0, at.reshape(-1), table.reshape(-1))[:pool]
    top = (s["count"].long() + back.sum()).clamp(max=pool)
    # new pages come from the top, request by request
    fits = held + add <= width * page
    need = torch.div(held + add + page - 1, page, rounding_mode="floor") - have
    need = torch.where(ended | ~fits, torch.zeros_like(need), need)
    before = torch.cumsum(need, 0) - need
    ok = (fits & ((need == 0) | (before + need <= top))) | ended
    j = col - have[:, None]
    new = (ok & ~ended)[:, None] & (j >= 0) & (j < need[:, None])
    table = torch.where(new, free[(top - 1 - before[:, None] - j).clamp(0, pool - 1)], table)
    taken = torch.where(ok, before + need, torch.zeros_like(need)).where(need > 0, torch.zeros_like(need)).amax()
    lens_out = torch.where(ended, torch.zeros_like(held), torch.where(ok, held + add, held))
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(add, 0)])
    t = torch.arange(cap, device=dev)
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=add.shape[0] - 1)
    live = t < cu[-1]
    pos = torch.where(live, held[seq] + t - cu[seq], torch.zeros_like(t))
    pg = table[seq, torch.div(pos, page, rounding_mode="floor").clamp(max=width - 1)].long()
    slot = torch.where(live & ok[seq] & (pg >= 0) & (pg < s["pages"]), pg * page + pos % page, torch.full_like(t, -1))
    i32 = torch.int32
    return {"lens_out": lens_out.to(i32), "count_out": torch.cat([top - taken, (~ok).sum()[None]]).to(i32),
            "cu": cu.to(i32), "slots": slot.to(i32), "pos": pos.to(i32), "table": table, "free": free}


def _plain_norm(s):
    u = s["x"].float()
    if s["post"] is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + s["eps"]) * s["post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = s["alpha"] * s["h"].float() + s["beta"] * u
    y = (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["pre"].float()).to(s["x"].dtype)
    if s["out"] == "int8":
        g = y.float().view(y.shape[0], -1, 128)
        top = g.abs().amax(-1, keepdim=True)
        sc = top / torch.full_like(top, 127.0)
        q = torch.round(g / torch.where(sc == 0, torch.ones_like(sc), sc)).clamp(-127, 127)
        y = (q * sc).half()
    return {"h": h.to(s["h"].dtype), "y": y}


# --------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "norm": _exact_norm}[case["op"]](s)


def _exact_attend(s):
    q, page, (t, hq, d) = s["q"].double(), s["page"], s["q"].shape
    cu, lens, hkv, g = s["cu"].tolist(), s["lens"].tolist(), s["cache"].shape[1], d // 64
    half, gq = page * d // 2, hq // hkv
    out = torch.zeros(t, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((t, hq), float("-inf"), dtype=torch.float64, device="cuda")
    # where a channel's nibble is: by its position in the key row and in the value words
    ch = torch.arange(d, device="cuda")
    kbyte = (ch % 32) // 8 * (d // 8) + ch // 32 * 4 + ch % 8 // 2
    vcol, vbyte = ch % 16, ch // 32
    for b, n in enumerate(lens):
        r = cu[b + 1] - cu[b]
        if not r or not n:
            continue
        tok = torch.arange(n, device="cuda")
        blk, off = s["table"][b, tok // page].long(), tok % page
        pos = torch.arange(n - r, n, device="cuda")
        hide = tok > pos[:, None]
        if s["window"]:
            hide = hide | (tok <= pos[:, None] - s["window"])
        for h in range(hkv):
            c = s["cache"][:, h]
            kc = c[blk[:, None], off[:, None] * (d // 2) + kbyte]
            kc = torch.where(ch % 2 == 0, kc & 15, kc >> 4).double()
            vc = c[blk[:, None], half + (((off // 4)[:, None] * 16 + vcol) * 4 + (off % 4)[:, None]) * (d // 32) + vbyte]
            vc = torch.where(ch // 16 % 2 == 0, vc & 15, vc >> 4).double()
            par = c[:, 2 * half:].contiguous().view(torch.float16).view(-1, 2, page, 2, g)[blk, :, off].double()
            k = par[:, 0, 1][:, ch // 64] + par[:, 0, 0][:, ch // 64] * kc
            v = par[:, 1, 1][:, ch // 64] + par[:, 1, 0][:, ch // 64] * vc
            for x in range(h * gq, (h + 1) * gq):
                sc = (q[cu[b]: cu[b + 1], x] @ k.t()) * s["scale"]
                sc = sc.masked_fill(hide, float("-inf"))
                z = torch.logsumexp(sc, -1, keepdim=True)
                out[cu[b]: cu[b + 1], x] = torch.exp(sc - z).nan_to_num(0.0) @ v
                lse[cu[b]: cu[b + 1], x] = z[:, 0]
    return {"out": out, "lse": lse}


def _f32(x):
    """A value of the definition that is held in 32 bits."""
    return x.float().double()


def _exact_append(s):
    def back(x):
        t, h, d = x.shape
        g = x.double().view(t, h, d // 64, 64)
        lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
        m = lo.half().double()
        sc = _f32(_f32(hi - lo) / 15.0).half().double()
        sc = torch.where((sc == 0) & (hi > lo), torch.full_like(sc, 2.0 ** -24), sc)
        f = _f32(_f32(g - m) / sc.clamp(min=2.0 ** -24))
        c = torch.floor(f)
        c = torch.where((f - c > 0.5) | ((f - c == 0.5) & (c % 2 == 1)), c + 1, c).clamp(0, 15)
        y = m + torch.where(sc == 0, torch.zeros_like(c), sc * c)
        return y.view(t, h, d) * (s["slots"] >= 0).double()[:, None, None]

    return {"k": back(s["k"]), "v": back(s["v"])}


def _exact_norm(s):
    d = lambda x: 1.0 if x is None else x.double()  # noqa: E731
    x, h = s["x"].double(), s["h"].double()
    if s["post"] is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * s["post"].double()
    h = s["alpha"] * h + s["beta"] * d(s["gate"]) * x
    y = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + s["eps"]) * s["pre"].double()
    if s["out"] == "int8":
        y = y.to(s["x"].dtype).double().view(y.shape[0], -1, 128)
        sc = _f32(y.abs().max(-1, keepdim=True).values / 127.0)
        y = torch.round(y / torch.where(sc == 0, torch.ones_like(sc), sc)) * sc
    return {"h": h, "y": y}
