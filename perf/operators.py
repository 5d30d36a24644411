"""Cases of the softmax-attention layer of a hybrid stack: the norm of queries and keys for each
head with the position rotation (forward and backward), the paged 8-bit key / value cache
(append and read back), and the attention over that cache.

``own`` false: the plain forms, elementary torch operations in fp32.  ``own`` true: the calls of
the package.  Layer sizes: 16 query heads of 128 (the layer of this repository's benchmark) or 8
of 64 (its smaller configuration), with 4 key / value heads or as many as query heads.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
CODE_MAX = {"i8": 127.0, "e4m3": 448.0}
CODE_TYPE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token for each of 64 running sequences: a serving step, where latency counts
        dict(name="rope step b64", op="rope", bwd=False, B=64, T=1, Hq=16, Hk=4, d=128, rot=128,
             style="halves", io="bf16", packed=True),
        # a training batch of the benchmark's layer, q and k read out of the packed projection
        dict(name="rope fwd b8 t4096", op="rope", bwd=False, B=8, T=4096, Hq=16, Hk=4, d=128,
             rot=128, style="halves", io="bf16", packed=True),
        # odd sizes in fp32: a head that is no power of two, rotated in part, adjacent pairs
        dict(name="rope fwd f32 odd", op="rope", bwd=False, B=3, T=1021, Hq=5, Hk=5, d=96, rot=32,
             style="pairs", io="f32", packed=False),
        # the backward pass of the training batch
        dict(name="rope bwd b8 t4096", op="rope", bwd=True, B=8, T=4096, Hq=16, Hk=4, d=128,
             rot=128, style="halves", io="bf16", packed=True),
        # the backward pass of the smaller layer in fp32, ragged length, rotated in part
        dict(name="rope bwd f32 odd", op="rope", bwd=True, B=2, T=777, Hq=8, Hk=2, d=64, rot=32,
             style="halves", io="f32", packed=False),
        # a serving step: one token appended for each of 64 sequences, the pages it touched read back
        dict(name="cache step b64", op="cache", code="i8", B=64, T=1, lo=1, hi=4000, H=4, d=128,
             page=64, io="bf16", out="f32"),
        # prompts of up to 4096 tokens written into an empty cache, and read back
        dict(name="cache prompts b8", op="cache", code="e4m3", B=8, T=4096, lo=0, hi=0, H=4, d=128,
             page=64, io="bf16", out="bf16"),
        # a step of a single short sequence: the smallest call
        dict(name="attn step b1", op="attn", code="i8", B=1, T=1, lo=1000, hi=1000, Hq=16, H=4,
             d=128, page=64, window=0, io="bf16", out="bf16"),
        # a step of a full batch with ragged lengths
        dict(name="attn step b64", op="attn", code="i8", B=64, T=1, lo=17, hi=8191, Hq=16, H=4,
             d=128, page=64, window=0, io="bf16", out="bf16"),
        # two very long documents: few rows, a long axis
        dict(name="attn step long", op="attn", code="e4m3", B=2, T=1, lo=200001, hi=262143, Hq=16,
             H=4, d=128, page=128, window=0, io="bf16", out="bf16"),
        # five drafted tokens checked at once, in fp32, heads of their own, sliding window, small pages
        dict(name="attn draft f32 window", op="attn", code="i8", B=13, T=5, lo=300, hi=5001, Hq=8,
             H=8, d=64, page=16, window=2048, io="f32", out="f32"),
        # chunks of four prompts over what is cached of them: many rows, bound by the products
        dict(name="attn chunk t512", op="attn", code="i8", B=4, T=512, lo=4000, hi=8191, Hq=16, H=4,
             d=128, page=64, window=0, io="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n == 3 << 10 else n


def draw(rng):
    op = rng.choice(["rope", "rope", "cache", "attn", "attn", "attn"])
    io = rng.choice(["bf16", "bf16", "f32"])
    H = rng.choice([1, 2, 4, 8])
    if op == "rope":
        d = rng.choice([64, 96, 128])
        Hq = H * rng.choice([1, 2, 4]) if H < 8 else 8
        # values over all tokens: at most those of the training batch
        tokens = _log(rng, 1, 32768 * 20 * 128 // ((Hq + H) * d * (1 if io == "bf16" else 2)))
        tokens = min(tokens, 65536)
        B = min(tokens, _log(rng, 1, 64))
        return dict(op=op, bwd=rng.random() < 0.5, B=B, T=max(1, tokens // B), Hq=Hq, Hk=H, d=d,
                    rot=rng.choice([r for r in (32, 64, 96, 128) if r <= d]),
                    style=rng.choice(["halves", "pairs"]), io=io, packed=rng.random() < 0.5)
    code, d, page = rng.choice(["i8", "e4m3"]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    out = "f32" if io == "f32" else rng.choice(["bf16", "bf16", "f32"])
    if op == "cache":
        T = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(64, 24576 * 4 * 128 // (T * H * d * (1 if out == "bf16" else 2)))))
        lo = rng.choice([0, 0, 37])
        return dict(op=op, code=code, B=B, T=T, lo=lo, hi=lo + _log(rng, 1, 4000) if lo else 0, H=H, d=d,
                    page=page, io=io, out=out)
    T = rng.choice([1, 1, 1, 1, _log(rng, 2, 16), _log(rng, 17, 512)])
    B = _log(rng, 1, 64 if T <= 16 else 4)
    Hq = H * rng.choice([1, 2, 4]) if H < 8 else 8
    # positions over all sequences: at most those of the largest listed cases, by the bytes that a
    # step reads and by the products of a chunk
    total = min(460000 * 4 * 128 // (H * d), 24000 * 512 * 16 * 128 // (T * Hq * d))
    hi = _log(rng, 16, max(16, min(total, 500000) // B))
    return dict(op=op, code=code, B=B, T=T, lo=rng.choice([0, hi // 3, hi]), hi=hi, Hq=Hq, H=H, d=d, page=page,
                window=rng.choice([0, 0, 0, 1 + hi // 2]), io=io, out=out)


def _lens(c):
    """The lengths before the call: spread evenly over lo .. hi (their order is the seed's)."""
    B = c["B"]
    return [c["hi"] if B == 1 else c["lo"] + (c["hi"] - c["lo"]) * b // (B - 1) for b in range(B)]


def _news(c):
    """The new tokens of each sequence: T, or spread over T / 2 .. T where a prompt is written."""
    B, T = c["B"], c["T"]
    return [T if c["op"] == "attn" or B == 1 or T == 1 else T - (T // 2) * b // (B - 1) for b in range(B)]


def _back_rows(c):
    """The rows of the pages that T tokens can touch."""
    return c["page"] * (1 + (c["page"] - 2 + c["T"]) // c["page"])


# ------------------------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _quantised_pool(gen, pages, c):
    """Codes and scales of a pool whose every page holds values of unit size."""
    H, page, d = c["H"], c["page"], c["d"]
    codes = torch.empty(pages, H, page, d, dtype=CODE_TYPE[c["code"]], device="cuda")
    scale = torch.empty(pages, H, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (H * page * d))
    for i in range(0, pages, step):
        x = _randn(gen, min(step, pages - i), H, page, d)
        s = x.abs().amax((2, 3)) * (1 / CODE_MAX[c["code"]])
        codes[i:i + step] = _to_codes(x / s[:, :, None, None], c["code"])
        scale[i:i + step] = s
    return codes, scale


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = np.random.RandomState(seed % (1 << 31))
    dt = DTYPES[c["io"]]
    B, T, d = c["B"], c["T"], c["d"]
    st = dict(case=c)
    if c["op"] == "rope":
        Hq, Hk = c["Hq"], c["Hk"]
        if c["packed"]:
            qkv = _randn(gen, B, T, Hq + 2 * Hk, d).to(dt)
            st["q"], st["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        else:
            st["q"], st["k"] = _randn(gen, B, T, Hq, d).to(dt), _randn(gen, B, T, Hk, d).to(dt)
        st["wq"] = 1 + 0.1 * _randn(gen, d)
        st["wk"] = 1 + 0.1 * _randn(gen, d)
        past = 4096 if T == 1 else 64
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
        ang = (torch.arange(past + T, dtype=torch.float64)[:, None] * freq).cuda()
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["start"] = torch.from_numpy(order.randint(0, past + 1, B).astype(np.int32)).cuda()
        if c["bwd"]:
            st["dyq"] = _randn(gen, B, T, Hq, d).to(dt)
            st["dyk"] = _randn(gen, B, T, Hk, d).to(dt)
        if own:
            from delta_rule_recurrent_gated_gb300 import binding
            st["plan"] = binding.HeadNormRope(B, T, Hq, Hk, d, rot=c["rot"], style=c["style"],
                                              io=c["io"], out=c["io"], grad=c["io"], eps=EPS)
        return st
    lens, news = np.array(_lens(c)), np.array(_news(c))
    order.shuffle(lens)
    order.shuffle(news)
    per = (int((lens + news).max()) + c["page"] - 1) // c["page"]
    pages = B * per
    st["k_codes"], st["k_scale"] = _quantised_pool(gen, pages, c)
    st["v_codes"], st["v_scale"] = _quantised_pool(gen, pages, c)
    # pages come in any order, as after a day of serving
    st["table"] = torch.from_numpy(order.permutation(pages).reshape(B, per).astype(np.int32)).cuda()
    st["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    st["news"] = torch.from_numpy(news.astype(np.int32)).cuda()
    if c["op"] == "cache":
        st["k"], st["v"] = _randn(gen, B, T, c["H"], d).to(dt), _randn(gen, B, T, c["H"], d).to(dt)
        first = (lens // c["page"]) * c["page"]
        st["back_T"] = _back_rows(c) if lens.any() else T
        st["first"] = torch.from_numpy(first.astype(np.int32)).cuda()
        st["back"] = torch.from_numpy((lens + news - first).astype(np.int32)).cuda()
    else:
        st["q"] = _randn(gen, B, T, c["Hq"], d).to(dt)
    if own:
        from delta_rule_recurrent_gated_gb300 import binding
        st["cache"] = binding.KvCache(pages, c["H"], d, page=c["page"], code=c["code"],
                                      buffers=(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"]))
        if c["op"] == "attn":
            st["plan"] = binding.CacheAttention(st["cache"], B, T, c["Hq"],
                                                io=c["io"], out=c["out"], scale=1 / math.sqrt(d),
                                                window=c["window"])
    return st


# ------------------------------------------------------------------------------- plain forms
def _to_codes(x, code):
    if code == "i8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _pick(codes, *at):
    """Indexing of the codes as bytes, whatever type they stand for."""
    return codes.view(torch.int8)[at].view(codes.dtype)


def _rotate(n, cos, sin, style):
    """The rotation of the leading channels of n [B, T, H, d] by cos, sin [B, T, 1, rot / 2]."""
    half = cos.shape[-1]
    rot = 2 * half
    if style == "halves":
        a, b = n[..., :half], n[..., half:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = n[..., 0:rot:2], n[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, n[..., rot:]], -1)


def _angles(st, kind):
    T = st["case"]["T"]
    pos = st["start"].long()[:, None] + torch.arange(T, device=st["start"].device)
    return st["cos"].to(kind)[pos][:, :, None], st["sin"].to(kind)[pos][:, :, None]


def _norm_fwd(x, w, cos, sin, style):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _rotate(x * r * w, cos, sin, style)


def _norm_bwd(x, w, cos, sin, style, dy):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    m = _rotate(dy, cos, -sin, style)
    g = m * w
    dx = r * g - x * r * r * r * (g * x).mean(-1, keepdim=True)
    return dx, (m * x * r).sum((0, 1, 2))


def _plain_rope(st):
    c = st["case"]
    dt = DTYPES[c["io"]]
    q, k = st["q"].float(), st["k"].float()
    cos, sin = _angles(st, torch.float32)
    if not c["bwd"]:
        return (_norm_fwd(q, st["wq"], cos, sin, c["style"]).to(dt),
                _norm_fwd(k, st["wk"], cos, sin, c["style"]).to(dt))
    dq, dwq = _norm_bwd(q, st["wq"], cos, sin, c["style"], st["dyq"].float())
    dk, dwk = _norm_bwd(k, st["wk"], cos, sin, c["style"], st["dyk"].float())
    return dict(dq=dq.to(dt), dk=dk.to(dt), dwq=dwq, dwk=dwk)


def _append(codes, scale, x, st):
    """Appends x [B, T, H, d] to the pool in place."""
    c = st["case"]
    code, page, T = c["code"], c["page"], c["T"]
    lens, news, table = st["lens"].long(), st["news"].long(), st["table"].long()
    B, dev = c["B"], codes.device
    # the pages that T tokens can touch, each as a window of `page` rows of the new tokens
    n = 1 + (page - 2 + T) // page
    first = lens // page
    at = (first[:, None] + torch.arange(n, device=dev))                        # [B, n]
    row = at[:, :, None] * page + torch.arange(page, device=dev)               # position
    t = row - lens[:, None, None]                                              # new token, [B, n, page]
    new = (t >= 0) & (t < news[:, None, None])
    old = t < 0
    touched = new.any(-1)                                                      # [B, n]
    ids = table.gather(1, at.clamp(max=table.shape[1] - 1))
    xs = x.gather(1, t.clamp(0, T - 1).reshape(B, n * page)[:, :, None, None].expand(-1, -1, *x.shape[2:]))
    xs = xs.reshape(B, n, page, *x.shape[2:]).transpose(2, 3).float()          # [B, n, H, page, d]
    newe = new[:, :, None, :, None]
    top = torch.where(newe, xs.abs(), 0.0).amax((3, 4)) * (1 / CODE_MAX[code])  # [B, n, H]
    s_old = torch.where(old.any(-1)[:, :, None], scale[ids], 0.0)
    s = torch.maximum(s_old, top)
    se, soe = s[..., None, None], s_old[..., None, None]
    was = _pick(codes, ids)
    kept = torch.where(se > soe, _to_codes(was.float() * soe / se, code).float(), was.float())
    got = torch.where(se > 0, _to_codes(xs / se, code).float(), 0.0)
    now = torch.where(newe, got, torch.where(old[:, :, None, :, None], kept, was.float())).to(codes.dtype)
    use = ids[touched]
    codes.view(torch.int8)[use] = now.view(torch.int8)[touched]
    scale[use] = s[touched]


def _values(codes, scale, table, page, lens, T, kind):
    """Tokens lens .. lens + T - 1 of every sequence as values [B, T, H, d]."""
    pos = lens.long()[:, None] + torch.arange(T, device=codes.device)
    ids = table.long().gather(1, (pos // page).clamp(max=table.shape[1] - 1))
    return _pick(codes, ids, slice(None), pos % page).to(kind) * scale[ids].to(kind)[..., None]


def _plain_cache(st):
    c = st["case"]
    _append(st["k_codes"], st["k_scale"], st["k"], st)
    _append(st["v_codes"], st["v_scale"], st["v"], st)
    T = st["back_T"]
    there = (torch.arange(T, device="cuda") < st["back"][:, None])[:, :, None, None]
    out = DTYPES[c["out"]]
    k = _values(st["k_codes"], st["k_scale"], st["table"], c["page"], st["first"], T, torch.float32)
    v = _values(st["v_codes"], st["v_scale"], st["table"], c["page"], st["first"], T, torch.float32)
    return dict(k=torch.where(there, k, 0.0).to(out), v=torch.where(there, v, 0.0).to(out),
                k_scale=st["k_scale"], v_scale=st["v_scale"])


def _whole(codes, scale, table, kind):
    x = _pick(codes, table.long()).to(kind) * scale[table.long()].to(kind)[..., None, None]  # [B, n, H, page, d]
    return x.transpose(1, 2).flatten(2, 3)                                           # [B, H, n * page, d]


def _attend(st, kind):
    c = st["case"]
    B, T, Hq, H, d = c["B"], c["T"], c["Hq"], c["H"], c["d"]
    k = _whole(st["k_codes"], st["k_scale"], st["table"], kind)
    v = _whole(st["v_codes"], st["v_scale"], st["table"], kind)
    q = st["q"].to(kind).reshape(B, T, H, Hq // H, d).permute(0, 2, 3, 1, 4).reshape(B, H, Hq // H * T, d)
    s = (q @ k.transpose(-1, -2)).reshape(B, H, Hq // H, T, -1) / math.sqrt(d)
    p = st["lens"].long()[:, None] + torch.arange(T, device="cuda")                  # [B, T]
    j = torch.arange(s.shape[-1], device="cuda")
    see = j <= p[..., None]
    if c["window"]:
        see &= j > p[..., None] - c["window"]
    s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = (s - top).exp_()
    tot = e.sum(-1, keepdim=True)
    o = ((e / tot).reshape(B, H, Hq // H * T, -1) @ v).reshape(B, H, Hq // H, T, d)
    lse = (top + tot.log())[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, d), lse.permute(0, 3, 1, 2).reshape(B, T, Hq)


def _plain_attn(st):
    o, lse = _attend(st, torch.float32)
    return dict(o=o.to(DTYPES[st["case"]["out"]]), lse=lse)


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "cache": _plain_cache, "attn": _plain_attn}[op](state)
    if op == "rope":
        a = [state[n] for n in ("q", "k", "wq", "wk", "cos", "sin")]
        if not state["case"]["bwd"]:
            return state["plan"].forward(*a, start=state["start"])
        return state["plan"].backward(*a, state["dyq"], state["dyk"], start=state["start"])
    if op == "cache":
        state["cache"].write(state["k"], state["v"], state["table"], state["lens"], state["news"])
        k, v = state["cache"].read(state["table"], state["first"], state["back"], state["back_T"],
                                   out=state["case"]["out"])
        return dict(k=k, v=v, k_scale=state["k_scale"], v_scale=state["v_scale"])
    o, lse = state["plan"].forward(state["q"], state["table"], state["lens"], want_lse=True)
    return dict(o=o, lse=lse)


# ------------------------------------------------------------------------------- work
def work(case):
    c = case
    B, T, d = c["B"], c["T"], c["d"]
    io = 2 if c["io"] == "bf16" else 4
    if c["op"] == "rope":
        n = B * T * (c["Hq"] + c["Hk"]) * d
        table = B * T * c["rot"] * 4 if T == 1 else (64 + T) * c["rot"] * 4
        return dict(bytes=n * io * (3 if c["bwd"] else 2) + table + (4 if c["bwd"] else 2) * d * 4,
                    flops=n * (16 if c["bwd"] else 8))
    lens, news = _lens(c), _news(c)
    out = 2 if c["out"] == "bf16" else 4
    if c["op"] == "cache":
        new = sum(news) * c["H"] * d
        back = sum(n + x % c["page"] for x, n in zip(lens, news)) * c["H"] * d
        rows = B * (_back_rows(c) if any(lens) else T) * c["H"] * d  # with the zeros behind the last token
        touched = sum((x + n - 1) // c["page"] - x // c["page"] + 1 for x, n in zip(lens, news)) * c["H"]
        return dict(bytes=2 * (new * (io + 1) + back + rows * out + 2 * touched * 4), flops=2 * (3 * new + back))
    seen = pairs = 0
    for x in lens:
        low = max(0, x + 1 - c["window"]) if c["window"] else 0
        seen += x + T - low
        pairs += sum(min(x + t + 1, c["window"] or x + t + 1) for t in range(T))
    return dict(bytes=2 * seen * c["H"] * d + B * T * c["Hq"] * (d * (io + out) + 4),
                flops=4 * d * c["Hq"] * pairs)


# ------------------------------------------------------------------------------- 64 bits
def _exact_rope(st):
    c = st["case"]
    d, rot = c["d"], c["rot"]
    pos = (st["start"].long()[:, None] + torch.arange(c["T"], device="cuda")).flatten()
    cos, sin = st["cos"].double()[pos], st["sin"].double()[pos]
    if c["style"] == "halves":
        ia, ib = torch.arange(rot // 2, device="cuda"), torch.arange(rot // 2, rot, device="cuda")
    else:
        ia = torch.arange(0, rot, 2, device="cuda")
        ib = ia + 1

    def one(x, w, dy):
        x, w = x.double().flatten(0, 1), w.double()
        inv = 1 / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
        if dy is None:
            n = x * inv * w
            y = n.clone()
            y[..., ia] = n[..., ia] * cos[:, None] - n[..., ib] * sin[:, None]
            y[..., ib] = n[..., ib] * cos[:, None] + n[..., ia] * sin[:, None]
            return y.reshape(c["B"], c["T"], -1, d)
        dy = dy.double().flatten(0, 1)
        m = dy.clone()
        m[..., ia] = dy[..., ia] * cos[:, None] + dy[..., ib] * sin[:, None]
        m[..., ib] = dy[..., ib] * cos[:, None] - dy[..., ia] * sin[:, None]
        hat = x * inv
        dw = torch.einsum("nhd,nhd->d", m, hat)
        g = m * w
        dx = inv * (g - hat * ((g * hat).sum(-1, keepdim=True) / d))
        return dx.reshape(c["B"], c["T"], -1, d), dw

    if not c["bwd"]:
        return one(st["q"], st["wq"], None), one(st["k"], st["wk"], None)
    (dq, dwq), (dk, dwk) = one(st["q"], st["wq"], st["dyq"]), one(st["k"], st["wk"], st["dyk"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _round_to_code(x, code):
    """The nearest code value of x, ties to even, from the grid's own spacing."""
    if code == "i8":
        return x.round().clamp(-127, 127)
    _, e = torch.frexp(x)                       # |x| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return ((x / step).round() * step).clamp(-448, 448)


def _exact_cache(st):
    """Sequence by sequence and page by page, as the definition reads."""
    c = st["case"]
    page, H, d, code = c["page"], c["H"], c["d"], c["code"]
    lens, back, table = st["lens"].tolist(), st["back"].tolist(), st["table"].tolist()
    news, res = st["news"].tolist(), {}
    for name in ("k", "v"):
        x, codes, scale = st[name].double(), st[name + "_codes"], st[name + "_scale"].double()
        out = torch.zeros(c["B"], st["back_T"], H, d, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            p, end, at = lens[b], lens[b] + news[b], 0
            while p < end:
                stop = min(end, (p // page + 1) * page)
                i, r = table[b][p // page], p % page
                new = x[b, p - lens[b]:stop - lens[b]]                         # [rows, H, d]
                s = (new.abs().amax((0, 2)) / CODE_MAX[code])                  # [H]
                if r:
                    kept = codes[i].double()[:, :r]
                    s_old = scale[i]
                    s = torch.maximum(s, s_old)
                    grown = _round_to_code(kept * (s_old / s)[:, None, None], code)
                    kept = torch.where((s > s_old)[:, None, None], grown, kept)
                    out[b, at:at + r] = (kept * s[:, None, None]).transpose(0, 1)
                    at += r
                scale[i] = s
                out[b, at:at + stop - p] = _round_to_code(new / s[:, None], code) * s[:, None]
                at += stop - p
                p = stop
        res[name], res[name + "_scale"] = out, scale
    return res


def _exact_attn(st):
    """One sequence at a time, the sums by the definition."""
    c = st["case"]
    T, Hq, H, d, page = c["T"], c["Hq"], c["H"], c["d"], c["page"]
    o = torch.zeros(c["B"], T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["B"], T, Hq, dtype=torch.float64, device="cuda")
    for b, x in enumerate(st["lens"].tolist()):
        ids = st["table"][b, :(x + T + page - 1) // page].long()
        kv = []
        for name in ("k", "v"):
            y = _pick(st[name + "_codes"], ids).double() * st[name + "_scale"][ids].double()[:, :, None, None]
            kv.append(y.permute(1, 0, 2, 3).reshape(H, -1, d)[:, :x + T])
        dist = (x + torch.arange(T, device="cuda"))[:, None] - torch.arange(x + T, device="cuda")
        hidden = (dist < 0) | (dist >= c["window"]) if c["window"] else dist < 0
        for h in range(Hq):
            s = st["q"][b, :, h].double() @ kv[0][h * H // Hq].T / d ** 0.5
            s[hidden] = -math.inf
            lse[b, :, h] = torch.logsumexp(s, -1)
            o[b, :, h] = torch.exp(s - lse[b, :, h, None]) @ kv[1][h * H // Hq]
    return dict(o=o, lse=lse)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "cache": _exact_cache, "attn": _exact_attn}[case["op"]](st)
