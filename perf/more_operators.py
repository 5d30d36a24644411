"""Cases of the token mixers that a hybrid stack has beside the delta rule: causal softmax attention
over whole prompts (forward and backward; grouped heads, packed sequences, sliding window) and linear
attention with a decay for each head (chunked forward and backward, recurrent step).

``own`` false: the plain forms, elementary torch operations in fp32.  ``own`` true: the calls of the
package.  Layer sizes: 16 heads of 128 (the layer of this repository's benchmark) or 8 of 64 (its
smaller configuration), for softmax attention with 4 or 2 key / value heads or as many as query heads.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # tokens of a chunk of the plain chunked form


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a short prompt of one user: the smallest call, where latency counts
        dict(name="attn prompt t100", op="attn", train=False, N=1, lo=100, hi=100, Hq=16, H=4, d=128,
             window=0, io="bf16", packed=False),
        # the training batch of the benchmark's layer, forward only, as in an evaluation
        dict(name="attn fwd b8 t4096", op="attn", train=False, N=8, lo=4096, hi=4096, Hq=16, H=4, d=128,
             window=0, io="bf16", packed=False),
        # a long document, sliding window, heads of their own
        dict(name="attn fwd long window", op="attn", train=False, N=1, lo=20011, hi=20011, Hq=8, H=8, d=64,
             window=2048, io="bf16", packed=False),
        # a training step of the benchmark's layer
        dict(name="attn train b8 t4096", op="attn", train=True, N=8, lo=4096, hi=4096, Hq=16, H=4, d=128,
             window=0, io="bf16", packed=False),
        # a training step over documents of 1 to 2500 tokens, packed one behind the other
        dict(name="attn train packed", op="attn", train=True, N=16, lo=1, hi=2500, Hq=16, H=4, d=128,
             window=0, io="bf16", packed=True),
        # fp32, packed, odd lengths, the smaller layer
        dict(name="attn train f32 odd", op="attn", train=True, N=5, lo=33, hi=1021, Hq=8, H=2, d=64,
             window=0, io="f32", packed=True),
        # one new token for each of 64 running sequences: a serving step, bound by the states
        dict(name="lin step b64", op="step", N=64, T=1, H=16, dk=128, dv=128, io="bf16"),
        # five drafted tokens of one sequence, in fp32: the smallest call
        dict(name="lin draft b1 f32", op="step", N=1, T=5, H=8, dk=64, dv=64, io="f32"),
        # one long prompt that continues from a state: few heads, a long axis
        dict(name="lin prompt long", op="lin", train=False, N=1, lo=16411, hi=16411, H=16, dk=128, dv=128,
             state=True, io="bf16", packed=False),
        # a training step of the benchmark's layer
        dict(name="lin train b8 t4096", op="lin", train=True, N=8, lo=4096, hi=4096, H=16, dk=128, dv=128,
             state=False, io="bf16", packed=False),
        # a training step over packed documents of 1 to 2500 tokens with states in and out
        dict(name="lin train packed", op="lin", train=True, N=16, lo=1, hi=2500, H=8, dk=64, dv=128,
             state=True, io="bf16", packed=True),
        # fp32, packed, odd lengths, small heads
        dict(name="lin train f32 odd", op="lin", train=True, N=5, lo=33, hi=1021, H=8, dk=32, dv=64,
             state=True, io="f32", packed=True),
    ]


def _log(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n == 3 << 10 else n


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "lin", "lin", "step"])
    io = rng.choice(["bf16", "bf16", "f32"])
    wide = [64, 128] if io == "bf16" else [16, 32, 64, 128]
    if op == "step":
        H, dk, dv = rng.choice([4, 8, 16, 32]), rng.choice(wide), rng.choice(wide)
        # values of the states: at most those of the serving step
        B = _log(rng, 1, min(512, 64 * 16 * 128 * 128 // (H * dk * dv)))
        return dict(op=op, N=B, T=rng.choice([1, 1, 1, 2, 5]), H=H, dk=dk, dv=dv, io=io)
    train, packed = rng.random() < 0.5, rng.random() < 0.5
    if op == "attn":
        H, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        Hq = H * rng.choice([1, 2, 4, 5]) if H < 8 else 8
        # scores of all padded sequences: at most those of the training batch, fewer in fp32
        scores = 8 * 4096 * 4096 * 16 // (1 if io == "bf16" else 16)
        hi = _log(rng, 16, min(20000, int((scores // Hq) ** 0.5)))
        N = _log(rng, 1, max(1, min(64, scores // Hq // (hi * hi), 65536 // hi)))
        return dict(op=op, train=train, N=N, lo=rng.choice([0, 1, hi // 3]) if packed else hi, hi=hi, Hq=Hq, H=H, d=d,
                    window=rng.choice([0, 0, 0, 1 + hi // 3]), io=io, packed=packed)
    H, dk, dv = rng.choice([1, 2, 4, 8, 16]), rng.choice(wide), rng.choice(wide)
    # tokens times heads and channels: at most those of the training batch, fewer in fp32
    tokens = 8 * 4096 * 16 * 256 // (H * (dk + dv)) // (1 if io == "bf16" else 8)
    hi = _log(rng, 16, min(32768, tokens))
    N = _log(rng, 1, max(1, min(64, tokens // hi)))
    return dict(op=op, train=train, N=N, lo=rng.choice([0, 1, hi // 3]) if packed else hi, hi=hi, H=H, dk=dk, dv=dv,
                state=rng.random() < 0.5, io=io, packed=packed)


def _lens(c):
    """Lengths of the sequences, spread evenly over lo .. hi (their order is the seed's)."""
    N = c["N"]
    return [c["hi"] if N == 1 else c["lo"] + (c["hi"] - c["lo"]) * b // (N - 1) for b in range(N)]


# ------------------------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _rates(H):
    """Log-decays of the heads: memories of 32 tokens for the first, longer and longer ones after it."""
    at = torch.arange(H, dtype=torch.float64)
    return torch.log1p(-torch.exp2(-5.0 - 6.0 * at / max(1, H - 1))).float().cuda()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = np.random.RandomState(seed % (1 << 31))
    dt = DTYPES[c["io"]]
    st = dict(case=c)
    if c["op"] == "step":
        B, T, H = c["N"], c["T"], c["H"]
        st["q"], st["k"] = _randn(gen, B, T, H, c["dk"]).to(dt), _randn(gen, B, T, H, c["dk"]).to(dt)
        st["v"], st["g"] = _randn(gen, B, T, H, c["dv"]).to(dt), _rates(H)
        st["state"] = 4 * _randn(gen, B, H, c["dk"], c["dv"])
        if own:
            from delta_rule_recurrent_gated_gb300 import binding
            st["plan"] = binding.LinearAttention(B, T, H, c["dk"], c["dv"], io=c["io"], scale=c["dk"] ** -0.5)
        return st
    lens = np.array(_lens(c))
    order.shuffle(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    total, N = int(cu[-1]), c["N"]
    st["cu"] = torch.from_numpy(cu.astype(np.int32)).cuda() if c["packed"] else None
    B, T = (1, total) if c["packed"] else (N, c["hi"])
    # where every token lies in a batch padded to the longest length, for the plain form
    st["row"] = torch.from_numpy(np.concatenate([b * c["hi"] + np.arange(n) for b, n in enumerate(lens)]).astype(np.int64)).cuda()
    st["lens"] = lens.tolist()
    if c["op"] == "attn":
        # q, k (normed and rotated) in tensors of their own, v still a head range of the packed projection
        Hq, H, d = c["Hq"], c["H"], c["d"]
        st["q"], st["k"] = _randn(gen, B, T, Hq, d).to(dt), _randn(gen, B, T, H, d).to(dt)
        st["v"] = _randn(gen, B, T, Hq + 2 * H, d).to(dt)[:, :, Hq + H:]
        if c["train"]:
            st["dO"] = _randn(gen, B, T, Hq, d).to(dt)
        if own:
            from delta_rule_recurrent_gated_gb300 import binding
            st["plan"] = binding.PromptAttention(B, T, Hq, H, d, seqs=N if c["packed"] else None, io=c["io"],
                                                 window=c["window"])
        return st
    H, dk, dv = c["H"], c["dk"], c["dv"]
    st["q"], st["k"] = _randn(gen, B, T, H, dk).to(dt), _randn(gen, B, T, H, dk).to(dt)
    st["v"], st["g"] = _randn(gen, B, T, H, dv).to(dt), _rates(H)
    st["h0"] = 4 * _randn(gen, N, H, dk, dv) if c["state"] else None
    if c["train"]:
        st["dO"] = _randn(gen, B, T, H, dv).to(dt)
        st["dhT"] = _randn(gen, N, H, dk, dv) if c["state"] else None
    if own:
        from delta_rule_recurrent_gated_gb300 import binding
        st["plan"] = binding.LinearAttention(B, T, H, dk, dv, seqs=N if c["packed"] else None, io=c["io"],
                                             scale=dk ** -0.5)
    return st


# ------------------------------------------------------------------------------- plain forms
def _pad(x, st, T):
    """x [B, T, H, d] as fp32 [N, H, T, d], zeros behind each sequence's tokens."""
    c = st["case"]
    y = torch.zeros(c["N"] * T, *x.shape[2:], dtype=torch.float32, device=x.device)
    row = st["row"] if T == c["hi"] else st["row"] // c["hi"] * T + st["row"] % c["hi"]
    y[row] = x.flatten(0, 1).float()
    return y.unflatten(0, (c["N"], T)).transpose(1, 2)


def _unpad(y, like, st):
    """Back to the layout and type of `like`."""
    c = st["case"]
    T = y.shape[2]
    row = st["row"] if T == c["hi"] else st["row"] // c["hi"] * T + st["row"] % c["hi"]
    return y.transpose(1, 2).flatten(0, 1)[row].to(like.dtype).reshape(*like.shape[:2], *y.shape[1:2], y.shape[3])


def _plain_attn(st):
    c = st["case"]
    N, T, Hq, H, d = c["N"], c["hi"], c["Hq"], c["H"], c["d"]
    G, scale = Hq // H, c["d"] ** -0.5
    q, k, v = (_pad(st[n], st, T) for n in "qkv")
    group = lambda x: x.reshape(N, H, G * T, d)                                         # noqa: E731
    s = (group(q) @ k.transpose(-1, -2)).view(N, H, G, T, T).mul_(scale)
    back = torch.arange(T, device="cuda")[:, None] - torch.arange(T, device="cuda")
    hidden = back < 0
    if c["window"]:
        hidden |= back >= c["window"]
    s.masked_fill_(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    tot = p.sum(-1, keepdim=True)
    p = p.div_(tot).view(N, H, G * T, T)
    o = p @ v
    lse = (top + tot.log()).view(N, Hq, T, 1)
    out = dict(o=_unpad(o.view(N, Hq, T, d), st["q"], st), lse=_unpad(lse, st["q"].new_empty(*st["q"].shape[:2], 1, 1, dtype=torch.float32), st)[..., 0])
    if not c["train"]:
        return out
    dO = group(_pad(st["dO"], st, T))
    dv = p.transpose(-1, -2) @ dO
    ds = dO @ v.transpose(-1, -2)
    ds.sub_((dO * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    out["dq"] = _unpad((ds @ k).view(N, Hq, T, d), st["q"], st)
    out["dk"] = _unpad(ds.transpose(-1, -2) @ group(q), st["k"], st)
    out["dv"] = _unpad(dv, st["k"], st)
    return out


def _decays(g, n):
    """e^{g (i - j)} for i >= j, else 0: [H, n, n]."""
    back = torch.arange(n, device=g.device)[:, None] - torch.arange(n, device=g.device)
    return torch.exp(g.double()[:, None, None] * back.clamp(min=0)).tril().float()


def _chunked(q, k, v, g):
    """o_t = S_t^T q_t, S_t = e^g S_{t-1} + k_t v_t^T from an empty state, over [N, H, T, d] in whole chunks."""
    N, H, T, dk = q.shape
    n, gd = T // CHUNK, g.double()
    q, k, v = (x.reshape(N, H, n, CHUNK, -1) for x in (q, k, v))
    o = ((q @ k.transpose(-1, -2)) * _decays(g, CHUNK)[:, None]) @ v
    i = torch.arange(CHUNK, device=q.device)
    to_end = torch.exp(gd[:, None] * (CHUNK - 1 - i)).float()[:, None, :, None]
    added = ((k * to_end).transpose(-1, -2) @ v).flatten(3)                    # of each chunk: [N, H, n, dk dv]
    # the state at a chunk's start: the sum of what the chunks before it added
    at = torch.arange(n, device=q.device)
    steps = (at[:, None] - 1 - at) * CHUNK
    mix = torch.where(steps >= 0, torch.exp(gd[:, None, None] * steps.clamp(min=0)), 0.0).float()
    from_start = torch.exp(gd[:, None] * (i + 1)).float()[:, None, :, None]
    o = o + from_start * (q @ (mix @ added).unflatten(-1, (dk, -1)))
    return o.reshape(N, H, T, -1)


def _plain_lin(st):
    c = st["case"]
    g, scale = st["g"], c["dk"] ** -0.5
    T = -(-max(1, c["hi"]) // CHUNK) * CHUNK
    lens = torch.tensor(st["lens"], dtype=torch.float64).cuda()[:, None, None]
    at = torch.arange(T, device="cuda", dtype=torch.float64)
    gd = g.double()[:, None]
    # decays from the first state to each token, from each token to the last state, and over the whole sequence
    up = torch.exp(gd * (at + 1)).float()[..., None]
    down = torch.where(at < lens, torch.exp(gd * (lens - 1 - at).clamp(min=0)), 0.0).float()[..., None]
    whole = torch.exp(gd * lens).float()[..., None]
    q, k, v = (_pad(st[n], st, T) for n in "qkv")
    o = _chunked(q, k, v, g)
    if c["state"]:
        o = o + up * (q @ st["h0"])
    out = dict(o=_unpad(o * scale, st["v"], st))
    if c["state"] or not c["train"]:
        hT = (k * down).transpose(-1, -2) @ v
        out["hT"] = hT + whole * st["h0"] if c["state"] else hT
    if not c["train"]:
        return out
    dO = _pad(st["dO"], st, T) * scale
    dq = _chunked(dO, v, k, g)
    dk = _chunked(v.flip(2), dO.flip(2), q.flip(2), g).flip(2)
    dv = _chunked(k.flip(2), q.flip(2), dO.flip(2), g).flip(2)
    if c["state"]:
        dq = dq + up * (dO @ st["h0"].transpose(-1, -2))
        dk = dk + down * (v @ st["dhT"].transpose(-1, -2))
        dv = dv + down * (k @ st["dhT"])
        out["dh0"] = (q * up).transpose(-1, -2) @ dO + whole * st["dhT"]
    return out | dict(dq=_unpad(dq, st["q"], st), dk=_unpad(dk, st["q"], st), dv=_unpad(dv, st["v"], st))


def _plain_step(st):
    """All T tokens at once, from the state before them."""
    c = st["case"]
    T, g = c["T"], st["g"].double()
    q, k, v = (st[n].float().transpose(1, 2) for n in "qkv")                   # [B, H, T, d]
    i = torch.arange(T, device="cuda")
    up = torch.exp(g[:, None] * (i + 1)).float()[..., None]
    down = torch.exp(g[:, None] * (T - 1 - i)).float()[..., None]
    o = ((q @ k.transpose(-1, -2)) * _decays(st["g"], T)) @ v + up * (q @ st["state"])
    st["state"].mul_(torch.exp(g * T).float()[:, None, None]).add_((k * down).transpose(-1, -2) @ v)
    return dict(o=(o * c["dk"] ** -0.5).transpose(1, 2).to(st["v"].dtype), state=st["state"])


def run(state):
    c = state["case"]
    if not own:
        return {"attn": _plain_attn, "lin": _plain_lin, "step": _plain_step}[c["op"]](state)
    plan = state["plan"]
    if c["op"] == "step":
        o = plan.step(state["q"], state["k"], state["v"], state["g"], state["state"])
        return dict(o=o, state=state["state"])
    a = [state[n] for n in "qkv"]
    if c["op"] == "attn":
        o, lse = plan.forward(*a, cu=state["cu"], want_lse=True)
        out = dict(o=o, lse=lse)
        if c["train"]:
            out |= plan.backward(*a, o, lse, state["dO"], cu=state["cu"])
        return out
    o, hT = plan.forward(*a, state["g"], h0=state["h0"], cu=state["cu"], want_hT=c["state"] or not c["train"])
    out = dict(o=o)
    if hT is not None:
        out["hT"] = hT
    if c["train"]:
        grads = plan.backward(*a, state["g"], state["dO"], h0=state["h0"], dhT=state["dhT"], cu=state["cu"])
        out |= {n: x for n, x in grads.items() if x is not None}
    return out


# ------------------------------------------------------------------------------- work
def work(case):
    c = case
    io = 2 if c["io"] == "bf16" else 4
    if c["op"] == "step":
        states, tokens = c["N"] * c["H"] * c["dk"] * c["dv"], c["N"] * c["T"] * c["H"]
        return dict(bytes=8 * states + tokens * 2 * (c["dk"] + c["dv"]) * io, flops=4 * c["T"] * states)
    lens = _lens(c)
    total = sum(lens)
    if c["op"] == "attn":
        w, heads = c["window"], 2 * c["Hq"] + 2 * c["H"]
        pairs = sum(n * (n + 1) // 2 - (max(0, n - w) * (max(0, n - w) + 1) // 2 if w else 0) for n in lens)
        values = heads + (2 * c["Hq"] + 2 * c["H"] if c["train"] else 0)
        return dict(bytes=total * (values * c["d"] * io + 4 * c["Hq"]), flops=(14 if c["train"] else 4) * c["d"] * c["Hq"] * pairs)
    dk, dv = c["dk"], c["dv"]
    states = c["N"] * ((2 if c["state"] else 0) * (2 if c["train"] else 1) + (0 if c["state"] or c["train"] else 1))
    values = 2 * (dk + dv) + (2 * dk + 2 * dv if c["train"] else 0)
    return dict(bytes=c["H"] * (total * values * io + states * dk * dv * 4),
                flops=(12 if c["train"] else 4) * total * c["H"] * dk * dv)


# ------------------------------------------------------------------------------- 64 bits
def _ranges(st):
    """(batch index, first token, end, sequence) of every sequence with tokens."""
    first = 0
    for s, n in enumerate(st["lens"]):
        if st["case"]["packed"]:
            if n:
                yield 0, first, first + n, s
            first += n
        else:
            yield s, 0, n, s


def _exact_attn(st):
    """Head by head, the softmax and its gradient by the definition."""
    c = st["case"]
    G, w = c["Hq"] // c["H"], c["window"]
    f64 = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")     # noqa: E731
    out = dict(o=f64(st["q"]), lse=f64(st["q"][..., 0]))
    if c["train"]:
        out |= dict(dq=f64(st["q"]), dk=f64(st["k"]), dv=f64(st["v"]))
    for b, lo, hi, _ in _ranges(st):
        at = torch.arange(hi - lo, device="cuda")
        for h in range(c["Hq"]):
            q, k, v = st["q"][b, lo:hi, h].double(), st["k"][b, lo:hi, h // G].double(), st["v"][b, lo:hi, h // G].double()
            s = q @ k.T / math.sqrt(c["d"])
            s[at[None] > at[:, None]] = -math.inf
            if w:
                s[at[None] + w <= at[:, None]] = -math.inf
            lse = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[:, None])
            out["o"][b, lo:hi, h], out["lse"][b, lo:hi, h] = p @ v, lse
            if c["train"]:
                dO = st["dO"][b, lo:hi, h].double()
                dp = dO @ v.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(c["d"])
                out["dq"][b, lo:hi, h] = ds @ k
                out["dk"][b, lo:hi, h // G] += ds.T @ q
                out["dv"][b, lo:hi, h // G] += p.T @ dO
    return out


def _exact_lin(st):
    """Head by head in the quadratic form: every pair of tokens with its decay."""
    c = st["case"]
    scale, train = c["dk"] ** -0.5, c["train"]
    f64 = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")     # noqa: E731
    like = torch.zeros(c["N"], c["H"], c["dk"], c["dv"], device="cuda")
    out = dict(o=f64(st["v"]))
    if c["state"] or not train:
        out["hT"] = f64(like) if st["h0"] is None else st["h0"].double()
    if train:
        out |= dict(dq=f64(st["q"]), dk=f64(st["k"]), dv=f64(st["v"]))
        if c["state"]:
            out["dh0"] = st["dhT"].double()
    for b, lo, hi, s in _ranges(st):
        at = torch.arange(hi - lo, device="cuda", dtype=torch.float64)
        for h in range(c["H"]):
            q, k, v = (st[n][b, lo:hi, h].double() for n in "qkv")
            a = torch.exp(st["g"][h].double())
            far = torch.where(at[:, None] >= at, a ** (at[:, None] - at).clamp(min=0), 0.0)
            w = scale * (q @ k.T) * far
            o = w @ v
            first, last = (a ** (at + 1))[:, None], (a ** (hi - lo - 1 - at))[:, None]
            if c["state"]:
                h0 = st["h0"][s, h].double()
                o += scale * first * (q @ h0)
            out["o"][b, lo:hi, h] = o
            if "hT" in out:
                out["hT"][s, h] = a ** (hi - lo) * out["hT"][s, h] + (last * k).T @ v
            if not train:
                continue
            dO = st["dO"][b, lo:hi, h].double()
            m = scale * (dO @ v.T) * far
            dq, dk, dv = m @ k, m.T @ q, w.T @ dO
            if c["state"]:
                dhT = st["dhT"][s, h].double()
                dq += scale * first * (dO @ h0.T)
                dk += last * (v @ dhT.T)
                dv += last * (k @ dhT)
                out["dh0"][s, h] = a ** (hi - lo) * dhT + scale * (first * q).T @ dO
            out["dq"][b, lo:hi, h], out["dk"][b, lo:hi, h], out["dv"][b, lo:hi, h] = dq, dk, dv
    return out


def _exact_step(st):
    """Token by token."""
    c = st["case"]
    S, a = st["state"].double(), torch.exp(st["g"].double())[:, None, None]
    o = torch.zeros(st["v"].shape, dtype=torch.float64, device="cuda")
    for t in range(c["T"]):
        S = a * S + st["k"][:, t].double()[..., None] * st["v"][:, t].double()[..., None, :]
        o[:, t] = torch.einsum("bhkv,bhk->bhv", S, st["q"][:, t].double()) / math.sqrt(c["dk"])
    return dict(o=o, state=S)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"attn": _exact_attn, "lin": _exact_lin, "step": _exact_step}[case["op"]](st)
