"""A small hybrid stack: delta-rule layers with a softmax-attention layer among them, run over a
prompt and then token by token, with random weights.

It shows the library's calls as a serving program makes them.  A delta-rule layer keeps one fp32
state for each sequence and head (dr_fwd for the prompt, dr_decode for a step), and so does linear
attention with a decay for each head, which may take its place (dr_linear_attn_fwd,
dr_linear_attn_step).  The attention layer norms and rotates its queries and keys (dr_norm_rope_fwd),
appends keys and values to the paged 8-bit cache (dr_cache_write) and attends over it
(dr_cache_attn); prompt and step are the same three calls.  The projections are plain matrix
products of torch.

TrainingStack runs such layers over packed documents and back: the softmax-attention layer as
dr_norm_rope, dr_prompt_attn and their gradients, linear attention as dr_linear_attn.

    python -m delta_rule_recurrent_gated_gb300.hybrid
"""
from __future__ import annotations

import torch

from . import binding


def rotation_table(rows, rot, device, base=10000.0):
    """cos and sin [rows, rot / 2] of the positions' angles."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return ang.cos().float().to(device), ang.sin().float().to(device)


def _weight(gen, rows, cols, device):
    return (torch.randn(rows, cols, generator=gen) / rows ** 0.5).bfloat16().to(device)


class DeltaLayer:
    """Gated DeltaNet with its input preparation inside the library."""

    def __init__(self, hidden, H, d, B, gen, device):
        self.H, self.d, self.B, self.device = H, d, B, device
        self.w_in = _weight(gen, hidden, 3 * H * d, device)
        self.w_gate = _weight(gen, hidden, 2 * H, device)
        self.w_out = _weight(gen, H * d, hidden, device)
        self.state = torch.zeros(B, H, d, d, device=device)
        self.decoder = binding.Decoder("gdn", B, 1, H, d, d, io="bf16", out="bf16", scale=d ** -0.5, prepare=True)

    def __call__(self, x):
        B, T, _ = x.shape
        q, k, v = (t.reshape(B, T, self.H, self.d).contiguous() for t in (x @ self.w_in).chunk(3, -1))
        beta, gate = (t.float().contiguous() for t in (x @ self.w_gate).chunk(2, -1))
        if T == 1:
            o = self.decoder.step(q, k, v, beta, gate, self.state)
        else:
            p = binding.Problem("gdn", B, T, self.H, self.d, self.d, out="bf16", scale=self.d ** -0.5, prepare=True)
            o, self.state = p.forward(q, k, v, beta, gate, self.state)
        return x + o.reshape(B, T, -1) @ self.w_out


def decay_rates(H, device):
    """Log-decays of H heads: memories of 32 tokens for the first, longer and longer ones after it."""
    return torch.log1p(-torch.exp2(-5.0 - 6.0 * torch.arange(H) / max(1, H - 1))).to(device)


class DecayLayer:
    """Linear attention with a fixed decay for each head."""

    def __init__(self, hidden, H, d, B, gen, device):
        self.H, self.d, self.B, self.device = H, d, B, device
        self.w_in = _weight(gen, hidden, 3 * H * d, device)
        self.w_out = _weight(gen, H * d, hidden, device)
        self.g = decay_rates(H, device)
        self.state = torch.zeros(B, H, d, d, device=device)
        self.decoder = binding.LinearAttention(B, 1, H, d, d, scale=d ** -0.5, device=device)

    def __call__(self, x):
        B, T, _ = x.shape
        q, k, v = (x @ self.w_in).reshape(B, T, 3 * self.H, self.d).split(self.H, 2)  # not copied
        if T == 1:
            o = self.decoder.step(q, k, v, self.g, self.state)
        else:
            p = binding.LinearAttention(B, T, self.H, self.d, self.d, scale=self.d ** -0.5, device=self.device,
                                        word=self.decoder.word)
            o, self.state = p.forward(q, k, v, self.g, h0=self.state)
        return x + o.reshape(B, T, -1) @ self.w_out

    def status(self):
        """Of the steps and of all prompts, whose plans end with them."""
        return self.decoder.status()


class AttentionLayer:
    """Softmax attention with norms of queries and keys, rotation, and a paged 8-bit cache."""

    def __init__(self, hidden, Hq, H, d, B, max_len, gen, device, code="i8", page=64, window=0, rot=None):
        self.Hq, self.H, self.d, self.B, self.window = Hq, H, d, B, window
        self.rot = d if rot is None else rot
        self.w_in = _weight(gen, hidden, (Hq + 2 * H) * d, device)
        self.w_out = _weight(gen, Hq * d, hidden, device)
        self.wq, self.wk = (1 + 0.1 * torch.randn(d, generator=gen).to(device) for _ in range(2))
        self.cos, self.sin = rotation_table(max_len, self.rot, device)
        per = -(-max_len // page)
        self.cache = binding.KvCache(B * per, H, d, page=page, code=code, device=device)
        # any assignment of pages will do: here they are shared out in turn
        self.table = torch.arange(B * per, dtype=torch.int32, device=device).reshape(per, B).t().contiguous()
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)
        self.plans = {}

    def _plan(self, T):
        if T not in self.plans:  # descriptors, once for each number of tokens
            self.plans[T] = (binding.HeadNormRope(self.B, T, self.Hq, self.H, self.d, rot=self.rot),
                             binding.CacheAttention(self.cache, self.B, T, self.Hq, window=self.window))
        return self.plans[T]

    def __call__(self, x):
        B, T, _ = x.shape
        norm, attend = self._plan(T)
        qkv = (x @ self.w_in).reshape(B, T, self.Hq + 2 * self.H, self.d)
        q, k, v = qkv.split((self.Hq, self.H, self.H), 2)  # head ranges of the projection, not copied
        q, k = norm.forward(q, k, self.wq, self.wk, self.cos, self.sin, start=self.lens)
        self.cache.write(k, v, self.table, self.lens)
        o, _ = attend.forward(q, self.table, self.lens)
        self.lens += T
        return x + o.reshape(B, T, -1) @ self.w_out

    def status(self):
        return self.cache.status()


class HybridStack:
    """`layers` delta-rule layers (linear="delta") or linear-attention layers ("decay") with an attention layer after
    every third one."""

    def __init__(self, B=2, layers=4, hidden=256, Hq=4, H=2, d=64, max_len=1024, seed=0, device="cuda", linear="delta",
                 **attention):
        gen = torch.Generator().manual_seed(seed)
        self.layers = []
        for i in range(layers):
            if i % 4 == 3:
                self.layers.append(AttentionLayer(hidden, Hq, H, d, B, max_len, gen, device, **attention))
            else:
                self.layers.append({"delta": DeltaLayer, "decay": DecayLayer}[linear](hidden, Hq, d, B, gen, device))

    def __call__(self, x):
        """x [B, T, hidden] bf16, the next T tokens of every sequence."""
        for layer in self.layers:
            x = layer(x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype))
        return x

    def status(self):
        """DR_OK, or what a call of the attention and linear-attention layers left in their status words."""
        return max((layer.status() for layer in self.layers if not isinstance(layer, DeltaLayer)), default=binding.DR_OK)


class _TrainedLayer:
    """x + mix(x w_in) w_out over the rows of packed documents, and back.  `io`: "bf16" or "f32"."""

    def __init__(self, hidden, wide, narrow, gen, device, io):
        kind = torch.bfloat16 if io == "bf16" else torch.float32
        self.w_in, self.w_out = (_weight(gen, *s, device).to(kind) for s in ((hidden, wide), (narrow, hidden)))

    def forward(self, x, cu, positions):
        self.x = x
        self.mixed = self.mix((x @ self.w_in).reshape(1, x.shape[0], -1, self.d), cu, positions).flatten(2)[0]
        return x + self.mixed @ self.w_out

    def backward(self, dy, cu, positions):
        """The gradient of x; those of the weights are left in `grads`."""
        dmixed = (dy @ self.w_out.T).reshape(1, dy.shape[0], -1, self.d)
        self.grads = {"w_out": self.mixed.T @ dy}
        dqkv = self.unmix(dmixed, cu, positions).flatten(2)[0]
        self.grads["w_in"] = self.x.T @ dqkv
        return dy + dqkv @ self.w_in.T


class TrainedAttention(_TrainedLayer):
    """Norm, rotation and causal softmax attention; the gradients of queries, keys and values go into the ranges of one
    tensor, the gradient of the projection."""

    def __init__(self, hidden, Hq, H, d, tokens, docs, gen, device, io="bf16", window=0):
        super().__init__(hidden, (Hq + 2 * H) * d, Hq * d, gen, device, io)
        self.d, self.heads = d, (Hq, H, H)
        self.wq, self.wk = (1 + 0.1 * torch.randn(d, generator=gen).to(device) for _ in range(2))
        self.cos, self.sin = rotation_table(tokens, d, device)
        self.norm = binding.HeadNormRope(1, tokens, Hq, H, d, io=io, out=io, grad=io, device=device)
        self.attend = binding.PromptAttention(1, tokens, Hq, H, d, seqs=docs, io=io, window=window, device=device)

    def mix(self, qkv, cu, positions):
        q, k, v = qkv.split(self.heads, 2)
        self.raw = (q, k, self.wq, self.wk, self.cos, self.sin)
        q, k = self.norm.forward(*self.raw, positions=positions)
        o, lse = self.attend.forward(q, k, v, cu=cu, want_lse=True)
        self.kept = (q, k, v, o, lse)
        return o

    def unmix(self, do, cu, positions):
        tokens = do.shape[1]
        dqkv = torch.zeros(1, tokens, sum(self.heads), self.d, dtype=do.dtype, device=do.device)
        dq, dk, dv = dqkv.split(self.heads, 2)
        g = self.attend.backward(*self.kept, do, cu=cu, out={"dv": dv})
        dw = {n: torch.empty_like(w) for n, w in (("dwq", self.wq), ("dwk", self.wk))}
        self.norm.backward(*self.raw, g["dq"], g["dk"], positions=positions, out={"dq": dq, "dk": dk, **dw})
        self.grads.update(wq=dw["dwq"], wk=dw["dwk"])
        return dqkv

    def status(self):
        return self.attend.status()


class TrainedDecay(_TrainedLayer):
    """Linear attention with a fixed decay for each head."""

    def __init__(self, hidden, H, d, tokens, docs, gen, device, io="bf16"):
        super().__init__(hidden, 3 * H * d, H * d, gen, device, io)
        self.d, self.H, self.g = d, H, decay_rates(H, device)
        self.plan = binding.LinearAttention(1, tokens, H, d, d, seqs=docs, io=io, scale=d ** -0.5, device=device)

    def mix(self, qkv, cu, positions):
        self.kept = (*qkv.split(self.H, 2), self.g)
        return self.plan.forward(*self.kept, cu=cu, want_hT=False)[0]

    def unmix(self, do, cu, positions):
        dqkv = torch.zeros(1, do.shape[1], 3 * self.H, self.d, dtype=do.dtype, device=do.device)
        self.plan.backward(*self.kept, do, cu=cu, out=dict(zip(("dq", "dk", "dv"), dqkv.split(self.H, 2))))
        return dqkv

    def status(self):
        return self.plan.status()


class TrainingStack:
    """Linear-attention layers with a softmax-attention layer after every third one, over `tokens` rows of up to `docs`
    packed documents: cu [docs + 1] int32, every row in one of them."""

    def __init__(self, tokens, docs, layers=4, hidden=256, Hq=4, H=2, d=64, seed=0, device="cuda", io="bf16"):
        gen = torch.Generator().manual_seed(seed)
        self.layers = [TrainedAttention(hidden, Hq, H, d, tokens, docs, gen, device, io) if i % 4 == 3 else
                       TrainedDecay(hidden, Hq, d, tokens, docs, gen, device, io) for i in range(layers)]

    @staticmethod
    def positions(cu, tokens):
        """The place of every row in its document."""
        at = torch.arange(tokens, device=cu.device)
        return (at - cu.long()[torch.searchsorted(cu.long(), at, right=True) - 1]).int()[None]

    def forward(self, x, cu):
        self.cu, self.pos = cu, self.positions(cu, x.shape[0])
        for layer in self.layers:
            x = layer.forward(x, self.cu, self.pos)
        return x

    def backward(self, dy):
        for layer in reversed(self.layers):
            dy = layer.backward(dy, self.cu, self.pos)
        return dy

    def status(self):
        """DR_OK, or DR_ERR_TIMEOUT after a bounded wait of a mixer's kernels ran out: results are then incomplete."""
        return max(layer.status() for layer in self.layers)


def main():
    B, T, steps, hidden = 2, 500, 16, 256
    x = torch.randn(B, T + steps, hidden, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    whole = HybridStack(B)(x)
    stack = HybridStack(B)
    parts = [stack(x[:, :T])] + [stack(x[:, T + i:T + i + 1]) for i in range(steps)]
    diff = (torch.cat(parts, 1) - whole).float()
    print(f"{T} tokens at once and {steps} one by one against {T + steps} at once: "
          f"relative difference {float(diff.norm() / whole.float().norm()):.2e}, status {stack.status()}")


if __name__ == "__main__":
    main()
