"""A small hybrid stack: delta-rule layers with a softmax-attention layer among them, run over a
prompt and then token by token, with random weights.

It shows the library's calls as a serving program makes them.  A delta-rule layer keeps one fp32
state for each sequence and head (dr_fwd for the prompt, dr_decode for a step).  The attention layer
norms and rotates its queries and keys (dr_norm_rope_fwd), appends keys and values to the paged
8-bit cache (dr_cache_write) and attends over it (dr_cache_attn); prompt and step are the same three
calls.  The projections are plain matrix products of torch.

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


class HybridStack:
    """`layers` delta-rule layers with an attention layer after every third one."""

    def __init__(self, B=2, layers=4, hidden=256, Hq=4, H=2, d=64, max_len=1024, seed=0, device="cuda", **attention):
        gen = torch.Generator().manual_seed(seed)
        self.layers = []
        for i in range(layers):
            if i % 4 == 3:
                self.layers.append(AttentionLayer(hidden, Hq, H, d, B, max_len, gen, device, **attention))
            else:
                self.layers.append(DeltaLayer(hidden, Hq, d, B, gen, device))

    def __call__(self, x):
        """x [B, T, hidden] bf16, the next T tokens of every sequence."""
        for layer in self.layers:
            x = layer(x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype))
        return x

    def status(self):
        return max(layer.cache.status() for layer in self.layers if isinstance(layer, AttentionLayer))


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
