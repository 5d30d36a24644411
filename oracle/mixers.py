"""fp64 restatement (numpy) of the token mixers beside the delta rule: causal softmax attention over whole
prompts and linear attention with a decay for each head, with their gradients.  Written from the definitions,
one sequence and head at a time; test infrastructure only.

Every function also returns, under the same names, the sums of the sizes of the terms of each result: what
rounding errors are measured against."""
from __future__ import annotations

import numpy as np


def attention(q, k, v, spans, scale, window, dO=None):
    """q [T, Hq, d], k, v [T, H, d]; spans: (first row, end) of every sequence.  ({o, lse, dq, dk, dv}, sizes)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    Hq, H, d = q.shape[1], k.shape[1], q.shape[2]
    out = dict(o=np.zeros(q.shape), lse=np.zeros(q.shape[:2]))
    if dO is not None:
        dO = np.asarray(dO, np.float64)
        out |= dict(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape))
    size = {n: np.zeros(x.shape) for n, x in out.items()}
    for lo, hi in spans:
        at = np.arange(hi - lo)
        see = at[None] <= at[:, None]
        if window:
            see &= at[None] > at[:, None] - window
        for h in range(Hq if hi > lo else 0):
            g = h // (Hq // H)
            Q, K, V = q[lo:hi, h], k[lo:hi, g], v[lo:hi, g]
            s = np.where(see, scale * (Q @ K.T), -np.inf)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            p = e / e.sum(1, keepdims=True)
            out["o"][lo:hi, h], out["lse"][lo:hi, h] = p @ V, (m + np.log(e.sum(1, keepdims=True)))[:, 0]
            size["o"][lo:hi, h] = p @ np.abs(V)
            size["lse"][lo:hi, h] = (abs(scale) * (np.abs(Q) @ np.abs(K).T) * see).max(1)
            if dO is None:
                continue
            G = dO[lo:hi, h]
            dp = G @ V.T
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            mag = p * (np.abs(G) @ np.abs(V).T + (np.abs(G) * (p @ np.abs(V))).sum(1, keepdims=True))
            out["dq"][lo:hi, h] = scale * ds @ K
            out["dk"][lo:hi, g] += scale * ds.T @ Q
            out["dv"][lo:hi, g] += p.T @ G
            size["dq"][lo:hi, h] = abs(scale) * mag @ np.abs(K)
            size["dk"][lo:hi, g] += abs(scale) * mag.T @ np.abs(Q)
            size["dv"][lo:hi, g] += p.T @ np.abs(G)
    return out, size


def linear(q, k, v, g, spans, scale, h0=None, dO=None, dhT=None):
    """q, k [T, H, dk], v [T, H, dv], g [H], states [N, H, dk, dv], token by token.  ({o, hT, dq, dk, dv, dh0},
    sizes)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    H, N = q.shape[1], len(spans)
    a = np.exp(np.asarray(g, np.float64))[:, None, None]
    shape = (N, H, q.shape[2], v.shape[2])
    zero = np.zeros(shape)
    h0, dhT = (zero if x is None else np.asarray(x, np.float64) for x in (h0, dhT))
    out = dict(o=np.zeros(v.shape), hT=np.zeros(shape))
    if dO is not None:
        dO = np.asarray(dO, np.float64)
        out |= dict(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape), dh0=np.zeros(shape))
    size = {n: np.zeros(x.shape) for n, x in out.items()}
    for res, f in ((out, lambda x: x), (size, np.abs)):
        for n, (lo, hi) in enumerate(spans):
            S = f(h0[n])
            before = []
            for t in range(lo, hi):
                S = a * S + f(k[t])[:, :, None] * f(v[t])[:, None]
                res["o"][t] = f(np.float64(scale)) * np.einsum("hkv,hk->hv", S, f(q[t]))
                before.append(S)
            res["hT"][n] = S
            if dO is None:
                continue
            R = f(dhT[n])
            for t in range(hi - 1, lo - 1, -1):
                G = f(np.float64(scale)) * f(dO[t])
                res["dq"][t] = np.einsum("hkv,hv->hk", before[t - lo], G)
                R = R + f(q[t])[:, :, None] * G[:, None]
                res["dk"][t] = np.einsum("hkv,hv->hk", R, f(v[t]))
                res["dv"][t] = np.einsum("hkv,hk->hv", R, f(k[t]))
                R = a * R
            res["dh0"][n] = R
    return out, size
