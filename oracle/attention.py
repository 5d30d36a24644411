"""fp64 restatement (numpy) of the softmax-attention layer's operators: the norm of queries and
keys for each head with the position rotation and its gradient, the paged 8-bit cache, and the
attention over it.  Written from the definitions, token by token; test infrastructure only.

The cache's arithmetic is fp32 by definition (each quotient and product rounded), so codes and
scales are restated in numpy float32 and have to agree bit for bit."""
from __future__ import annotations

import numpy as np

CODE_MAX = {"i8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ norm and rotation
def pair_index(rot, style):
    """Channels (i, j) of every pair."""
    if style == "halves":
        i = np.arange(rot // 2)
        return i, i + rot // 2
    i = np.arange(0, rot, 2)
    return i, i + 1


def norm_rope(x, w, cos, sin, pos, rot, style, eps):
    """x [B, T, H, d] -> y; pos [B, T]: rows of cos, sin."""
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n = x * r * (1.0 if w is None else np.asarray(w, np.float64))
    y = n.copy()
    if rot:
        i, j = pair_index(rot, style)
        c, s = (np.asarray(t, np.float64)[pos][:, :, None] for t in (cos, sin))
        y[..., i] = n[..., i] * c - n[..., j] * s
        y[..., j] = n[..., j] * c + n[..., i] * s
    return y


def norm_rope_grad(x, w, cos, sin, pos, rot, style, eps, dy):
    """(dx, dw) of L = sum(dy * y)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    d = x.shape[-1]
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    dn = dy.copy()
    if rot:
        i, j = pair_index(rot, style)
        c, s = (np.asarray(t, np.float64)[pos][:, :, None] for t in (cos, sin))
        dn[..., i] = dy[..., i] * c + dy[..., j] * s
        dn[..., j] = dy[..., j] * c - dy[..., i] * s
    dw = np.sum(dn * x * r, axis=(0, 1, 2))
    dxr = dn * (1.0 if w is None else np.asarray(w, np.float64))
    # x r: d r / d x_c = -r^3 x_c / d
    dx = dxr * r - x * r ** 3 * np.sum(dxr * x, axis=-1, keepdims=True) / d
    return dx, dw


# ------------------------------------------------------------------ codes
def e4m3_value(byte):
    """The value of e4m3 bytes (NaN for the two NaN codes)."""
    b = np.asarray(byte, np.uint8).astype(np.int64)
    sign = np.where(b & 0x80, -1.0, 1.0)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    return np.where((b & 0x7f) == 0x7f, np.nan, sign * v)


_GRID = e4m3_value(np.arange(0x7f))  # the non-negative values, by code


def to_code(x, code):
    """Bytes of the nearest codes of x (finite), ties to even."""
    x = np.asarray(x, np.float64)
    if code == "i8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_GRID, a), 1, 0x7e)
    lo = hi - 1
    up, down = _GRID[hi] - a, a - _GRID[lo]
    even_hi = hi % 2 == 0
    pick = np.where((up < down) | ((up == down) & even_hi), hi, lo)
    return (pick | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def code_value(byte, code):
    return np.asarray(byte, np.uint8).view(np.int8).astype(np.float64) if code == "i8" else e4m3_value(byte)


# ------------------------------------------------------------------ the cache
def cache_write(codes, scale, x, table, lens, counts, code):
    """Appends x [B, T, H, d] (float32 values) to codes [P, H, page, d] (uint8), scale [P, H] in place."""
    f32 = np.float32
    page = codes.shape[2]
    inv = f32(1.0) / f32(CODE_MAX[code])
    for b in range(x.shape[0]):
        p, end = int(lens[b]), int(lens[b] + counts[b])
        while p < end:
            stop, row, i = min(end, (p // page + 1) * page), p % page, table[b][p // page]
            for h in range(x.shape[2]):
                new = x[b, p - lens[b]:stop - lens[b], h].astype(f32)
                s_old = scale[i, h] if row else f32(0)
                if np.isfinite(new).all() and np.isfinite(s_old):
                    s = max(s_old, f32(np.abs(new).max() * inv))
                else:
                    s = f32(np.nan)
                if s > 0:
                    codes[i, h, row:row + stop - p] = to_code((new / s).astype(f32), code)
                else:
                    codes[i, h, row:row + stop - p] = 0
                if s > s_old > 0:
                    was = code_value(codes[i, h, :row], code).astype(f32)
                    codes[i, h, :row] = to_code(((was * s_old).astype(f32) / s).astype(f32), code)
                scale[i, h] = s
            p = stop


def cache_values(codes, scale, table_row, n, code):
    """Values [n, H, d] of a sequence's first n positions."""
    page = codes.shape[2]
    out = np.zeros((n, codes.shape[1], codes.shape[3]))
    for i in range(-(-n // page)):
        pg = table_row[i]
        m = min(page, n - i * page)
        v = code_value(codes[pg, :, :m], code) * scale[pg].astype(np.float64)[:, None, None]
        out[i * page:i * page + m] = v.transpose(1, 0, 2)
    return out


# ------------------------------------------------------------------ attention
def attention(q, k_codes, k_scale, v_codes, v_scale, table, lens, counts, code, scale, window):
    """o, lse and, for error bounds, mean |v| under the weights, the largest scale sum |q k|, and the
    largest weight times value scale times the sum of |codes|."""
    B, T, Hq, d = q.shape
    H = k_codes.shape[1]
    G = Hq // H
    o, lse = np.zeros((B, T, Hq, d)), np.full((B, T, Hq), -np.inf)
    mag, top, floor = np.zeros((B, T, Hq, d)), np.zeros((B, T, Hq)), np.zeros((B, T, Hq, d))
    for b in range(B):
        n = int(lens[b] + counts[b])
        if counts[b] == 0:
            continue
        k = cache_values(k_codes, k_scale, table[b], n, code)
        v = cache_values(v_codes, v_scale, table[b], n, code)
        c = np.abs(cache_values(v_codes, np.ones_like(v_scale), table[b], n, code))
        vs = v_scale[table[b][np.arange(n) // k_codes.shape[2]]].astype(np.float64)
        for t in range(int(counts[b])):
            p = int(lens[b]) + t
            lo = max(0, p - window + 1) if window else 0
            for h in range(Hq):
                qr = q[b, t, h].astype(np.float64)
                kk, vv = k[lo:p + 1, h // G], v[lo:p + 1, h // G]
                s = scale * (kk @ qr)
                m = s.max()
                e = np.exp(s - m)
                o[b, t, h] = e @ vv / e.sum()
                lse[b, t, h] = m + np.log(e.sum())
                mag[b, t, h] = e @ np.abs(vv) / e.sum()
                top[b, t, h] = abs(scale) * (np.abs(kk) @ np.abs(qr)).max()
                floor[b, t, h] = (e * vs[lo:p + 1, h // G]).max() / e.sum() * c[lo:p + 1, h // G].sum(0)
    return o, lse, mag, top, floor
