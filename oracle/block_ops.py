"""Float64 CPU oracle of the operators around the layer: layer norm, the
balance loss over sequences, and the AdamW step.

TEST INFRASTRUCTURE, like ``moe_oracle``: only ``tests/`` may import it.  The
formulas are those stated in ``include/moe.h``; the gradients here are pinned
by finite differences of the forwards here (tests/test_oracle_block_pins.py).
"""
from __future__ import annotations

import numpy as np

BLOCK = 256


# ------------------------------------------------------------------ layer norm
def layer_norm(h, gamma=None, beta=None, eps=1e-5):
    """y, mean, rstd of the rows of h (float64)."""
    mu = h.mean(1)
    c = h - mu[:, None]
    r = 1.0 / np.sqrt((c * c).mean(1) + eps)
    y = c * r[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mu, r


def layer_norm_backward(dy, h, mean, rstd, gamma=None, dsum=None):
    """dh, dgamma, dbeta for the given row statistics."""
    xh = (h - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    dh = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    if dsum is not None:
        dh = dh + dsum
    return dh, (dy * xh).sum(0), dy.sum(0)


# ---------------------------------------------------------------- balance loss
def probabilities(z, score="softmax"):
    """p[T, E]; a row of -inf alone has none (zeros)."""
    with np.errstate(invalid="ignore", over="ignore"):
        empty = (z == -np.inf).all(1)
        zs = np.where(empty[:, None], 0.0, z)
        if score == "softmax":
            e = np.exp(zs - zs.max(1, keepdims=True))
        else:   # sigmoid(z) up to a common factor of the row, which its sum takes out
            m = np.minimum(zs.max(1, keepdims=True), 0.0)
            e = np.exp(np.minimum(zs, 0.0) - m) / (1.0 + np.exp(-np.abs(zs)))
        p = e / e.sum(1, keepdims=True)
    return np.where(empty[:, None], 0.0, p)


def balance(z, topk, k, E, offsets=None, mask=None, score="softmax", coef=1.0, counts=None):
    """loss, counts[S, E], coef * dloss/dz."""
    T = z.shape[0]
    offsets = np.array([0, T]) if offsets is None else np.asarray(offsets)
    S = len(offsets) - 1
    keep = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    toks = [np.arange(offsets[s], offsets[s + 1])[keep[offsets[s]:offsets[s + 1]]] for s in range(S)]
    if counts is None:
        counts = np.zeros((S, E), np.int64)
        for s, u in enumerate(toks):
            i = np.asarray(topk)[u].reshape(-1)
            counts[s] = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
    G = sum(len(u) > 0 for u in toks)
    loss, dz = 0.0, np.zeros((T, E))
    for s, u in enumerate(toks):
        if len(u) == 0:
            continue
        tot = counts[s].sum()
        f = E * counts[s] / tot if tot else np.zeros(E)
        p = probabilities(z[u], score)
        dot = p @ f
        w = 1.0 / (G * len(u))
        loss += w * dot.sum()
        g = p * (f - dot[:, None])
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                g = g / (1.0 + np.exp(z[u]))
        dz[u] = coef * w * g
    return loss, counts, dz


# ----------------------------------------------------------------------- AdamW
def e4m3_table():
    """Values of the 127 non-negative finite E4M3 codes, ascending (code = index)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def e4m3_encode(x):
    """Nearest E4M3 code, ties to even, saturating at 448; NaN for what is not finite."""
    tab = e4m3_table()
    x = np.asarray(x, np.float64)
    a = np.minimum(np.where(np.isfinite(x), np.abs(x), 0.0), 448.0)
    hi = np.clip(np.searchsorted(tab, a), 1, 126)
    lo = hi - 1
    dl, dh = a - tab[lo], tab[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    c = np.where(a == 0, 0, c)
    c = np.where(np.signbit(x), c | 0x80, c).astype(np.uint8)
    return np.where(np.isfinite(x), c, 0x7F).astype(np.uint8)


def e4m3_decode(c):
    c = np.asarray(c, np.uint8)
    v = np.append(e4m3_table(), np.nan)[c & 0x7F]
    return np.where(c & 0x80, -v, v)


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def decode_state(codes, scale):
    return e4m3_decode(codes) * np.repeat(scale, BLOCK)[: len(codes)]


def encode_state(x, root, f32=np.float32):
    """codes, scale of an 8-bit state, in the fp32 steps of the definition when f32 is np.float32."""
    n = len(x)
    with np.errstate(invalid="ignore", over="ignore"):
        xp = np.zeros(blocks(n) * BLOCK, f32)
        xp[:n] = x
        b = xp.reshape(-1, BLOCK)
        top = np.maximum(np.where(np.isfinite(b), np.abs(b), 0).max(1), f32(2.0 ** -100)).astype(f32)
        q = (b * ((f32(1) / top).astype(f32) * f32(448)).astype(f32)[:, None]).astype(f32)
        c = e4m3_encode(np.where(np.isfinite(b), np.clip(q, -448, 448), np.nan))
        if root:
            c = np.where((b > 0) & (c == 0), np.uint8(1), c)
    return c.reshape(-1)[:n], (top * f32(1.0 / 448.0)).astype(f32)


def adamw(p, g, m, v, t, lr, beta1, beta2, eps, decay):
    """p, m, v after step number t (float64 arrays)."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    c1, c2 = 1 - beta1 ** t, 1 - beta2 ** t
    return p * (1 - lr * decay) - lr * (m / c1) / (np.sqrt(v / c2) + eps), m, v


def adamw_f32_moments(g, m, v, beta1, beta2):
    """m and v in the separately rounded fp32 steps that the 8-bit codes are taken from."""
    f = np.float32
    with np.errstate(invalid="ignore", over="ignore"):
        m = (m * f(beta1) + (g * f(1 - beta1)).astype(f)).astype(f)
        v = (v * f(beta2) + ((g * g).astype(f) * f(1 - beta2)).astype(f)).astype(f)
    return m, v
