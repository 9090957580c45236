"""Float64 oracle of the layer for a few tokens and of the MXFP4 weight form,
with the error bounds the GPU results are held to -- test infrastructure only.

The layer (UniEP article, section 1.1): top-k, SwiGLU expert FFN, weighted
sum; unlike the staged oracle nothing is rounded between logits and out.
MXFP4 (OCP Microscaling): 32 weights along the reduction dim share a power of
two, codes are E2M1.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import route_select, route_weights, widen

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EPS = 2.0 ** -23        # one float32 operation (an addition inside a matrix instruction may truncate)


def _ffn(x, w1, w3, w2, parts_err):
    """y of rows x and a bound on a float32 kernel's distance from it.

    a and b are sums of H products: each of the H additions (and as many again
    inside the reduction over waves, far fewer) is off by at most EPS of the
    partial sum, which |x| @ |W| bounds.  |silu'| <= 1.1.  h loses parts_err of
    itself where it is split for the second product, and 2^-20 in exp and the
    division.  y adds its own I additions."""
    H, I = w1.shape
    a, b = x @ w1, x @ w3
    ea, eb = (H + 16) * EPS * (np.abs(x) @ np.abs(w1)), (H + 16) * EPS * (np.abs(x) @ np.abs(w3))
    s = a / (1.0 + np.exp(-a))
    h = s * b
    eh = 1.1 * ea * (np.abs(b) + eb) + np.abs(s) * eb + (parts_err + 2.0 ** -20) * np.abs(h)
    y = h @ w2
    return y, (eh + (I + 32) * EPS * (np.abs(h) + eh)) @ np.abs(w2)


def decode(inp: dict, K: int, dtype: str, weights: dict | None = None, n_tokens: int | None = None):
    """topk_idx, topk_w (float64), out (float64) and the bound on |out_gpu - out|
    of the rows in use.  weights: float64 matrices in place of inp's."""
    logits, x = inp["logits"], widen(inp["x"], dtype).astype(np.float64)
    n = logits.shape[0] if n_tokens is None else n_tokens
    w = weights or {k: widen(inp[k], dtype).astype(np.float64) for k in
                    ("w1", "w3", "w2", "ws1", "ws3", "ws2") if k in inp}
    idx = route_select(logits[:n], K)
    g = np.asarray(route_weights(logits[:n].astype(np.float64), idx), np.float64)
    # bf16 rows: h goes into the second product as two bf16 parts, 2^-8 of 2^-8; float32 rows: whole
    parts_err = 2.0 ** -16 if dtype == "bf16" else 2.0 ** -23
    out, err = np.zeros((n, x.shape[1])), np.zeros((n, x.shape[1]))
    mag = np.zeros_like(out)
    for e in np.unique(idx) if n else []:
        t, k = np.nonzero(idx == e)
        y, ey = _ffn(x[t], w["w1"][e], w["w3"][e], w["w2"][e], parts_err)
        out[t] += g[t, k, None] * y
        # g: exp and a division, 2^-20 of it
        err[t] += g[t, k, None] * (ey * (1 + 2.0 ** -20) + 2.0 ** -20 * np.abs(y))
        mag[t] += np.abs(g[t, k, None] * y) + g[t, k, None] * ey
    for s in range(w["ws1"].shape[0] if "ws1" in w and n else 0):
        y, ey = _ffn(x[:n], w["ws1"][s], w["ws3"][s], w["ws2"][s], parts_err)
        out += y
        err += ey
        mag += np.abs(y) + ey
    err += (K + 16) * EPS * mag
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24      # the final rounding, half a step
    return {"topk_idx": idx, "topk_w": g, "out": out, "bound": err + half * (np.abs(out) + err) + 1e-38}


def mx_quantize(w: np.ndarray):
    """Codes [G, K/32, 32, N] (0..15) and scale exponents [G, K/32, N] of w [G, K, N]."""
    G, K, N = w.shape
    g = w.astype(np.float64).reshape(G, K // 32, 32, N)
    big = np.abs(g).max(2)
    _, e = np.frexp(big)                                   # big = m 2^e, m in [0.5, 1)
    s = np.where(big > 0, np.maximum(e - 1 - 2, -126), -126)
    v = np.abs(g) / np.exp2(s.astype(np.float64))[:, :, None]
    d = np.abs(v[..., None] - MAGNITUDES)
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])             # even codes win ties
    code = order[np.argmin(d[..., order], -1)]
    return (code + 8 * np.signbit(g)).astype(np.uint8), s.astype(np.int64)


def mx_pack(code: np.ndarray, s: np.ndarray) -> np.ndarray:
    """The packed bytes: codes [G, K/32, N, 16], then scales [G, K/32, N]."""
    c = np.moveaxis(code, 2, 3)
    return np.concatenate([(c[..., 0::2] | (c[..., 1::2] << 4)).ravel(), (s + 127).astype(np.uint8).ravel()])


def mx_values(code: np.ndarray, s: np.ndarray) -> np.ndarray:
    """Float64 matrices [G, K, N]."""
    v = np.where(code >= 8, -1.0, 1.0) * MAGNITUDES[code & 7] * np.exp2(s.astype(np.float64))[:, :, None]
    return v.reshape(v.shape[0], -1, v.shape[3])
