"""Oracle of the router's losses and of the update by Newton-Schulz products:
numpy, float64, from the formulas; shares no code with the library.

`newton_model` repeats the documented arithmetic of the products (fp16 factors,
float32 sums) in numpy, so a test can hold the kernels against what that
arithmetic itself loses."""
from __future__ import annotations

import numpy as np

COEF = ((3.4445, -4.7750, 2.0315),) * 5


def softmax_rows(logits):
    """(p, lse) in float64."""
    l = np.asarray(logits, np.float64)
    top = l.max(1, keepdims=True)
    z = np.exp(l - top)
    s = z.sum(1, keepdims=True)
    return z / s, (top + np.log(s))[:, 0]


def balance(logits, topk_idx, mask, seq_len, E, K):
    """dict(loss, counts, tokens, probs) as documented in moe_train.h."""
    T = len(logits)
    S = -(-T // seq_len)
    counts, probs, n = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    zsum = 0.0
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        s = t // seq_len
        p, lse = softmax_rows(logits[t:t + 1])
        n[s] += 1
        probs[s] += p[0]
        zsum += lse[0] ** 2
        for e in topk_idx[t]:
            if 0 <= e < E:
                counts[s, e] += 1
    some = int((n > 0).sum())
    loss0 = sum(E / (K * n[s] ** 2) * float((counts[s] * probs[s]).sum()) for s in range(S) if n[s]) / max(some, 1)
    loss1 = zsum / max(int(n.sum()), 1)
    return dict(loss=np.array([loss0, loss1]), counts=counts, tokens=np.concatenate([n, [n.sum(), some]]), probs=probs)


def balance_bwd(logits, mask, seq_len, E, K, counts, tokens, dloss, route=None):
    """dlogits [T, E]; route: (dtopk_w, topk_w, topk_idx) or None."""
    T = len(logits)
    d = np.zeros((T, E))
    for t in range(T):
        if mask is None or mask[t]:
            s = t // seq_len
            p, lse = softmax_rows(logits[t:t + 1])
            p = p[0]
            q = dloss[0] * E / (K * float(tokens[s]) ** 2 * tokens[-1]) * counts[s]
            d[t] = p * (q - (p * q).sum() + dloss[1] * 2 / tokens[-2] * lse[0])
        if route is not None:
            dw, w, idx = (a[t] for a in route)
            inner = float((np.asarray(w, np.float64) * dw).sum())
            for k, e in enumerate(idx):
                if 0 <= e < E:
                    d[t, e] += float(w[k]) * (float(dw[k]) - inner)
    return d


def newton(u, coef=COEF):
    """The iteration on one matrix, float64."""
    x = np.asarray(u, np.float64)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    norm = np.sqrt((x * x).sum())
    x = x / norm if norm > 0 else x
    for a, b, c in coef:
        g = x @ x.T
        x = a * x + (b * g + c * g @ g) @ x
    return x.T if tall else x


def _half(v, scale):
    return (v * np.float32(scale)).astype(np.float16).astype(np.float32) / np.float32(scale)


def _parts(v, scale):
    h = _half(v, scale)
    return h, _half(v - h, scale)


def _chain(p, q):
    """p @ q in float32, summed 16 terms at a time in ascending order as a matrix instruction does: the
    roundings of a long chain are part of the arithmetic (a blocked sum would have fewer)."""
    out = np.zeros((p.shape[0], q.shape[1]), np.float32)
    for k in range(0, p.shape[1], 16):
        out += p[:, k:k + 16] @ q[k:k + 16]
    return out


def newton_model(u, exact, coef=COEF):
    """The iteration as the products round it.  X has two fp16 parts, of which the lower one is dropped from
    the step on whose |a|, with those of the later steps, make at most 12 (never in the exact form, always
    for the last step otherwise).  a is part of B's diagonal; a times the lower part is added.  Factors have one
    part (exact: two).  A and B are stored times 256, the last step's B, which may be of any size, times a power of two
    that keeps it inside fp16."""
    x = np.asarray(u, np.float64)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    norm = np.sqrt((x * x).sum())
    x = (x / norm if norm > 0 else x).astype(np.float32)

    def mul(p, q):
        if exact:
            return _chain(np.concatenate([p[1], p[0], p[0]], 1), np.concatenate([q[0], q[1], q[0]], 0))
        return _chain(p[0], q[0])
    f = np.float32
    for k, (a, b, c) in enumerate(coef):
        low = exact or (k + 1 < len(coef) and np.prod([max(1.0, abs(s[0])) for s in coef[k:]]) > 12)
        xs = _parts(x, 1024) if low else (_half(x, 1024), np.zeros_like(x))
        A = _parts(mul(xs, (xs[0].T, xs[1].T)), 256)
        whole = A[0] + A[1] if exact else A[0]
        B = f(b) * whole + f(c) * mul(A, A) + f(a) * np.eye(len(A[0]), dtype=f)
        scale = 256.0
        while k + 1 == len(coef) and np.isfinite(B).all() and np.abs(B).max() * scale > 32768:
            scale /= 2
        x = mul(_parts(B, scale), xs)
        if low and not exact:
            x = f(a) * xs[1] + x
    return x.T if tall else x


def muon(grad, mom, master, lr, momentum, weight_decay, scale, nesterov, coef=COEF):
    """(mom, master, update O) of one step on a stack [G, R, C], float64."""
    grad = np.asarray(grad, np.float64)
    mom = momentum * np.asarray(mom, np.float64) + grad
    u = grad + momentum * mom if nesterov else mom
    o = np.stack([newton(x, coef) for x in u])
    return mom, (1 - lr * weight_decay) * np.asarray(master, np.float64) - lr * scale * o, o
