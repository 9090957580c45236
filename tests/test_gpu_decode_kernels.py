"""Every product kernel of the layer for a few tokens against float64: the shapes
whose plans reach them, with the bounds of oracle/decode_oracle.py."""
import numpy as np
import pytest
import torch

import combine_moe_route_histogram_amd as M
import decode_kernels as DK
from combine_moe_route_histogram_amd import layer as L
from oracle import decode_oracle as D

pytestmark = pytest.mark.gpu


def _inputs(fmt, shape):
    """Device inputs (weights packed for the 4-bit formats) and their float64 weights, by name and group."""
    T, H, E, K, I, Ns = shape
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    dt = torch.bfloat16 if fmt.startswith("bf16") else torch.float32
    draw = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(dt)
    p = {"logits": torch.randn(T, E, generator=gen, device="cuda"), "x": draw(T, H)}
    for G, pre in ((E, "w"), (Ns, "ws")):
        if G:
            p.update({pre + "1": draw(G, H, I, scale=H ** -0.5), pre + "3": draw(G, H, I, scale=H ** -0.5),
                      pre + "2": draw(G, I, H, scale=I ** -0.5)})
    if not fmt.endswith("mx"):
        return p, lambda name, g: p[name][g].double()
    q = L.quantize_weights(p)
    values = {}
    for name in q:
        if name.startswith("w"):
            values[name] = torch.empty(p[name].shape, device="cuda")
            M.moe_mx_dequantize(*p[name].shape, q[name], values[name])
    return q, lambda name, g: values[name][g].double()


def _reference(p, weight, shape, dtype):
    """out of the picks that were made and the bound on the distance to it (see D.decode)."""
    T, H, E, K, I, Ns = shape
    x, logits = p["x"].double(), p["logits"]
    idx = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :K]
    top = torch.gather(logits, 1, idx).double()
    g = torch.softmax(top, 1)
    eps, parts = D.EPS, 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -23
    out, err, mag = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(3))

    def add(names, e, rows, gate, slack):
        w1, w3, w2 = (weight(n, e) for n in names)
        a, b = x[rows] @ w1, x[rows] @ w3
        ea, eb = ((H + 16) * eps * (x[rows].abs() @ w.abs()) for w in (w1, w3))
        s = a * torch.sigmoid(a)
        h = s * b
        eh = 1.1 * ea * (b.abs() + eb) + s.abs() * eb + (parts + 2.0 ** -20) * h.abs()
        y = h @ w2
        ey = (eh + (I + 32) * eps * (h.abs() + eh)) @ w2.abs()
        out[rows] += gate * y
        err[rows] += gate * (ey * (1 + slack) + slack * y.abs())
        mag[rows] += gate * (y.abs() + ey)

    pairs = idx.cpu().numpy()
    for e in np.unique(pairs):
        t, k = (torch.from_numpy(i).cuda() for i in np.nonzero(pairs == e))
        add(("w1", "w3", "w2"), int(e), t, g[t, k, None], 2.0 ** -20)
    for s in range(Ns):
        add(("ws1", "ws3", "ws2"), s, torch.arange(T, device="cuda"), 1.0, 0.0)
    err += (K + 16) * eps * mag
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    return idx, g, out, err + half * (out.abs() + err) + 1e-38


@pytest.mark.parametrize("fmt,shape", [(f, s) for f in DK.FORMATS for s in DK.KERNEL_SHAPES[f]],
                         ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
def test_kernel_against_float64(fmt, shape):
    print(f"case {fmt} {shape} kernels {DK.kernels_of(fmt, shape)}", flush=True)
    T, H, E, K, I, Ns = shape
    p, weight = _inputs(fmt, shape)
    b = L.DecodeBuffers(L.make_dims(T, H, E, K, I, Ns, "bf16" if fmt.startswith("bf16") else "f32"))
    b.ws.fill_(0xA5)
    L.decode(b, p)
    idx, g, want, bound = _reference(p, weight, shape, b.out.dtype)
    assert torch.equal(b.topk_idx, idx.int())
    assert ((b.topk_w.double() - g).abs() <= (K + 16) * D.EPS * g + 1e-38).all()
    assert ((b.out.double() - want).abs() / bound).max() <= 1.0
