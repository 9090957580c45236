"""What is measured of the layer for a few tokens and its 4-bit weights.

Four operators, each with a plain form in elementary torch operations and the
call a user makes of the framework:

 decode        one MoE layer, logits to output rows, for 1 to 256 tokens
 decode_mx     the same on weights packed to 4 bits (E2M1 codes, one power-of-
               two scale for 32 weights along the reduction dim: OCP MXFP4)
 quantize      weight matrices [G, K, N] to that packed form
 dequantize    the packed form back to matrices [G, K, N]

Packed matrix: G*(K/32)*N*16 bytes of codes, [G, K/32, N, 16] with weight
32 i + 2 j of column n in the low half of byte j and weight 32 i + 2 j + 1 in
the high half, then G*(K/32)*N scale bytes [G, K/32, N]; byte b stands for
2^(b - 127).
"""
import math

import torch

own = False

# Layer sizes of the repository's workloads: (H, E, K, I, n_shared).
SMALL = dict(H=128, E=8, K=2, I=256, n_shared=0)
FINE = dict(H=2048, E=64, K=6, I=1408, n_shared=2)
LONG = dict(H=2048, E=32, K=4, I=1408, n_shared=0)
WIDE = dict(H=4096, E=8, K=2, I=14336, n_shared=0)
MAX_TOKENS = 256


def listed():
    return [
        # the smallest layer: launches and latency are all there is
        dict(name="decode small f32 T1", op="decode", dtype="f32", T=1, tokens=1, **SMALL),
        # one sequence being generated, fine-grained experts with two shared ones
        dict(name="decode fine bf16 T1", op="decode", dtype="bf16", T=1, tokens=1, **FINE),
        # a batch padded to a fixed size, as a captured graph takes it: 13 of 16 rows are in use
        dict(name="decode long bf16 T16", op="decode", dtype="bf16", T=16, tokens=13, **LONG),
        # a batch that touches every expert of a layer with few, large ones (the largest case)
        dict(name="decode wide bf16 T32", op="decode", dtype="bf16", T=32, tokens=32, **WIDE),
        # one sequence on 4-bit weights: a quarter of the bytes, so launches and latency weigh most
        dict(name="mx fine bf16 T1", op="decode_mx", dtype="bf16", T=1, tokens=1, **FINE),
        # a few sequences, large experts
        dict(name="mx wide bf16 T7", op="decode_mx", dtype="bf16", T=7, tokens=7, **WIDE),
        # float32 activations on 4-bit weights
        dict(name="mx small f32 T33", op="decode_mx", dtype="f32", T=33, tokens=33, **SMALL),
        # a large decode batch: every expert has about 25 tokens
        dict(name="mx long bf16 T200", op="decode_mx", dtype="bf16", T=200, tokens=200, **LONG),
        # packing one projection of a whole layer when weights are loaded
        dict(name="quantize fine bf16", op="quantize", dtype="bf16", G=64, K=2048, N=1408),
        # float32 masters, odd sizes
        dict(name="quantize odd f32", op="quantize", dtype="f32", G=3, K=224, N=1000),
        # plain weights of a layer for a long prompt, which runs the grouped GEMMs
        dict(name="dequantize wide bf16", op="dequantize", dtype="bf16", G=8, K=4096, N=14336),
        dict(name="dequantize odd f32", op="dequantize", dtype="f32", G=5, K=416, N=264),
    ]


def _log(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode_mx", "decode_mx", "quantize", "dequantize"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("quantize", "dequantize"):
        K, N = _log(rng, 32, 4096, 32), _log(rng, 8, 14336, 8)
        most = max(1, min(64, 8 * 4096 * 14336 // (2 * K * N)))
        return dict(op=op, dtype=dtype, G=_log(rng, 1, most, 1) if most > 1 else 1, K=K, N=N)
    step = 32 if op == "decode_mx" else 8
    H, I = _log(rng, 64, 4096, step), _log(rng, 64, 14336, step)
    most = max(1, min(256, 8 * 4096 * 14336 // (2 * H * I)))
    E = _log(rng, 1, most, 1) if most > 1 else 1
    T = _log(rng, 1, MAX_TOKENS, 1)
    return dict(op=op, dtype=dtype, T=T, tokens=T if rng.random() < 0.7 else rng.randint(1, T), H=H, E=E,
                K=min(E, rng.randint(1, 8)), I=I, n_shared=rng.choice([0, 0, 1, 2]))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _matrices(case):
    """(name, groups, reduction dim, columns) of the layer's weights."""
    H, I, E, Ns = case["H"], case["I"], case["E"], case["n_shared"]
    got = [("w1", E, H, I), ("w3", E, H, I), ("w2", E, I, H)]
    return got + ([("ws1", Ns, H, I), ("ws3", Ns, H, I), ("ws2", Ns, I, H)] if Ns else [])


# ---------------------------------------------------------------- plain forms

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _scale_bytes(w32):
    """[.., K/32, N] scale bytes of [.., K/32, 32, N] weights: the exponent of the group's largest
    magnitude less that of the largest code (6 = 1.5 * 2^2), kept in the normal range."""
    e = torch.frexp(w32.abs().amax(-2))[1] - 1          # floor(log2), exact
    return (e - 2 + 127).clamp(1, 254)


def _round_e2m1(v):
    """Nearest E2M1 value, ties to the even code, magnitudes above 6 to 6."""
    a = v.abs()
    r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(r.clamp(max=6.0), v)


def _grouped(w):
    return w.float().unflatten(-2, (-1, 32))


def _pack(w):
    """Packed bytes of the matrices w [G, K, N]: (codes [G, K/32, N, 16], scales [G, K/32, N])."""
    g = _grouped(w)
    b = _scale_bytes(g)
    v = _round_e2m1(torch.ldexp(g, 127 - b.unsqueeze(-2)))
    a = v.abs()
    mag = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (mag + torch.signbit(v).to(torch.uint8) * 8).transpose(-1, -2)
    return code[..., 0::2] + code[..., 1::2] * 16, b.to(torch.uint8)


def _unpack(codes, scales):
    """float32 matrices [G, K, N] of packed ones."""
    lut = torch.tensor(E2M1, device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)   # [G, K/32, N, 32]
    return torch.ldexp(v, scales.int().unsqueeze(-1) - 127).transpose(-1, -2).flatten(1, 2)


def _mx_views(mx, G, K, N):
    n = G * (K // 32) * N
    return mx[:16 * n].view(G, K // 32, N, 16), mx[16 * n:17 * n].view(G, K // 32, N)


def _plain_weights(state, name, pick):
    """float32 matrices of the picked groups (all of them where pick is None)."""
    case = state["case"]
    _, G, K, N = next(m for m in _matrices(case) if m[0] == name)
    w = state[name]
    if case["op"] == "decode":
        return (w if pick is None else w[pick]).float()
    codes, scales = _mx_views(w, G, K, N)
    return _unpack(codes, scales) if pick is None else _unpack(codes[pick], scales[pick])


def _plain_ffn(state, names, x, pick):
    """SwiGLU of the rows x [.., rows, H] by the picked groups."""
    a = torch.matmul(x, _plain_weights(state, names[0], pick))
    b = torch.matmul(x, _plain_weights(state, names[1], pick))
    h = a * torch.sigmoid(a) * b
    del a, b
    return torch.matmul(h, _plain_weights(state, names[2], pick))


def _plain_decode(state):
    case = state["case"]
    T, E, K = case["T"], case["E"], case["K"]
    logits, x = state["logits"], state["x"].float()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)     # equal logits: lower expert first
    idx, w = idx[:, :K], torch.softmax(top[:, :K], 1)
    if T * K <= E:           # the picked experts' weights for each pair
        rows = x.repeat_interleave(K, 0).unsqueeze(1)
        y = _plain_ffn(state, ("w1", "w3", "w2"), rows, idx.reshape(-1)).view(T, K, -1)
    else:                    # every expert on every token
        y = _plain_ffn(state, ("w1", "w3", "w2"), x.unsqueeze(0), None)
        y = y[idx, torch.arange(T, device=x.device).unsqueeze(1)]
    out = (w.unsqueeze(-1) * y).sum(1)
    if case["n_shared"]:
        out = out + _plain_ffn(state, ("ws1", "ws3", "ws2"), x.unsqueeze(0), None).sum(0)
    used = torch.arange(T, device=x.device).unsqueeze(1) < state["n_tokens"]
    return {"out": torch.where(used, out, torch.zeros_like(out)).to(_dtype(case)),
            "topk_idx": torch.where(used, idx, torch.zeros_like(idx)).int(),
            "topk_w": torch.where(used, w, torch.zeros_like(w))}


# ---------------------------------------------------------------- the framework's calls

def _own_decode(state):
    from combine_moe_route_histogram_amd import layer as L
    case = state["case"]
    if "buffers" not in state:                       # buffers and workspace: a program keeps them
        d = L.make_dims(*(case[k] for k in ("T", "H", "E", "K", "I", "n_shared", "dtype")))
        state["buffers"] = L.DecodeBuffers(d)
        for t in (state["buffers"].out, state["buffers"].topk_idx, state["buffers"].topk_w):
            t.zero_()                                # rows that are not in use stay as they are
    b = state["buffers"]
    L.decode(b, state)
    return {"out": b.out, "topk_idx": b.topk_idx, "topk_w": b.topk_w}


def _own_quantize(state):
    import combine_moe_route_histogram_amd as M
    G, K, N = (state["case"][k] for k in "GKN")
    if "mx" not in state:
        state["mx"] = torch.empty(M.moe_mx_bytes(G, K, N), dtype=torch.uint8, device="cuda")
        state["back"] = torch.empty_like(state["w"])
    M.moe_mx_quantize(G, K, N, state["w"], state["mx"])
    M.moe_mx_dequantize(G, K, N, state["mx"], state["back"])     # the values the codes stand for
    return state["back"]


def _own_dequantize(state):
    import combine_moe_route_histogram_amd as M
    case = state["case"]
    G, K, N = (case[k] for k in "GKN")
    if "back" not in state:
        state["back"] = torch.empty(G, K, N, dtype=_dtype(case), device="cuda")
    M.moe_mx_dequantize(G, K, N, state["packed"], state["back"])
    return state["back"]


# ---------------------------------------------------------------- cases

def _draw_weights(gen, G, K, N, dtype):
    return torch.randn(G, K, N, generator=gen, device="cuda", dtype=dtype) * 0.02


def _packed(gen, G, K, N, dtype):
    """A packed draw, group by group (the float32 steps of a whole layer would be large)."""
    n = G * (K // 32) * N
    mx = torch.empty(17 * n, dtype=torch.uint8, device="cuda")
    codes, scales = _mx_views(mx, G, K, N)
    per = max(1, (1 << 26) // (K * N))
    for g in range(0, G, per):
        c, s = _pack(_draw_weights(gen, min(per, G - g), K, N, dtype))
        codes[g:g + per], scales[g:g + per] = c, s
    return mx


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)
    state = {"case": case}
    if case["op"] == "quantize":
        state["w"] = _draw_weights(gen, case["G"], case["K"], case["N"], dt)
    elif case["op"] == "dequantize":
        state["packed"] = _packed(gen, case["G"], case["K"], case["N"], dt)
    else:
        T = case["T"]
        state["logits"] = torch.randn(T, case["E"], generator=gen, device="cuda")
        state["x"] = torch.randn(T, case["H"], generator=gen, device="cuda", dtype=dt)
        state["n_tokens"] = torch.tensor([case["tokens"]], dtype=torch.int32, device="cuda")
        make = _draw_weights if case["op"] == "decode" else _packed
        for name, G, K, N in _matrices(case):
            state[name] = make(gen, G, K, N, dt)
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        return {"quantize": _own_quantize, "dequantize": _own_dequantize}.get(op, _own_decode)(state)
    if op == "quantize":
        g = _grouped(state["w"])
        b = _scale_bytes(g).unsqueeze(-2)
        return torch.ldexp(_round_e2m1(torch.ldexp(g, 127 - b)), b - 127).flatten(-3, -2).to(_dtype(state["case"]))
    if op == "dequantize":
        case = state["case"]
        return _unpack(*_mx_views(state["packed"], case["G"], case["K"], case["N"])).to(_dtype(case))
    return _plain_decode(state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("quantize", "dequantize"):
        n = case["G"] * case["K"] * case["N"]
        # quantize: the codes are written, read and given back as values
        return {"bytes": n * (2 * size + 34 / 32) if case["op"] == "quantize" else n * (size + 17 / 32), "flops": 2 * n}
    H, I, E, K, Ns, T = case["H"], case["I"], case["E"], case["K"], case["n_shared"], case["tokens"]
    per = 3 * H * I * (size if case["op"] == "decode" else 17 / 32)
    experts = E * (1 - (1 - K / E) ** T) + (Ns if T else 0)      # expected number with a token
    return {"bytes": experts * per + T * (2 * H * size + 4 * E + 8 * K) + 4, "flops": 6 * H * I * T * (K + Ns)}


# ---------------------------------------------------------------- in 64 bits

def _exact_values(mx, G, K, N):
    """float64 matrices of packed ones, from the bit fields: (-1)^s 2^max(e,1) (m/2 + [e > 0]) / 2."""
    codes, scales = _mx_views(mx, G, K, N)
    out = torch.empty(G, K // 32, 32, N, dtype=torch.float64, device=mx.device)
    for j in range(32):
        c = (codes[..., j // 2].int() >> (4 * (j % 2))) & 15
        e, m = (c >> 1) & 3, (c & 1).double()
        v = torch.exp2(e.clamp(min=1).double() - 1) * ((e > 0).double() + m / 2)
        out[:, :, j] = torch.where(c >= 8, -v, v) * torch.exp2(scales.double() - 127)
    return out.view(G, K, N)


def _exact_nearest(w):
    """float64 values of the packed form of one matrix w [K, N]: by distance to the eight magnitudes."""
    g = w.double().view(-1, 32, w.shape[-1])
    big = g.abs().amax(1, keepdim=True)
    step = torch.full_like(big, 2.0 ** -126)             # the scale of a group: 2^floor(log2(big)) / 4
    for _ in range(260):
        step = torch.where(step * 8 <= big, step * 2, step)
    mags = torch.tensor(E2M1[:8], dtype=torch.float64, device=w.device)
    best, at = torch.full_like(g, math.inf), torch.zeros_like(g)
    for k in (0, 2, 4, 6, 1, 3, 5, 7):                   # even codes first: they win ties
        far = (g.abs() / step - mags[k]).abs()
        at = torch.where(far < best, mags[k], at)
        best = torch.minimum(best, far)
    return (at * step * torch.sign(g)).view(w.shape)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        return torch.stack([_exact_nearest(w) for w in state["w"]])
    if case["op"] == "dequantize":
        one = case["K"] // 32 * case["N"]
        n = case["G"] * one
        mx, out = state["packed"], torch.empty(case["G"], case["K"], case["N"], dtype=torch.float64, device="cuda")
        for g in range(case["G"]):
            part = torch.cat((mx[16 * one * g:16 * one * (g + 1)], mx[16 * n + one * g:16 * n + one * (g + 1)]))
            out[g] = _exact_values(part, 1, case["K"], case["N"])[0]
        return out
    shapes = {m[0]: m[1:] for m in _matrices(case)}

    def matrix(name, g):
        G, K, N = shapes[name]
        if case["op"] == "decode":
            return state[name][g].double()
        one = K // 32 * N
        mx = state[name]
        return _exact_values(torch.cat((mx[16 * one * g:16 * one * (g + 1)], mx[16 * one * G + one * g:16 * one * G + one * (g + 1)])), 1, K, N)[0]

    def ffn(x, names, g):
        a = x @ matrix(names[0], g)
        return (a / (1 + torch.exp(-a)) * (x @ matrix(names[1], g))) @ matrix(names[2], g)

    T, K, n = case["T"], case["K"], case["tokens"]
    x, logits = state["x"].double(), state["logits"].double().cpu()
    out = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
    idx, w = torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K, dtype=torch.float64)
    for t in range(n):
        order = sorted(range(case["E"]), key=lambda e: (-float(logits[t, e]), e))[:K]
        z = torch.exp(logits[t, order] - logits[t, order[0]])
        idx[t], w[t] = torch.tensor(order), z / z.sum()
    for e in sorted(set(idx[:n].flatten().tolist())):
        rows, slot = torch.nonzero(idx[:n] == e, as_tuple=True)
        out[rows.cuda()] += w[rows, slot].cuda().unsqueeze(1) * ffn(x[rows.cuda()], ("w1", "w3", "w2"), e)
    if n:
        for s in range(case["n_shared"]):
            out[:n] += ffn(x[:n], ("ws1", "ws3", "ws2"), s)
    return {"out": out, "topk_idx": idx, "topk_w": w}
