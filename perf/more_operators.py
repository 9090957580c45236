"""What is measured of the operators of a training step beside the layer itself.

Four operators, each with a plain form in elementary torch operations and the
call a user makes of the framework:

 balance        the router's losses: load balance over sequences and the squared
                log-sum-exp of the logits, with per-expert counts
 balance_bwd    their gradient for the logits, with that of the selected
                experts' softmax weights (moe_route_bwd's) in the same pass
 orthogonalize  stacked matrices [G, R, C] made nearly orthogonal by
                Newton-Schulz products, as an update of a stack of weights is
 muon           the whole update of a stack of weights: momentum, the same
                products, decay, the float32 weights and their bf16 copy

Tokens are cut into sequences of seq_len (the last one may be shorter); mask is
0 for padding.  With p = softmax(logits), n = a sequence's tokens, c = its picks
of an expert, P = its sum of p:  balance = mean over the sequences with tokens
of E / (K n^2) sum_e c_e P_e;  z = mean over all tokens of logsumexp^2.
"""
import math

import torch

own = False

# Sizes of the repository's workloads.
SMALL = dict(T=256, E=8, K=2)
FINE = dict(T=8192, E=64, K=6)
LONG = dict(T=131072, E=32, K=4)

STEPS = 5
COEF = (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # the smallest layer's batch: launches and latency are all there is
        dict(name="balance small T256 E8", op="balance", seq_len=256, masked=0.0, **SMALL),
        # a batch of padded sequences of an odd length, the last one cut short
        dict(name="balance padded T8192 E64", op="balance", seq_len=1000, masked=0.2, **FINE),
        # one long sequence
        dict(name="balance long T131072 E32", op="balance", seq_len=131072, masked=0.0, **LONG),
        # few tokens, an odd number of experts, short padded sequences
        dict(name="balance_bwd odd T1000 E63", op="balance_bwd", T=1000, E=63, K=6, seq_len=100, masked=0.3),
        # the gradient of the long sequence
        dict(name="balance_bwd long T131072 E32", op="balance_bwd", seq_len=131072, masked=0.0, **LONG),
        # as many experts as the layer takes, several sequences
        dict(name="balance_bwd many T16384 E256", op="balance_bwd", T=16384, E=256, K=8, seq_len=4096, masked=0.1),
        # the smallest layer's gate projections, float32 all the way
        dict(name="orthogonalize small f32", op="orthogonalize", dtype="f32", G=8, R=128, C=256),
        # odd sizes, taller than wide
        dict(name="orthogonalize odd f32", op="orthogonalize", dtype="f32", G=3, R=1001, C=227),
        # one projection of a layer of many small experts, taller than wide
        dict(name="orthogonalize fine bf16", op="orthogonalize", dtype="bf16", G=64, R=2048, C=1408),
        # the step of a small float32 stack, plain momentum
        dict(name="muon odd f32", op="muon", dtype="f32", G=5, R=264, C=416, nesterov=False),
        # the step of the down projections of the long-sequence layer
        dict(name="muon long bf16", op="muon", dtype="bf16", G=32, R=1408, C=2048, nesterov=True),
        # few, large experts (the largest case)
        dict(name="muon wide bf16", op="muon", dtype="bf16", G=8, R=4096, C=14336, nesterov=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _products(G, R, C):
    s, l = min(R, C), max(R, C)
    return G * s * s * (2 * l + s)


def draw(rng):
    op = rng.choice(["balance", "balance_bwd", "orthogonalize", "muon"])
    if op in ("balance", "balance_bwd"):
        T, E = _log(rng, 1, 131072), _log(rng, 1, 256)
        if T * E > 131072 * 32:
            T = 131072 * 32 // E
        return dict(op=op, T=T, E=E, K=rng.randint(1, min(E, 8)), seq_len=T if rng.random() < 0.4 else _log(rng, 1, T),
                    masked=rng.choice([0.0, 0.0, 0.1, 0.5]))
    R, C = _log(rng, 8, 4096), _log(rng, 8, 14336)
    if rng.random() < 0.5:
        R, C = C, R
    most = max(1, min(64, _products(8, 4096, 14336) // (2 * _products(1, R, C)), 8 * 4096 * 14336 // (2 * R * C)))
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), G=_log(rng, 1, most) if most > 1 else 1, R=R, C=C)
    if op == "muon":
        case["nesterov"] = rng.random() < 0.5
    return case


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ---------------------------------------------------------------- plain forms

def _sequences(case, v):
    """v [T, ...] as [S, seq_len, ...], filled up with zeros."""
    T, n = case["T"], case["seq_len"]
    S = -(-T // n)
    full = v.new_zeros((S * n,) + v.shape[1:])
    full[:T] = v
    return full.view((S, n) + v.shape[1:])


def _softmax(state):
    """Probabilities and log-sum-exp of the unmasked rows, zeros in the others."""
    used = state["mask"].bool().unsqueeze(1)
    l = torch.where(used, state["logits"], torch.zeros_like(state["logits"]))
    top = l.amax(1, keepdim=True)
    z = torch.exp(l - top)
    total = z.sum(1, keepdim=True)
    zero = torch.zeros_like(top)
    return torch.where(used, z / total, zero), torch.where(used, torch.log(total) + top, zero)


def _plain_balance(state):
    case = state["case"]
    E, K = case["E"], case["K"]
    mask = state["mask"].bool()
    p, lse = _softmax(state)
    picks = torch.zeros_like(p, dtype=torch.int32).scatter_(1, state["topk_idx"].long(), 1) * mask.unsqueeze(1)
    counts = _sequences(case, picks).sum(1)
    probs = _sequences(case, p).sum(1)
    n = _sequences(case, mask.int()).sum(1)
    full = n.clamp(min=1).float()
    each = E / K * (counts.float() / full.unsqueeze(1) * (probs / full.unsqueeze(1))).sum(1)
    some, total = (n > 0).sum(), n.sum()
    loss = torch.stack((each.sum() / some.clamp(min=1), (lse * lse).sum() / total.clamp(min=1)))
    return {"loss": loss, "counts": counts.int(), "tokens": torch.cat((n, total.view(1), some.view(1))).int(), "probs": probs}


def _plain_balance_bwd(state):
    case = state["case"]
    E, K, T = case["E"], case["K"], case["T"]
    p, lse = _softmax(state)
    counts, tokens, dloss = state["counts"].float(), state["tokens"].float(), state["dloss"]
    n, total, some = tokens[:-2], tokens[-2].clamp(min=1), tokens[-1].clamp(min=1)
    q = dloss[0] * (E / K) * counts / (n.clamp(min=1).square() * some).unsqueeze(1)
    q = q[torch.arange(T, device=p.device) // case["seq_len"]]
    d = p * (q - (p * q).sum(1, keepdim=True) + 2 * dloss[1] * lse / total)
    w, dw = state["topk_w"], state["dtopk_w"]
    return d.scatter_add(1, state["topk_idx"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))


def _plain_orthogonal(u):
    """float32 [G, R, C] of the matrices u: five products' worth of the quintic."""
    a, b, c = COEF
    tall = u.shape[1] > u.shape[2]
    x = u.mT.contiguous() if tall else u
    x = x / x.square().sum((1, 2), keepdim=True).sqrt()
    for _ in range(STEPS):
        gram = torch.matmul(x, x.mT.contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return x.mT.contiguous() if tall else x


def _plain_muon(state):
    case, h = state["case"], state["hyper"]
    mom, master = state["mom"], state["master"]
    mom.mul_(h["momentum"]).add_(state["grad"])
    u = state["grad"] + h["momentum"] * mom if case["nesterov"] else mom
    master.mul_(1 - h["lr"] * h["weight_decay"]).sub_(h["lr"] * h["scale"] * _plain_orthogonal(u))
    got = {"mom": mom, "master": master}
    if case["dtype"] == "bf16":
        state["w"].copy_(master)
        got["w"] = state["w"]
    return got


# ---------------------------------------------------------------- the framework's calls

def _own_balance(state):
    from combine_moe_route_histogram_amd import layer as L
    case = state["case"]
    if "buffers" not in state:
        d = L.make_dims(case["T"], 8, case["E"], case["K"], 8)
        state["buffers"] = L.BalanceBuffers(d, case["seq_len"])
    b = state["buffers"]
    L.balance(b, state["logits"], state["topk_idx"], state["mask"])
    return {"loss": b.loss, "counts": b.counts, "tokens": b.tokens, "probs": b.probs}


def _own_balance_bwd(state):
    import combine_moe_route_histogram_amd as M
    from combine_moe_route_histogram_amd import layer as L
    case = state["case"]
    if "dims" not in state:
        state["dims"] = L.make_dims(case["T"], 8, case["E"], case["K"], 8)
        state["dlogits"] = torch.empty_like(state["logits"])
    M.moe_balance_bwd(state["dims"], case["seq_len"], state["logits"], state["mask"], state["counts"], state["tokens"],
                      state["dloss"], state["dtopk_w"], state["topk_w"], state["topk_idx"], state["dlogits"])
    return state["dlogits"]


def _workspace(state):
    import combine_moe_route_histogram_amd as M
    case = state["case"]
    code = M.BF16 if case["dtype"] == "bf16" else M.F32
    return torch.empty(M.moe_muon_workspace_bytes(case["G"], case["R"], case["C"], code), dtype=torch.uint8, device="cuda")


def _own_orthogonalize(state):
    import combine_moe_route_histogram_amd as M
    case = state["case"]
    if "ws" not in state:
        state["ws"] = _workspace(state)
        state["out"] = torch.empty(state["g"].shape, dtype=_dtype(case), device="cuda")
    M.moe_orthogonalize(case["G"], case["R"], case["C"], state["g"], state["out"], state["ws"])
    return state["out"]


def _own_muon(state):
    import combine_moe_route_histogram_amd as M
    case = state["case"]
    if "ws" not in state:
        state["ws"] = _workspace(state)
    M.moe_muon(case["G"], case["R"], case["C"], state["grad"], state["mom"], state["master"], state.get("w"), state["ws"],
               nesterov=case["nesterov"], **state["hyper"])
    return {k: state[k] for k in ("mom", "master", "w") if k in state}


# ---------------------------------------------------------------- cases

def _gradients(gen, case):
    """Draws of full rank whose rows and columns differ in size, as gradients' do."""
    G, R, C = (case[k] for k in "GRC")
    g = torch.randn(G, R, C, generator=gen, device="cuda")
    g *= torch.exp(0.5 * torch.randn(G, R, 1, generator=gen, device="cuda"))
    g *= 1e-4 * torch.exp(0.5 * torch.randn(G, 1, C, generator=gen, device="cuda"))
    return g


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "orthogonalize":
        state["g"] = _gradients(gen, case)
        return state
    if case["op"] == "muon":
        G, R, C = (case[k] for k in "GRC")
        state["grad"] = _gradients(gen, case)
        state["mom"] = _gradients(gen, case) * 3
        state["master"] = torch.randn(G, R, C, generator=gen, device="cuda") * 0.02
        if case["dtype"] == "bf16":
            state["w"] = state["master"].to(torch.bfloat16)
        state["hyper"] = dict(lr=3e-4, momentum=0.95, weight_decay=0.1, scale=0.2 * math.sqrt(max(R, C)))
        return state
    T, E, K, n = case["T"], case["E"], case["K"], case["seq_len"]
    logits = torch.randn(T, E, generator=gen, device="cuda")
    logits += 0.7 * torch.randn(E, generator=gen, device="cuda")              # some experts are liked better
    state["logits"] = logits
    state["mask"] = (torch.rand(T, generator=gen, device="cuda") >= case["masked"]).to(torch.uint8)
    state["mask"][0] = 1                                                      # a batch has a token
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    state["topk_idx"] = idx[:, :K].int().contiguous()
    if case["op"] == "balance_bwd":
        state["topk_w"] = torch.softmax(top[:, :K], 1)
        state["dtopk_w"] = torch.randn(T, K, generator=gen, device="cuda") / T
        state["dloss"] = torch.tensor([0.01, 0.001], device="cuda") * (1 + torch.rand(2, generator=gen, device="cuda"))
        mask = state["mask"].int()
        picks = torch.zeros(T, E, dtype=torch.int32, device="cuda").scatter_(1, idx[:, :K], 1) * mask.unsqueeze(1)
        state["counts"] = _sequences(case, picks).sum(1).int()
        tokens = _sequences(case, mask).sum(1)
        state["tokens"] = torch.cat((tokens, tokens.sum().view(1), (tokens > 0).sum().view(1))).int()
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        return {"balance": _own_balance, "balance_bwd": _own_balance_bwd, "orthogonalize": _own_orthogonalize,
                "muon": _own_muon}[op](state)
    if op == "orthogonalize":
        return _plain_orthogonal(state["g"]).to(_dtype(state["case"]))
    return {"balance": _plain_balance, "balance_bwd": _plain_balance_bwd, "muon": _plain_muon}[op](state)


def work(case):
    if case["op"] in ("balance", "balance_bwd"):
        T, E, K = case["T"], case["E"], case["K"]
        S = -(-T // case["seq_len"])
        if case["op"] == "balance":
            return {"bytes": T * (4 * E + 4 * K + 1) + S * (8 * E + 4), "flops": 6 * T * E}
        return {"bytes": T * (8 * E + 12 * K + 1) + S * (4 * E + 4), "flops": 10 * T * E}
    G, R, C = (case[k] for k in "GRC")
    s, l, n = min(R, C), max(R, C), G * R * C
    size = 2 if case["dtype"] == "bf16" else 4
    # of the two symmetric products of a step, one half each
    flops = STEPS * G * (3 * s * s * l + s ** 3) + 3 * n
    if case["op"] == "orthogonalize":
        return {"bytes": n * (4 + size), "flops": flops}
    return {"bytes": n * (4 + 8 + 8 + (2 if size == 2 else 0)), "flops": flops + 8 * n}


# ---------------------------------------------------------------- in 64 bits

def _exact_orthogonal(u):
    """float64 of one matrix: the quintic on the other side, in nested form."""
    a, b, c = COEF
    u = u.double()
    x = u if u.shape[0] >= u.shape[1] else u.T.contiguous()                   # tall
    x = x / torch.linalg.vector_norm(x)
    for _ in range(STEPS):
        gram = x.T.contiguous() @ x
        y = x @ gram
        x = a * x + b * y + c * (y @ gram)
    return x if u.shape[0] >= u.shape[1] else x.T


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "orthogonalize":
        return torch.stack([_exact_orthogonal(g) for g in state["g"]])
    if case["op"] == "muon":
        h = state["hyper"]
        mom, master = state["mom"].double(), state["master"].double()
        for g in range(case["G"]):
            grad = state["grad"][g].double()
            mom[g] = h["momentum"] * mom[g] + grad
            step = _exact_orthogonal(grad + h["momentum"] * mom[g] if case["nesterov"] else mom[g])
            master[g] -= h["lr"] * (h["weight_decay"] * master[g] + h["scale"] * step)
        got = {"mom": mom, "master": master}
        return {**got, "w": master} if case["dtype"] == "bf16" else got
    T, E, K, n = case["T"], case["E"], case["K"], case["seq_len"]
    S = -(-T // n)
    rows = torch.nonzero(state["mask"]).flatten()
    seq = rows // n
    l = state["logits"][rows].double()
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse.unsqueeze(1))
    if case["op"] == "balance":
        chosen = state["topk_idx"][rows].long() + (seq * E).unsqueeze(1)
        counts = torch.bincount(chosen.flatten(), minlength=S * E).view(S, E)
        tokens = torch.bincount(seq, minlength=S)
        probs = torch.zeros(S, E, dtype=torch.float64, device="cuda").index_add_(0, seq, p)
        full = tokens > 0
        each = E / K * (counts[full] * probs[full]).sum(1) / tokens[full].double() ** 2
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        loss = torch.stack((each.mean() if len(each) else zero, lse.square().mean() if len(rows) else zero))
        return {"loss": loss, "counts": counts.int(), "tokens": torch.cat((tokens, tokens.sum().view(1), full.sum().view(1))).int(),
                "probs": probs}
    g0, g1 = state["dloss"].double()
    tokens = state["tokens"].double()
    share = state["counts"][seq].double() * (g0 * E / K / tokens[-1]) / (tokens[seq] ** 2).unsqueeze(1)
    slope = share + (2 * g1 / tokens[-2]) * lse.unsqueeze(1)
    d = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    d[rows] = p * slope - p * (p * share).sum(1, keepdim=True)
    w, dw = state["topk_w"].double(), state["dtopk_w"].double()
    inner = (w * dw).sum(1)
    for k in range(K):
        d[torch.arange(T, device="cuda"), state["topk_idx"][:, k].long()] += w[:, k] * (dw[:, k] - inner)
    return d
