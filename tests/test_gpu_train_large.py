"""Router losses and stacked weights with more than 2^31 elements: offsets beyond 32 bits."""
import numpy as np
import pytest
import torch

import combine_moe_route_histogram_amd as M
from combine_moe_route_histogram_amd import layer as L
from oracle import train_oracle as TO

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def _room(gib):
    free, _ = torch.cuda.mem_get_info()
    if free < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def test_losses_of_many_rows():
    """8.4 million rows of 256 experts: all logits 0 but in the last rows, which are their own sequence."""
    _room(40)
    T, E, K, n = (1 << 23) + 37, 256, 1, 1 << 16
    tail = T % n                                          # the last sequence
    g = np.random.default_rng(1)
    last = g.standard_normal((tail, E)).astype(np.float32)
    l = torch.zeros(T, E, device="cuda")
    l[T - tail:] = torch.from_numpy(last).cuda()
    assert l.numel() > 2 ** 31
    idx = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    pick = np.argsort(-last, 1)[:, :K].astype(np.int32)
    idx[T - tail:] = torch.from_numpy(pick).cuda()
    d = L.make_dims(T, 8, E, K, 8)
    b = L.BalanceBuffers(d, n)
    print(f"case balance T={T} E={E} seq_len={n}", flush=True)
    L.balance(b, l, idx)
    dloss = torch.tensor([1.0, 0.0], device="cuda")
    out = torch.empty_like(l)
    M.moe_balance_bwd(d, n, l, None, b.counts, b.tokens, dloss, None, None, None, out)
    torch.cuda.synchronize()
    ref = TO.balance(last, pick, None, tail, E, K)
    S = b.counts.shape[0]
    tokens = b.tokens.cpu().numpy()
    assert tokens[S - 1] == tail and tokens[S] == T and tokens[S + 1] == S
    assert np.array_equal(b.counts[-1].cpu().numpy(), ref["counts"][0])
    assert np.all(np.abs(b.probs[-1].cpu().numpy() - ref["probs"][0]) <= 128 * EPS * ref["probs"][0])
    # every other sequence: p = 1/256 exactly, all picks on expert 0: balance 1; gradient p (q_0 - q_0 / 256) for expert 0
    assert torch.all(b.probs[:-1] == n / 256) and torch.all(b.counts[:-1, 0] == n)
    assert float(b.loss[0]) == pytest.approx(((S - 1) + ref["loss"][0]) / S, rel=256 * EPS)
    q = E / (K * n * S)
    row = out[T // 2].cpu().numpy()
    assert row[0] == pytest.approx(q * (1 - 1 / 256) / 256, rel=16 * EPS)
    assert row[1:] == pytest.approx(-q / 256 / 256, rel=16 * EPS)
    counts = np.concatenate([ref["tokens"][:1], [T, S]])
    want = TO.balance_bwd(last, None, tail, E, K, ref["counts"], counts, np.array([1.0, 0.0]))
    assert np.max(np.abs(out[T - tail:].cpu().numpy() - want)) <= 512 * EPS * np.abs(want).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_stack_of_many_elements(dtype):
    """2.2e9 elements, worked on part by part: the last matrix against float64 from its own entries."""
    _room(80)
    G, R, C = 33, 64, 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(3)
    g = torch.randn(G, R, C, generator=gen, device="cuda")
    assert g.numel() > 2 ** 31
    dt, code = (torch.bfloat16, M.BF16) if dtype == "bf16" else (torch.float32, M.F32)
    out = torch.empty(G, R, C, dtype=dt, device="cuda")
    ws = torch.empty(M.moe_muon_workspace_bytes(G, R, C, code), dtype=torch.uint8, device="cuda")
    print(f"case orthogonalize G={G} R={R} C={C} {dtype}", flush=True)
    M.moe_orthogonalize(G, R, C, g, out, ws)
    torch.cuda.synchronize()
    for i in (0, 16, G - 1):
        x = g[i].double()
        x /= x.square().sum().sqrt()
        for a, b, c in TO.COEF:
            gram = x @ x.T.contiguous()
            x = a * x + (b * gram + c * gram @ gram) @ x
        off = float((out[i].double() - x).norm() / x.norm())
        # bf16: the result's rounding and the factors' (1e-3 to 3e-3); float32: chains of 2^16 sums of 16 products with
        # half a step each, in five steps that each enlarge it at most 4-fold in sum
        assert off <= (2.0 ** -9 + 3e-3 if dtype == "bf16" else 5 * 4 * (1 << 16) ** 0.5 * EPS), (i, off)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_stack_of_many_elements_and_rows(dtype):
    """2.3e9 elements of matrices with more rows."""
    _room(80)
    G, R, C = 17, 130, 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(4)
    g = torch.randn(G, R, C, generator=gen, device="cuda")
    assert g.numel() > 2 ** 31
    dt, code = (torch.bfloat16, M.BF16) if dtype == "bf16" else (torch.float32, M.F32)
    out = torch.empty(G, R, C, dtype=dt, device="cuda")
    ws = torch.empty(M.moe_muon_workspace_bytes(G, R, C, code), dtype=torch.uint8, device="cuda")
    print(f"case orthogonalize G={G} R={R} C={C} {dtype}", flush=True)
    M.moe_orthogonalize(G, R, C, g, out, ws)
    torch.cuda.synchronize()
    for i in (0, G - 1):
        x = g[i].double()
        x /= x.square().sum().sqrt()
        for a, b, c in TO.COEF:
            gram = x @ x.T.contiguous()
            x = a * x + (b * gram + c * gram @ gram) @ x
        off = float((out[i].double() - x).norm() / x.norm())
        # as above
        assert off <= (2.0 ** -9 + 3e-3 if dtype == "bf16" else 5 * 4 * (1 << 16) ** 0.5 * EPS), (i, off)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bits_do_not_depend_on_the_place_in_the_stack(dtype):
    """9 matrices are worked on as 5 and 4, whose numbers of tiles lie on either side of where the products
    change to smaller ones: the first matrix once more as the last one gives the same bits."""
    _room(40)
    G, R, C = 9, 960, 1 << 17
    gen = torch.Generator(device="cuda").manual_seed(5)
    g = torch.randn(G, R, C, generator=gen, device="cuda")
    g[G - 1] = g[0]
    dt, code = (torch.bfloat16, M.BF16) if dtype == "bf16" else (torch.float32, M.F32)
    out = torch.empty(G, R, C, dtype=dt, device="cuda")
    ws = torch.empty(M.moe_muon_workspace_bytes(G, R, C, code), dtype=torch.uint8, device="cuda")
    print(f"case orthogonalize G={G} R={R} C={C} {dtype}", flush=True)
    M.moe_orthogonalize(G, R, C, g, out, ws)
    torch.cuda.synchronize()
    assert torch.isfinite(out[0]).all() and torch.equal(out[0], out[G - 1])


COEF32 = tuple(tuple(float(np.float32(v)) for v in abc) for abc in TO.COEF)   # as the kernels hold them


def _newton_on_device(u, coef):
    """float64 on the GPU."""
    x = u.double()
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x
    x = x / x.square().sum().sqrt()
    for a, b, c in coef:
        gram = x @ x.T.contiguous()
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.T if tall else x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", [(64, 1 << 20), (1 << 20, 64)])
def test_few_rows_of_many_elements(R, C, dtype):
    """2.2e9 elements of matrices with few rows, which are worked on in 64 bits: half a step of the result, and of
    float32 on the way to bf16."""
    _room(80)
    G = 33
    gen = torch.Generator(device="cuda").manual_seed(6)
    g = torch.randn(G, R, C, generator=gen, device="cuda")
    assert g.numel() > 2 ** 31
    dt, code = (torch.bfloat16, M.BF16) if dtype == "bf16" else (torch.float32, M.F32)
    out = torch.empty(G, R, C, dtype=dt, device="cuda")
    ws = torch.empty(M.moe_muon_workspace_bytes(G, R, C, code), dtype=torch.uint8, device="cuda")
    print(f"case orthogonalize G={G} R={R} C={C} {dtype}", flush=True)
    M.moe_orthogonalize(G, R, C, g, out, ws, coef=COEF32)
    torch.cuda.synchronize()
    step = EPS + (2.0 ** -8 if dtype == "bf16" else EPS / 4)
    for i in (0, 16, G - 1):
        x = _newton_on_device(g[i], COEF32)
        off = float((out[i].double() - x).norm() / x.norm())
        assert off <= step, (i, off)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", [(50, 1 << 20), (1 << 20, 50), (130, 1 << 20)])
def test_muon_step_of_many_elements(R, C, dtype):
    """A whole step on more than 2^31 elements: momentum, weights and bf16 copy of the first and last matrix.  mom: two
    roundings.  master: three, and lr scale times the update's error: of its direction (2^-23, up to 485-fold in null
    directions) for few rows; for more, 5e-3 of its norm (bf16) and what chains of 2^16 sums make (float32)."""
    _room(120)
    G = (1 << 31) // (R * C) + 1
    gen = torch.Generator(device="cuda").manual_seed(7)
    grad, mom, master = (torch.randn(G, R, C, generator=gen, device="cuda") for _ in range(3))
    assert grad.numel() > 2 ** 31
    code = M.BF16 if dtype == "bf16" else M.F32
    w = torch.empty(G, R, C, dtype=torch.bfloat16, device="cuda") if dtype == "bf16" else None
    ws = torch.empty(M.moe_muon_workspace_bytes(G, R, C, code), dtype=torch.uint8, device="cuda")
    picked = (0, G - 1)
    old = {i: (mom[i].clone(), master[i].clone()) for i in picked}
    print(f"case muon G={G} R={R} C={C} {dtype}", flush=True)
    lr, momentum, decay, scale = (float(np.float32(v)) for v in (0.02, 0.9, 0.1, 30.0))
    M.moe_muon(G, R, C, grad, mom, master, w, ws, lr=lr, momentum=momentum, weight_decay=decay, scale=scale, coef=COEF32)
    torch.cuda.synchronize()
    for i in picked:
        m = momentum * old[i][0].double() + grad[i].double()
        assert torch.all((mom[i].double() - m).abs() <= 2 * EPS * (old[i][0].double().abs() + grad[i].double().abs()))
        o = _newton_on_device(grad[i].double() + momentum * m, COEF32)
        want = (1 - lr * decay) * old[i][1].double() - lr * scale * o
        few = min(R, C) <= 64
        update = 2.0 ** -23 * (485 + float(o.norm())) if few else \
            float(o.norm()) * (5e-3 if dtype == "bf16" else 5 * 4 * (1 << 16) ** 0.5 * EPS)
        assert float((master[i].double() - want).norm()) <= lr * scale * update + 3 * EPS * float(want.norm()), i
        if w is not None:
            assert torch.equal(w[i], master[i].to(torch.bfloat16))


def test_losses_of_one_long_sequence():
    """16.8 million tokens as one sequence: 32768 chunks through one joining block, whose lanes add 1024 of them one
    after the other; a p is off by its argument's rounding and 8 steps, a chunk by 64 + 6 + 8 sums."""
    _room(20)
    T, E, K = (1 << 24) + 77, 8, 2
    gen = torch.Generator(device="cuda").manual_seed(8)
    l = torch.randn(T, E, generator=gen, device="cuda")
    idx = torch.topk(l, K, dim=1).indices.int().contiguous()
    mask = torch.rand(T, generator=gen, device="cuda") < 0.9
    d = L.make_dims(T, 8, E, K, 8)
    b = L.BalanceBuffers(d)
    print(f"case balance T={T} E={E} one sequence", flush=True)
    L.balance(b, l, idx, mask)
    torch.cuda.synchronize()
    x = l[mask].double()
    probs, n = torch.softmax(x, 1).sum(0), int(mask.sum())
    counts = torch.bincount(idx[mask].flatten().long(), minlength=E)
    assert torch.equal(b.counts[0].long(), counts) and b.tokens.tolist() == [n, n, 1]
    rel = EPS * (float(l.amax() - l.amin()) + 8 + 64 + 6 + 8 + 1024 + 32)
    assert torch.all((b.probs[0].double() - probs).abs() <= rel * probs)
    want = float(E / (K * n * n) * (counts.double() * probs).sum())
    assert abs(float(b.loss[0]) - want) <= (rel + EPS * (32 + E)) * want
    z = float(torch.logsumexp(x, 1).square().mean())
    top = float(l.abs().max()) + np.log(E) + 4
    assert abs(float(b.loss[1]) - z) <= 2 * top * top * 4 * EPS + rel * z
