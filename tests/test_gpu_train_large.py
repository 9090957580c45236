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
