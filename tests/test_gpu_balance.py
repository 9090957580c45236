"""The router's losses, counts and gradient (moe_balance, moe_balance_bwd) against float64."""
import numpy as np
import pytest
import torch

import combine_moe_route_histogram_amd as M
from combine_moe_route_histogram_amd import layer as L
from gpu_util import custom_config, device_inputs, host
from oracle import train_oracle as TO
import oracle as O
import synth

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24   # half a step of float32, relative

# T, E, K, seq_len, share of padding
SHAPES = [
    (1, 1, 1, 1, 0.0), (1, 8, 2, 1, 0.0), (2, 3, 3, 1, 0.5), (7, 4, 1, 3, 0.0), (65, 5, 2, 64, 0.3),
    (64, 16, 4, 64, 0.0), (65, 12, 2, 65, 0.3), (300, 17, 6, 7, 0.2), (511, 64, 6, 511, 0.0), (513, 63, 6, 513, 0.1),
    (513, 64, 8, 512, 0.1), (1025, 20, 20, 1025, 0.5), (1500, 32, 4, 700, 0.0), (2000, 65, 3, 2000, 0.1),
    (900, 128, 8, 65, 0.1), (700, 130, 7, 700, 0.0), (600, 255, 8, 600, 0.2), (600, 256, 256, 550, 0.2),
    (3000, 8, 2, 1030, 0.9), (20000, 4, 1, 1, 0.5), (20001, 6, 2, 2, 0.1), (1000, 70, 9, 8, 0.3), (999, 256, 12, 9, 0.3), (123, 130, 130, 5, 0.2), (68000, 3, 1, 66, 0.1), (115000, 2, 2, 112, 0.0),
]


def _case(T, E, K, masked, seed, spread=1.0):
    g = np.random.default_rng(seed)
    l = (spread * (g.standard_normal((T, E)) + 0.5 * g.standard_normal(E))).astype(np.float32)
    idx = np.argsort(-l, 1, kind="stable")[:, :K].astype(np.int32)
    mask = (g.random(T) >= masked).astype(np.uint8)
    w = np.abs(g.standard_normal((T, K))).astype(np.float32)
    w /= w.sum(1, keepdims=True)
    dw = g.standard_normal((T, K)).astype(np.float32)
    return l, idx, mask, w, dw


def _cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _forward(l, idx, mask, n, guard=0):
    T, E = l.shape
    d = L.make_dims(T, 8, E, idx.shape[1], 8)
    b = L.BalanceBuffers(d, n)
    b.ws.fill_(0xA5)                                     # any state of the workspace
    if guard:                                            # sentinels behind the outputs
        for name in ("counts", "tokens", "probs", "loss"):
            t = getattr(b, name)
            full = torch.full((t.numel() + guard,), 7, dtype=t.dtype, device="cuda")
            setattr(b, name, full)
    L.balance(b, _cuda(l), _cuda(idx), _cuda(mask))
    torch.cuda.synchronize()
    return d, b


def _check_forward(b, ref, l, mask, S, E):
    """p is off by the argument's rounding in exp (|l - max| EPS), 2 ulp of exp and of the division; a
    sum of n non-negative terms by EPS for each addition in its longest chain: 64 rows of a wave, 6
    exchanges, 8 waves, and 64 chunks with their 32 rows; a mean over the sequences by 16 for a wave's or a
    thread's share of them."""
    used = l[mask.astype(bool)] if mask is not None else l
    span = float(np.ptp(used, axis=1).max()) if used.size else 0.0
    rel = EPS * (span + 8 + 64 + 6 + 8 + 64 + 32)
    assert np.array_equal(host(b.counts).ravel()[:S * E].reshape(S, E), ref["counts"])
    assert np.array_equal(host(b.tokens).ravel()[:S + 2], ref["tokens"])
    probs, loss = host(b.probs).ravel()[:S * E].reshape(S, E), host(b.loss).ravel()[:2]
    assert np.all(np.abs(probs - ref["probs"]) <= rel * ref["probs"] + 1e-37)
    assert abs(loss[0] - ref["loss"][0]) <= (rel + EPS * (32 + E)) * ref["loss"][0]
    # lse = max + log(sum): off by EPS (|max| + |log| + 4); its square by twice |lse| of that
    top = float(np.abs(used).max()) + np.log(E) + 4 if used.size else 0.0
    assert abs(loss[1] - ref["loss"][1]) <= 2 * top * top * 4 * EPS + rel * ref["loss"][1]


@pytest.mark.parametrize("T,E,K,n,masked", SHAPES)
def test_losses_and_counts(T, E, K, n, masked):
    print(f"case balance T={T} E={E} K={K} seq_len={n} masked={masked}", flush=True)
    l, idx, mask, _, _ = _case(T, E, K, masked, T + E)
    for m in (mask, None):
        d, b = _forward(l, idx, m, n, guard=64)
        S = -(-T // n)
        _check_forward(b, TO.balance(l, idx, m, n, E, K), l, m, S, E)
        for t, used in ((b.counts, S * E), (b.tokens, S + 2), (b.probs, S * E), (b.loss, 2)):
            assert (host(t)[used:] == 7).all()           # nothing behind the outputs


def _backward(d, n, l, mask, counts, tokens, dloss, route, out=None):
    out = torch.full_like(l, 7.0) if out is None else out
    dw, w, idx = route if route is not None else (None, None, None)
    M.moe_balance_bwd(d, n, l, mask, counts, tokens, dloss, dw, w, idx, out)
    torch.cuda.synchronize()
    return out


def _check_gradient(got, ref, l, mask, counts, tokens, dloss, E, K, route):
    """Every term of p (q - sum p q + r lse) is off by (span + 16 + E) EPS of its size: p as above, the sum
    of up to E non-negative terms, lse by (|lse| + 4) EPS; the picks' part by (K + 4) EPS of its terms."""
    n = np.maximum(tokens[:-2].astype(np.float64), 1)
    used = mask.astype(bool) if mask is not None else np.ones(len(l), bool)
    p, lse = TO.softmax_rows(l)
    q = (abs(dloss[0]) * E / (K * n ** 2 * max(tokens[-1], 1)))[:, None] * counts
    q = q[np.arange(len(l)) // route["seq_len"]]
    r = abs(dloss[1]) * 2 / max(tokens[-2], 1)
    size = p * (q + (p * q).sum(1, keepdims=True) + r * (np.abs(lse) + np.abs(l).max(1) + 4)[:, None])
    bound = EPS * (np.ptp(l, axis=1).max() + 16 + E) * size * used[:, None]
    if route["on"]:
        w, dw = np.abs(route["w"].astype(np.float64)), np.abs(route["dw"].astype(np.float64))
        part = w * (dw + (w * dw).sum(1, keepdims=True)) * EPS * (K + 4)
        for t in range(len(l)):
            for k, e in enumerate(route["idx"][t]):
                bound[t, e] += part[t, k] + 2 * EPS * abs(ref[t, e])
    assert np.all(np.abs(got - ref) <= bound + 1e-37)


@pytest.mark.parametrize("T,E,K,n,masked", SHAPES)
def test_gradient(T, E, K, n, masked):
    print(f"case balance_bwd T={T} E={E} K={K} seq_len={n} masked={masked}", flush=True)
    l, idx, mask, w, dw = _case(T, E, K, masked, 3 * T + E)
    dloss = np.array([0.4, -0.3], np.float32)
    for m in (mask, None):
        d, b = _forward(l, idx, m, n)
        ref = TO.balance(l, idx, m, n, E, K)
        dev = [_cuda(a) for a in (l, m, dloss, dw, w, idx)]
        for on in (False, True):
            got = host(_backward(d, n, dev[0], dev[1], b.counts, b.tokens, dev[2], dev[3:] if on else None))
            want = TO.balance_bwd(l, m, n, E, K, ref["counts"], ref["tokens"], dloss, (dw, w, idx) if on else None)
            _check_gradient(got, want, l, m, ref["counts"], ref["tokens"], dloss, E, K,
                            dict(on=on, w=w, dw=dw, idx=idx, seq_len=n))


def test_gradient_is_the_kernels_own_difference():
    """Central differences of the losses that the forward kernel gives, along random directions.  The losses
    are float32 (half a step of about 1 and 10), the step is 2^-6 and the third derivatives are below 50, so the
    quotient is within 2 * 10 * EPS / 2^-6 + 50 / 6 * 2^-12 of the slope, with norms of 1 along the direction."""
    T, E, K, n = 96, 8, 2, 40
    l, idx, mask, _, _ = _case(T, E, K, 0.2, 11)
    d, b = _forward(l, idx, mask, n)
    for which in (0, 1):
        dl = np.zeros(2, np.float32)
        dl[which] = 1
        grad = host(_backward(d, n, _cuda(l), _cuda(mask), b.counts, b.tokens, _cuda(dl), None)).astype(np.float64)
        for seed in range(4):
            v = np.random.default_rng(seed).standard_normal((T, E))
            v /= np.linalg.norm(v)
            h = 2.0 ** -6
            up, dn = ((l + s * h * v).astype(np.float32) for s in (1, -1))
            real = (up.astype(np.float64) - dn) / (2 * h)
            lo = [host(_forward(x, idx, mask, n)[1].loss)[which].astype(np.float64) for x in (up, dn)]
            assert abs((lo[0] - lo[1]) / (2 * h) - (grad * real).sum()) <= 2 * 10 * EPS / h + 50 / 6 * h * h


def test_route_part_is_route_bwd():
    """With both losses' gradients 0 the call gives moe_route_bwd's values (which side rounds a product is
    left open: half a step of each term)."""
    T, E, K = 777, 60, 6
    l, idx, mask, w, dw = _case(T, E, K, 0.0, 5)
    d, b = _forward(l, idx, None, T)
    dev = [_cuda(a) for a in (dw, w, idx)]
    want = torch.empty(T, E, device="cuda")
    M.moe_route_bwd(d, *dev, want)
    got = _backward(d, T, _cuda(l), None, b.counts, b.tokens, torch.zeros(2, device="cuda"), dev)
    big = (np.abs(w) * (np.abs(dw) + np.abs(w * dw).sum(1, keepdims=True))).max()
    assert np.max(np.abs(host(got) - host(want))) <= 2 * (K + 2) * EPS * big


@pytest.mark.parametrize("E", [8, 30, 64, 256])
def test_padding_may_hold_anything(E):
    """NaN, infinities and the lowest float in padded rows: the other rows' results keep their bits."""
    T, K, n = 700, 2, 300
    l, idx, mask, w, dw = _case(T, E, K, 0.4, 21)
    bad = l.copy()
    rows = np.flatnonzero(mask == 0)
    for i, v in enumerate([np.nan, np.inf, -np.inf, np.finfo(np.float32).min]):
        bad[rows[i::4]] = v
    bad[rows[::5], 0] = np.nan
    idx_bad = idx.copy()
    idx_bad[rows] = -5
    d, a = _forward(l, idx, mask, n)
    _, b = _forward(bad, idx_bad, mask, n)
    dloss = torch.tensor([0.5, 0.5], device="cuda")
    for name in ("counts", "tokens", "probs", "loss"):
        assert np.array_equal(host(getattr(a, name)), host(getattr(b, name))), name
    ga = host(_backward(d, n, _cuda(l), _cuda(mask), a.counts, a.tokens, dloss, None))
    gb = host(_backward(d, n, _cuda(bad), _cuda(mask), a.counts, a.tokens, dloss, None))
    assert np.array_equal(ga, gb) and (gb[rows] == 0).all()


def test_batches_without_tokens():
    T, E, K, n = 130, 8, 2, 50
    l, idx, _, w, dw = _case(T, E, K, 0.0, 2)
    for mask in (np.zeros(T, np.uint8), (np.arange(T) >= 50).astype(np.uint8)):   # none at all; none in the first sequence
        d, b = _forward(l, idx, mask, n)
        ref = TO.balance(l, idx, mask, n, E, K)
        _check_forward(b, ref, l, mask, 3, E)
        dev = [_cuda(a) for a in (dw, w, idx)]
        got = host(_backward(d, n, _cuda(l), _cuda(mask), b.counts, b.tokens, torch.ones(2, device="cuda"), dev))
        want = TO.balance_bwd(l, mask, n, E, K, ref["counts"], ref["tokens"], np.ones(2), (dw, w, idx))
        _check_gradient(got, want, l, mask, ref["counts"], ref["tokens"], np.ones(2), E, K,
                        dict(on=True, w=w, dw=dw, idx=idx, seq_len=n))
        if not mask.any():
            assert (host(b.loss) == 0).all()


def test_masked_experts_and_bad_rows():
    """A logit of -inf takes its expert out; a row of only -inf makes its own sequence's sums NaN, no other's."""
    T, E, K, n = 200, 16, 2, 100
    l, idx, _, _, _ = _case(T, E, K, 0.0, 9)
    l[:, 3] = -np.inf
    idx = np.argsort(-l, 1, kind="stable")[:, :K].astype(np.int32)
    d, b = _forward(l, idx, None, n)
    with np.errstate(invalid="ignore"):
        ref = TO.balance(l, idx, None, n, E, K)
    finite = l.copy()
    finite[:, 3] = l[:, :3].min()
    _check_forward(b, ref, finite, None, 2, E)
    got = host(_backward(d, n, _cuda(l), None, b.counts, b.tokens, torch.ones(2, device="cuda"), None))
    assert (got[:, 3] == 0).all() and np.isfinite(got).all()
    l[150] = -np.inf
    d, b = _forward(l, idx, None, n)
    probs = host(b.probs)
    assert np.isnan(probs[1]).all() and np.isfinite(probs[0]).all() and np.isnan(host(b.loss)).all()


def test_bits_do_not_depend_on_the_run_and_ids_outside_are_skipped():
    T, E, K, n = 5000, 48, 4, 2048
    l, idx, mask, w, dw = _case(T, E, K, 0.1, 31)
    idx[::7, 1] = E
    idx[::11, 0] = -1
    d, a = _forward(l, idx, mask, n)
    ref = TO.balance(l, idx, mask, n, E, K)
    _check_forward(a, ref, l, mask, 3, E)
    for _ in range(5):
        _, b = _forward(l, idx, mask, n)
        for name in ("counts", "tokens", "probs", "loss"):
            assert np.array_equal(host(getattr(a, name)), host(getattr(b, name))), name
    got = host(_backward(d, n, _cuda(l), _cuda(mask), a.counts, a.tokens, torch.ones(2, device="cuda"),
                         [_cuda(x) for x in (dw, w, idx)]))
    want = TO.balance_bwd(l, mask, n, E, K, ref["counts"], ref["tokens"], np.ones(2), (dw, w, idx))
    assert np.max(np.abs(got - want)) <= 64 * EPS * np.abs(want).max()


def test_gradient_in_place_of_the_logits():
    for E in (7, 32, 200):
        T, K, n = 333, 2, 100
        l, idx, mask, w, dw = _case(T, E, K, 0.2, 41)
        d, b = _forward(l, idx, mask, n)
        dev = [_cuda(x) for x in (dw, w, idx)]
        dloss = torch.tensor([0.1, 0.2], device="cuda")
        want = _backward(d, n, _cuda(l), _cuda(mask), b.counts, b.tokens, dloss, dev)
        x = _cuda(l)
        _backward(d, n, x, _cuda(mask), b.counts, b.tokens, dloss, dev, out=x)
        assert torch.equal(x, want)


def test_bool_mask_and_streams():
    T, E, K, n = 3000, 32, 4, 3000
    l, idx, mask, _, _ = _case(T, E, K, 0.3, 51)
    _, a = _forward(l, idx, mask, n)
    s, logits, picks, m = torch.cuda.Stream(), _cuda(l), _cuda(idx), _cuda(mask).bool()
    b = L.BalanceBuffers(a.d, n)
    torch.cuda.synchronize()
    L.balance(b, logits, picks, m, stream=s)             # a stream by argument
    c = L.BalanceBuffers(a.d, n)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):                           # the current one
        L.balance(c, logits, picks, m)
    torch.cuda.synchronize()
    for x in (b, c):
        assert torch.equal(x.probs, a.probs) and torch.equal(x.loss, a.loss) and torch.equal(x.counts, a.counts)


def test_captured_step_replays():
    """Losses and gradient in a graph, replayed with other inputs in the same buffers and eager work between."""
    T, E, K, n = 4000, 64, 6, 1500
    d = L.make_dims(T, 8, E, K, 8)
    b = L.BalanceBuffers(d, n)
    cases = [_case(T, E, K, 0.1, 60 + i) for i in range(3)]
    l, idx, mask, w, dw = (_cuda(a) for a in cases[0])
    dloss = torch.tensor([0.3, 0.2], device="cuda")
    out = torch.empty_like(l)

    def step():
        L.balance(b, l, idx, mask)
        M.moe_balance_bwd(d, n, l, mask, b.counts, b.tokens, dloss, dw, w, idx, out)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in (0, 1, 2, 1):
        for t, a in zip((l, idx, mask, w, dw), cases[i]):
            t.copy_(_cuda(a))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (b.loss, b.counts, b.probs, b.tokens, out)]
        for t in (b.loss, b.probs, out):
            t.fill_(3.0)
        b.ws.fill_(0x5A)
        g.replay()
        torch.cuda.synchronize()
        for t, x in zip((b.loss, b.counts, b.probs, b.tokens, out), want):
            assert torch.equal(t, x)


def test_gradient_over_the_tokens_of_two_ranks():
    """Two halves of a batch, each with the counts and tokens of both, give the rows of the whole batch's
    gradient (same arithmetic for a row: same bits)."""
    T, E, K = 1200, 24, 3
    l, idx, mask, w, dw = _case(T, E, K, 0.2, 71)
    d, b = _forward(l, idx, mask, T)
    dloss = torch.tensor([0.4, 0.3], device="cuda")
    want = _backward(d, T, _cuda(l), _cuda(mask), b.counts, b.tokens, dloss, [_cuda(x) for x in (dw, w, idx)])
    cut = 500
    halves = [slice(0, cut), slice(cut, T)]
    ranks = [_forward(l[h], idx[h], mask[h], len(l[h])) for h in halves]
    counts = ranks[0][1].counts + ranks[1][1].counts
    tokens = ranks[0][1].tokens + ranks[1][1].tokens
    tokens[2] = 1
    assert torch.equal(counts, b.counts) and torch.equal(tokens, b.tokens)
    for h, (dr, _) in zip(halves, ranks):
        got = _backward(dr, dr.T, _cuda(l[h]), _cuda(mask[h]), counts, tokens, dloss, [_cuda(x[h]) for x in (dw, w, idx)])
        assert torch.equal(got, want[h])


def test_two_calls_at_once():
    """Two batches on two streams, each with its own buffers."""
    cases = [_case(3000, 32, 4, 0.1, 81), _case(2500, 100, 6, 0.3, 82)]
    want = [_forward(l, i, m, 700)[1] for l, i, m, _, _ in cases]
    dev = [[_cuda(a) for a in c[:3]] for c in cases]
    bufs = [L.BalanceBuffers(b.d, 700) for b in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, (l, i, m), s in zip(bufs, dev, streams):
            L.balance(b, l, i, m, stream=s)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        for n in ("counts", "tokens", "probs", "loss"):
            assert torch.equal(getattr(b, n), getattr(w, n)), n


def test_a_layer_step_with_losses():
    """forward, losses, backward of a whole layer: dlogits is route_bwd's plus the losses' gradient, and
    everything else keeps its bits."""
    cfg = custom_config(300, 64, 6, 2, 96)
    inp = synth.make_inputs(cfg)
    p = device_inputs(inp)
    d = L.make_dims(cfg.T, cfg.H, cfg.E, cfg.K, cfg.I)
    b = L.Buffers(d)
    L.forward(b, p, fused=True)
    L.backward(b, p, fused=True)
    torch.cuda.synchronize()
    before = {n: getattr(b, n).clone() for n in ("dx", "dw1", "dw2", "dlogits", "topk_idx", "counts")}
    mask = (np.arange(cfg.T) % 5 != 0).astype(np.uint8)
    p["mask"], p["dloss"] = _cuda(mask), torch.tensor([0.2, 0.1], device="cuda")
    losses = L.BalanceBuffers(d, 128)
    L.forward(b, p, fused=True)
    L.balance(losses, p["logits"], b.topk_idx, p["mask"])
    L.backward(b, p, fused=True, losses=losses)
    L.check()
    for n in ("dx", "dw1", "dw2", "topk_idx", "counts"):
        assert torch.equal(getattr(b, n), before[n]), n
    l, idx = host(p["logits"]), host(b.topk_idx)
    ref = TO.balance(l, idx, mask, 128, cfg.E, cfg.K)
    want = TO.balance_bwd(l, mask, 128, cfg.E, cfg.K, ref["counts"], ref["tokens"], np.array([0.2, 0.1], np.float32))
    want = want + host(before["dlogits"])
    assert np.max(np.abs(host(b.dlogits) - want)) <= 64 * EPS * max(1.0, np.abs(want).max())


def test_backward_of_a_layer_takes_the_mask_of_its_losses():
    """The mask is given once; padding gets no gradient of the losses, and a later call without one has none.
    w (dw - sum w dw) of two picks, w <= 1: 2 roundings of the sum, 2 of the difference and 2 of the product
    at most of size max |dw|, on either side; the losses' gradient of a token is 1e-4 and more."""
    cfg = custom_config(100, 64, 6, 2, 96)
    p = device_inputs(synth.make_inputs(cfg))
    d = L.make_dims(cfg.T, cfg.H, cfg.E, cfg.K, cfg.I)
    b, losses = L.Buffers(d), L.BalanceBuffers(d)
    L.forward(b, p, fused=True)
    L.backward(b, p, fused=True)
    torch.cuda.synchronize()
    plain = b.dlogits.clone()
    mask = torch.arange(cfg.T, device="cuda") % 3 != 0
    p["dloss"] = torch.tensor([0.2, 0.1], device="cuda")
    for m in (mask, None):
        L.balance(losses, p["logits"], b.topk_idx, m)
        L.backward(b, p, fused=True, losses=losses)
        L.check()
        same = (b.dlogits - plain).abs().amax(1) <= 12 * EPS * b.dtopk_w.abs().amax(1)
        assert torch.equal(same, torch.zeros_like(same) if m is None else ~mask)
