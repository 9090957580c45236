"""Newton-Schulz products and the update of stacked weights (moe_orthogonalize, moe_muon) against float64.

Bounds.  The kernels' arithmetic is documented (fp16 factors in one or two parts, X in two, float32
sums); train_oracle.newton_model repeats it in numpy.  The two differ by the order of the float32 sums
and by single roundings only, so the kernels may be off float64 by twice what the model is, plus the
rounding of the result (2^-9 of it for bf16, 2^-24 for float32) and, in the exact form, 2^-20 for the sums'
order in small models that happen to be nearly exact."""
import numpy as np
import pytest
import torch

import combine_moe_route_histogram_amd as M
from combine_moe_route_histogram_amd import layer as L
from gpu_util import custom_config, device_inputs, host
from oracle import train_oracle as TO
import synth

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": M.BF16, "f32": M.F32}

SHAPES = [  # G, R, C
    (1, 1, 1), (2, 1, 8), (2, 8, 1), (3, 7, 5), (1, 64, 64), (2, 65, 63), (1, 63, 66), (1, 130, 257), (2, 257, 130),
    (5, 128, 256), (1, 3, 4000), (1, 4001, 3), (2, 512, 1000), (1, 1030, 300), (1, 700, 701), (300, 16, 24),
    (260, 70, 40), (2049, 8, 8), (2051, 3, 5), (40, 520, 264),
]


def _grad(G, R, C, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((G, R, C)) * np.exp(0.5 * g.standard_normal((G, R, 1))) * np.exp(0.5 * g.standard_normal((G, 1, C)))
    return (1e-3 * x).astype(np.float32)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _ws(G, R, C, dtype, guard=0):
    n = M.moe_muon_workspace_bytes(G, R, C, CODE[dtype])
    return torch.full((n + guard,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN in every format


def _ortho(x, dtype, coef=None, stream=None):
    G, R, C = x.shape
    ws = _ws(G, R, C, dtype, 256)
    out = torch.full((G * R * C + 64,), 7.0, dtype=DT[dtype], device="cuda")
    src = _dev(x)
    M.moe_orthogonalize(G, R, C, src, out, ws[:-256], coef=coef, stream=stream)
    torch.cuda.synchronize()
    assert np.array_equal(host(src), x, equal_nan=True)
    assert (ws[-256:] == 0xFF).all() and (out[G * R * C:] == 7).all()        # nothing behind either
    return out[:G * R * C].view(G, R, C).float().cpu().numpy().astype(np.float64)


def _exact(x, dtype):
    return dtype == "f32" or min(x.shape[-2:]) < 32      # as documented


def _check(got, x, dtype, coef=TO.COEF, what=""):
    ref, model = TO.newton(x, coef), TO.newton_model(x, _exact(x, dtype), coef)
    norm = np.linalg.norm(ref)
    off, model_off = np.linalg.norm(got - ref), np.linalg.norm(model - ref)
    rounding = 2.0 ** -9 if dtype == "bf16" else 2.0 ** -20
    assert off <= 2 * model_off + rounding * norm, (what, off / norm, model_off / norm)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,R,C", SHAPES)
def test_orthogonalize(G, R, C, dtype):
    print(f"case orthogonalize G={G} R={R} C={C} {dtype}", flush=True)
    x = _grad(G, R, C, G + R + C)
    got = _ortho(x, dtype)
    for g in {0, G // 2, G - 1}:
        _check(got[g], x[g], dtype, what=f"matrix {g}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,R,C", [(3, 700, 1500), (4, 2100, 400), (60, 500, 520), (61, 400, 330), (1, 1410, 1400), (1, 100, 9000)])
def test_orthogonalize_with_products_of_different_tiles(G, R, C, dtype):
    """Stacks whose first two products take other tiles than the third, or all the largest."""
    print(f"case orthogonalize G={G} R={R} C={C} {dtype}", flush=True)
    x = _grad(G, R, C, G + R + C)
    got = _ortho(x, dtype)
    for g in {0, G - 1}:
        _check(got[g], x[g], dtype, what=f"matrix {g}")


COEF32 = tuple(tuple(float(np.float32(v)) for v in abc) for abc in TO.COEF)   # as the kernels hold them


def _check_few(got, x, dtype, coef=COEF32, what=""):
    """In 64 bits up to the result: half a step of it, and of float32 on the way to bf16."""
    ref = TO.newton(x, coef)
    step = 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -26)     # eps / 2 of 8 and of 24 bits
    assert np.linalg.norm(got - ref) <= step * np.linalg.norm(ref), (what, np.linalg.norm(got - ref) / np.linalg.norm(ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,R,C", [(1, 1, 1), (2, 1, 9), (3, 15, 17), (2, 16, 4001), (2, 4001, 17), (3, 33, 31), (5, 32, 64),
                                   (2, 48, 129), (3, 1000, 47), (2, 64, 2048), (1, 2111, 49), (1030, 40, 20), (4100, 3, 5)])
def test_few_rows_are_as_exact_as_the_result(G, R, C, dtype):
    print(f"case few rows G={G} R={R} C={C} {dtype}", flush=True)
    x = _grad(G, R, C, G + R + C)
    got = _ortho(x, dtype, COEF32)
    for g in {0, G // 2, G - 1}:
        _check_few(got[g], x[g], dtype, what=f"matrix {g}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_rows_of_low_rank_and_of_other_iterations(dtype):
    """Null directions under coefficients that make them up to 4096 times larger; zeros, infinities and scales; and
    more steps than the form for few rows takes, which are worked on like larger matrices."""
    g = np.random.default_rng(4)
    for R, C in ((20, 300), (300, 41)):
        x = np.stack([(g.standard_normal((R, r)) @ g.standard_normal((r, C))).astype(np.float32) for r in (1, 4, 16)])
        for coef in (COEF32, ((1.5, -0.5, 0.0),) * 16, ((1.875, -1.25, 0.375),) * 13, ((32.0, -30.0, 0.0), (32.0, 0.0, 0.0), (4.0, 1.0, 0.5))):
            got = _ortho(x, dtype, coef)
            for i in range(3):
                _check_few(got[i], x[i], dtype, coef, what=str(coef))
        for e in (-140, 100):
            y = np.ldexp(np.sign(x), e).astype(np.float32)
            assert np.array_equal(_ortho(y, dtype), _ortho(np.sign(x), dtype))
        bad = x.copy()
        bad[0], bad[1, 3, 4] = 0, -np.inf
        got = _ortho(bad, dtype, COEF32)
        assert (got[0] == 0).all() and np.isnan(got[1]).all()
        _check_few(got[2], x[2], dtype)
        long = TO.COEF[:1] * 6 + ((1.5, -0.5, 0.0),) * 4       # 3.44^6 1.5^4 = 8455
        got = _ortho(x, dtype, long)
        for i in range(3):
            _check(got[i], x[i], dtype, long)


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,R,C", [(3, 45, 500), (2, 1201, 37), (1, 64, 2100), (1, 2500, 50), (2060, 9, 6)])
def test_muon_steps_of_few_rows(G, R, C, dtype, nesterov):
    """mom: two roundings a step.  master: three, and lr scale times half a step of the update.  The direction
    is rounded twice (grad + momentum mom by one fma, of mom's own): 2^-23 of its norm, which the iteration makes larger by
    at most 485 / 1 of null directions; its part there is below that of 485 2^-23."""
    print(f"case muon of few rows G={G} R={R} C={C} {dtype} nesterov={nesterov}", flush=True)
    grads, mom0, w0, mom, master, w = _muon(G, R, C, dtype, nesterov)
    for g in sorted({0, G // 2, G - 1}):
        m, x = mom0[g:g + 1].astype(np.float64), w0[g:g + 1].astype(np.float64)
        allowed, big = 0.0, np.abs(mom0[g]) + sum(np.abs(gr[g]) for gr in grads)
        for gr in grads:
            m, x, o = TO.muon(gr[g:g + 1], m, x, **HYPER, nesterov=nesterov)
            allowed += HYPER["lr"] * HYPER["scale"] * (2.0 ** -23 * np.linalg.norm(o) + 485 * 2.0 ** -23)
            allowed += 3 * 2.0 ** -24 * np.linalg.norm(x)
        assert np.all(np.abs(host(mom[g]).astype(np.float64) - m[0]) <= 4 * 2.0 ** -24 * big)
        assert np.linalg.norm(host(master[g]).astype(np.float64) - x[0]) <= allowed
    if w is not None:
        assert torch.equal(w, master.to(torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_low_rank(dtype):
    """Gradients of experts with few tokens: null directions must not gather roundings."""
    g = np.random.default_rng(2)
    for R, C in ((200, 300), (300, 200)):
        x = np.stack([(g.standard_normal((R, r)) @ g.standard_normal((r, C))).astype(np.float32) for r in (1, 4, 16, 100)])
        got = _ortho(x, dtype)
        for i in range(4):
            _check(got[i], x[i], dtype, what=f"rank {(1, 4, 16, 100)[i]}")
            if dtype == "bf16":
                ref = TO.newton(x[i])
                assert np.linalg.norm(got[i] - ref) <= 5e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_iterations(dtype):
    """Coefficients and numbers of steps of the caller's: one, sixteen, a cubic, other ones in every step."""
    x = _grad(2, 100, 180, 7)
    cubic = (1.5, -0.5, 0.0)
    for coef in ((cubic,), (cubic,) * 16, ((1.875, -1.25, 0.375),) * 3, ((3.4445, -4.7750, 2.0315),) * 2 + (cubic,) * 3):
        got = _ortho(x, dtype, coef)
        for g in range(2):
            _check(got[g], x[g], dtype, coef, what=str(len(coef)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_largest_singular_values(dtype):
    """A step that leaves a singular value of 15, the largest documented, and ones that bring it back; the last
    step may leave any."""
    g = np.random.default_rng(9)
    x = (g.standard_normal((1, 90, 1)) @ g.standard_normal((1, 1, 150))).astype(np.float32)
    for coef in (((15.0, 0.0, 0.0), (1.5, -0.5 / 225, 0.0)), ((15.0, 0.0, 0.0), (32.0, 0.0, 0.0))):
        got = _ortho(x, dtype, coef)
        assert np.isfinite(got).all()
        _check(got[0], x[0], dtype, coef)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scale_has_no_effect(dtype):
    """Powers of two, down to subnormal entries and up to the largest, leave the bits."""
    x = np.sign(_grad(1, 90, 150, 3)) * (1 + np.random.default_rng(1).integers(0, 8, (1, 90, 150)) / 8)
    want = _ortho(x.astype(np.float32), dtype)
    for e in (-140, -100, -40, 40, 100, 126):
        y = np.ldexp(x, e).astype(np.float32)
        if e == -140:
            assert np.all(np.abs(y) < 2.0 ** -126)       # subnormal and exact
        assert np.array_equal(_ortho(y, dtype), want), e


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", [(70, 130), (130, 70)])
def test_zeros_and_non_finite_matrices(R, C, dtype):
    """Zeros give zeros; an infinity or NaN makes its own matrix NaN and leaves the others' bits."""
    x = _grad(6, R, C, 4)
    want = _ortho(x, dtype)
    bad = x.copy()
    bad[1] = 0
    bad[3, 2, 5] = np.inf
    bad[4, R - 1, C - 1] = np.nan
    got = _ortho(bad, dtype)
    assert (got[1] == 0).all() and np.isnan(got[3]).all() and np.isnan(got[4]).all()
    for g in (0, 2, 5):
        assert np.array_equal(got[g], want[g])


def test_bits_repeat_and_do_not_depend_on_the_others():
    """The same stack again, and the same matrix among others, in stacks of few and of many matrices."""
    for G, R, C in ((3, 90, 70), (300, 90, 70), (40, 300, 200)):
        x = _grad(G, R, C, 12)
        other = _grad(G, R, C, 13)
        other[G // 2] = x[G // 2]
        for dtype in ("bf16", "f32"):
            a, b = _ortho(x, dtype), _ortho(x, dtype)
            assert np.array_equal(a, b)
            assert np.array_equal(_ortho(other, dtype)[G // 2], a[G // 2])


HYPER = dict(lr=0.02, momentum=0.9, weight_decay=0.1, scale=2.0)


def _muon(G, R, C, dtype, nesterov, steps=2, lr=None, seed=0):
    rng = np.random.default_rng(seed)
    grads = [_grad(G, R, C, seed + 10 + k) for k in range(steps)]
    mom0 = 2 * _grad(G, R, C, seed + 1)
    w0 = (0.02 * rng.standard_normal((G, R, C))).astype(np.float32)
    mom, master, ws = _dev(mom0), _dev(w0), _ws(G, R, C, dtype)
    w = torch.full((G, R, C), 9.0, dtype=torch.bfloat16, device="cuda") if dtype == "bf16" else None
    hyper = dict(HYPER) if lr is None else dict(HYPER, lr=lr)
    for g in grads:
        src = _dev(g)
        M.moe_muon(G, R, C, src, mom, master, w, ws, nesterov=nesterov, **hyper)
        assert torch.equal(src, _dev(g))
    torch.cuda.synchronize()
    return grads, mom0, w0, mom, master, w


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,R,C", [(1, 1, 1), (2, 5, 9), (3, 64, 72), (2, 130, 70), (2, 257, 511), (1, 301, 1000),
                                   (257, 24, 40), (2049, 8, 4)])
def test_muon_steps(G, R, C, dtype, nesterov):
    """Two steps.  mom: two roundings a step.  master: three roundings a step, and lr scale times the
    error of the update (bounded as above, without the rounding to bf16).  w: the rounded master."""
    print(f"case muon G={G} R={R} C={C} {dtype} nesterov={nesterov}", flush=True)
    grads, mom0, w0, mom, master, w = _muon(G, R, C, dtype, nesterov)
    m, x = mom0.astype(np.float64), w0.astype(np.float64)
    picked = sorted({0, G // 2, G - 1})
    for g in picked:
        mg, xg, allowed = m[g:g + 1], x[g:g + 1], 0.0
        for gr in grads:
            mg, xg, o = TO.muon(gr[g:g + 1], mg, xg, **HYPER, nesterov=nesterov)
            u = gr[g].astype(np.float64) + HYPER["momentum"] * mg[0] if nesterov else mg[0]
            model = TO.newton_model(u, _exact(u, dtype))
            allowed += HYPER["lr"] * HYPER["scale"] * (2 * np.linalg.norm(model - o[0]) + 2.0 ** -20 * np.linalg.norm(o[0]))
            allowed += 3 * 2.0 ** -24 * np.linalg.norm(xg)
        got_m, got_x = host(mom[g]).astype(np.float64), host(master[g]).astype(np.float64)
        big = np.abs(mom0[g]) + sum(np.abs(gr[g]) for gr in grads)
        assert np.all(np.abs(got_m - mg[0]) <= 4 * 2.0 ** -24 * big)
        assert np.linalg.norm(got_x - xg[0]) <= allowed
    if w is not None:
        assert torch.equal(w, master.to(torch.bfloat16))


def test_learning_rate_on_the_device():
    for dtype in ("bf16", "f32"):
        a = _muon(2, 40, 70, dtype, True, lr=0.01)
        b = _muon(2, 40, 70, dtype, True, lr=torch.tensor([0.01], device="cuda"))
        assert torch.equal(a[4], b[4]) and torch.equal(a[3], b[3])


def test_streams_and_two_calls_at_once():
    """Two stacks on two streams, each with its own workspace, against one after the other."""
    xs = [_grad(3, 300, 500, 1), _grad(2, 500, 260, 2)]
    want = [_ortho(x, "bf16") for x in xs]
    src = [_dev(x) for x in xs]
    outs = [torch.empty(x.shape, dtype=torch.bfloat16, device="cuda") for x in xs]
    wss = [_ws(*x.shape, "bf16") for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, s, o, w, st in zip(xs, src, outs, wss, streams):
            M.moe_orthogonalize(*x.shape, s, o, w, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.float().cpu().numpy().astype(np.float64), w)


def test_captured_update_replays():
    """A captured step with its learning rate on the device, replayed on new gradients, with eager work between."""
    G, R, C = 2, 200, 330
    grads = [_grad(G, R, C, 70 + k) for k in range(3)]
    w0 = (0.02 * np.random.default_rng(0).standard_normal((G, R, C))).astype(np.float32)
    lrs = (0.02, 0.01, 0.0)

    def fresh():
        return dict(grad=_dev(grads[0]), mom=torch.zeros(G, R, C, device="cuda"), master=_dev(w0),
                    w=torch.zeros(G, R, C, dtype=torch.bfloat16, device="cuda"), lr=torch.zeros(1, device="cuda"),
                    ws=_ws(G, R, C, "bf16"))

    def step(s):
        M.moe_muon(G, R, C, s["grad"], s["mom"], s["master"], s["w"], s["ws"], lr=s["lr"], momentum=0.9, weight_decay=0.1,
                   scale=2.0)
    eager, held = fresh(), fresh()
    step(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held)
    held["mom"].zero_()
    held["master"].copy_(_dev(w0))
    for g, lr in zip(grads, lrs):
        for s in (eager, held):
            s["grad"].copy_(_dev(g))
            s["lr"].fill_(lr)
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("mom", "master", "w"):
            assert torch.equal(eager[n], held[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_training_step_of_a_layer(dtype):
    """forward, losses, backward and the update of every weight, shared experts among them, with the calls a
    program makes; an expert without tokens keeps its weights but for the decay."""
    cfg = custom_config(64, 64, 6, 2, 96, Ns=1, dtype=dtype)
    inp = synth.make_inputs(cfg)
    inp["logits"][:, 5] = -50.0                          # nobody picks expert 5
    p = device_inputs(inp)
    p["dloss"] = torch.tensor([0.01, 0.001], device="cuda")
    d = L.make_dims(cfg.T, cfg.H, cfg.E, cfg.K, cfg.I, cfg.n_shared, dtype)
    b, losses, m = L.Buffers(d), L.BalanceBuffers(d, 16), L.MuonState(p)
    assert m.names == list(L.WEIGHTS)
    old = {n: p[n].float().clone() for n in m.names}
    for _ in range(2):
        L.forward(b, p, fused=True)
        L.balance(losses, p["logits"], b.topk_idx)
        L.backward(b, p, fused=True, losses=losses)
        L.muon_step(m, p, b, lr=0.01, weight_decay=0.5)
    L.check()
    for n in m.names:
        moved = m.master[n] - old[n]
        assert torch.isfinite(moved).all()
        if dtype == "bf16":
            assert torch.equal(p[n], m.master[n].to(torch.bfloat16))
        else:
            assert p[n].data_ptr() == m.master[n].data_ptr()
        # 0.2 lr a step and entry on average, the first steps' directions nearly alike
        rms = float(moved[:5].square().mean().sqrt())
        assert 0.2 * 0.01 * 0.3 < rms < 2 * 0.2 * 0.01 * 1.5 + 0.01 * 0.5 * 2 * float(old[n].abs().max())
    for n in ("w1", "w3", "w2"):
        kept = old[n][5].double() * (1 - 0.01 * 0.5) ** 2
        assert torch.allclose(m.master[n][5].double(), kept, rtol=4 * 2.0 ** -24, atol=0)


def _large_last_step(G, R, C, seed):
    """One row that is not zero, rank one, full rank, in turn."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((G, R, C)).astype(np.float32)
    for i in range(0, G, 3):
        x[i] = 0
        x[i, R // 3] = g.standard_normal(C)
        if i + 1 < G:
            x[i + 1] = np.outer(g.standard_normal(R), g.standard_normal(C))
    return x


def _check_result(got, x, dtype, coef, what):
    """As _check, with half a step of a result in bf16 (2^-8) for each element."""
    ref, model = TO.newton(x, coef), TO.newton_model(x, _exact(x, dtype), coef)
    rounding = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20
    allowed = 2 * np.linalg.norm(model - ref) + rounding * np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= allowed, (what, np.linalg.norm(got - ref), allowed)


LARGE_LAST = (((2.0, 0.0, 0.0), (1.0, 0.0, 20.0)), ((15.0, 0.0, 0.0), TO.COEF[0]), ((15.0, 0.0, 0.0), (32.0, 32.0, 32.0)),
              ((15.0, 0.0, 0.0), (-32.0, 32.0, -32.0)), ((3.0, -1.0, 0.0), (4.0, 0.75, 0.0), (2.0, 32.0, 32.0)), ((32.0, 32.0, 32.0),))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,R,C", [(3, 90, 150), (3, 150, 90), (40, 520, 264)])
def test_last_step_may_leave_any_singular_value(G, R, C, dtype):
    """Steps that leave singular values of 2 to 15, and last ones whose B = a + b s^2 + c s^4 is 321 to 1.6e6: beyond what
    fp16 holds at the scale of the other steps' B.  Small and large tiles, both orientations."""
    print(f"case large last step G={G} R={R} C={C} {dtype}", flush=True)
    x = _large_last_step(G, R, C, R)
    for coef in LARGE_LAST:
        got = _ortho(x, dtype, coef)
        assert np.isfinite(got).all(), coef
        for g in range(3):
            _check_result(got[g], x[g], dtype, coef, f"matrix {g} of {coef}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_update_by_a_last_step_that_leaves_large_singular_values(dtype):
    """As above, into the weights: master is off by lr scale times the update's error (bounded as in _check_result, without the
    result's rounding) and three roundings of its own."""
    G, R, C = 3, 90, 150
    x, coef = _large_last_step(G, R, C, 5), LARGE_LAST[1]
    w0 = (0.02 * np.random.default_rng(6).standard_normal((G, R, C))).astype(np.float32)
    mom, master, ws = torch.zeros(G, R, C, device="cuda"), _dev(w0), _ws(G, R, C, dtype)
    w = torch.empty(G, R, C, dtype=torch.bfloat16, device="cuda") if dtype == "bf16" else None
    hyper = dict(lr=1e-4, momentum=0.0, weight_decay=0.1, scale=1.0)
    M.moe_muon(G, R, C, _dev(x), mom, master, w, ws, nesterov=False, coef=coef, **hyper)
    torch.cuda.synchronize()
    assert torch.isfinite(master).all()
    _, want, o = TO.muon(x, np.zeros_like(x), w0, nesterov=False, coef=coef, **hyper)
    for g in range(G):
        off = np.linalg.norm(TO.newton_model(x[g], dtype == "f32", coef) - o[g])
        allowed = 1e-4 * (2 * off + 2.0 ** -20 * np.linalg.norm(o[g])) + 3 * 2.0 ** -24 * np.linalg.norm(want[g])
        assert np.linalg.norm(host(master[g]).astype(np.float64) - want[g]) <= allowed, g
    if w is not None:
        assert torch.equal(w, master.to(torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,R,C", [(2049, 50, 60), (2049, 60, 50)])
def test_orthogonalize_by_products_part_by_part(G, R, C, dtype):
    """1025 and 1024 matrices at a time through the chain of products, which stacks of fewer rows do not take: the
    ends of both parts."""
    print(f"case orthogonalize G={G} R={R} C={C} {dtype}", flush=True)
    x = _grad(G, R, C, R)
    got = _ortho(x, dtype)
    for g in (0, 1024, 1025, G - 1):
        _check_result(got[g], x[g], dtype, TO.COEF, f"matrix {g}")


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,R,C", [(2049, 50, 60), (2049, 60, 50), (2049, 50, 61)])
def test_muon_steps_by_products_part_by_part(G, R, C, dtype, nesterov):
    """Two steps, as in test_muon_steps: momentum, master and w of the second part, which finds the first one's
    workspace."""
    print(f"case muon G={G} R={R} C={C} {dtype} nesterov={nesterov}", flush=True)
    grads, mom0, w0, mom, master, w = _muon(G, R, C, dtype, nesterov)
    for g in (0, 1024, 1025, G - 1):
        mg, xg, allowed = mom0[g:g + 1].astype(np.float64), w0[g:g + 1].astype(np.float64), 0.0
        big = np.abs(mom0[g]) + sum(np.abs(gr[g]) for gr in grads)
        for gr in grads:
            mg, xg, o = TO.muon(gr[g:g + 1], mg, xg, **HYPER, nesterov=nesterov)
            u = gr[g].astype(np.float64) + HYPER["momentum"] * mg[0] if nesterov else mg[0]
            model = TO.newton_model(u, dtype == "f32")
            allowed += HYPER["lr"] * HYPER["scale"] * (2 * np.linalg.norm(model - o[0]) + 2.0 ** -20 * np.linalg.norm(o[0]))
            allowed += 3 * 2.0 ** -24 * np.linalg.norm(xg)
        assert np.all(np.abs(host(mom[g]).astype(np.float64) - mg[0]) <= 4 * 2.0 ** -24 * big)
        assert np.linalg.norm(host(master[g]).astype(np.float64) - xg[0]) <= allowed, g
    if w is not None:
        assert torch.equal(w, master.to(torch.bfloat16))


@pytest.mark.parametrize("coef,bound", [
    (((4.0, -6.8, 2.9), (3.9, -6.3, 2.6), (3.7, -5.6, 2.3), (2.9, -3.1, 1.2), (2.8, -3.0, 1.2)), 1.8e-2),
    (((8.2, -22.9, 16.5), (4.0, -2.9, 0.52), (3.9, -2.8, 0.52), (3.3, -2.4, 0.49), (2.3, -1.6, 0.4)), 5.6e-2)])
def test_low_rank_of_steps_that_differ(coef, bound):
    """Coefficients of its own for every step, low ranks, bf16.  The documented arithmetic (newton_model) is off by at most
    6.8e-3 and 2.6e-2 of the norm over a dozen draws; twice that, and half a step of the result."""
    g = np.random.default_rng(3)
    for R, C in ((200, 300), (300, 200)):
        x = np.stack([(g.standard_normal((R, r)) @ g.standard_normal((r, C))).astype(np.float32) for r in (1, 4, 16)])
        got = _ortho(x, "bf16", coef)
        for i in range(3):
            ref = TO.newton(x[i], coef)
            assert np.linalg.norm(got[i] - ref) <= bound * np.linalg.norm(ref), (R, C, i)


@pytest.mark.parametrize("G,R,C", [(2, 65, 63), (1, 130, 257), (3, 257, 130), (40, 520, 264), (40, 264, 520), (3, 20, 90)])
def test_exact_products_of_bf16_results(G, R, C):
    """The float32 call's bits, rounded: results of both types, small and large tiles, both orientations."""
    print(f"case exact G={G} R={R} C={C}", flush=True)
    x = _dev(_grad(G, R, C, R))
    f32, out = torch.empty(G, R, C, device="cuda"), torch.empty(G, R, C, dtype=torch.bfloat16, device="cuda")
    ws = [torch.full((M.moe_muon_workspace_bytes(G, R, C, dt),), 0xFF, dtype=torch.uint8, device="cuda")
          for dt in (M.F32, M.BF16 | M.EXACT)]
    M.moe_orthogonalize(G, R, C, x, f32, ws[0])
    M.moe_orthogonalize(G, R, C, x, out, ws[1], exact=True)
    torch.cuda.synchronize()
    assert torch.equal(out, f32.to(torch.bfloat16))
    again = torch.empty_like(f32)
    M.moe_orthogonalize(G, R, C, x, again, ws[0], exact=True)       # float32 is exact with or without
    assert torch.equal(again, f32)


@pytest.mark.parametrize("G,R,C", [(2, 130, 70), (40, 520, 264), (40, 264, 522), (3, 20, 90)])
def test_exact_steps_of_bf16_weights(G, R, C):
    print(f"case exact muon G={G} R={R} C={C}", flush=True)
    grads, mom0, w0, mom, master, _ = _muon(G, R, C, "f32", True)
    m, x, w = _dev(mom0), _dev(w0), torch.full((G, R, C), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((M.moe_muon_workspace_bytes(G, R, C, M.BF16 | M.EXACT),), 0xFF, dtype=torch.uint8, device="cuda")
    for g in grads:
        M.moe_muon(G, R, C, _dev(g), m, x, w, ws, nesterov=True, exact=True, **HYPER)
    torch.cuda.synchronize()
    assert torch.equal(m, mom) and torch.equal(x, master) and torch.equal(w, master.to(torch.bfloat16))


def test_exact_step_of_a_layer():
    """The layer's own call: a state made for exact products updates bf16 weights by them."""
    cfg = custom_config(64, 64, 6, 2, 96)
    p = device_inputs(synth.make_inputs(cfg))
    d = L.make_dims(cfg.T, cfg.H, cfg.E, cfg.K, cfg.I)
    b = L.Buffers(d)
    L.forward(b, p, fused=True)
    L.backward(b, p, fused=True)
    q = {n: p[n].float() for n in ("w1", "w3", "w2")}              # the same weights in float32
    exact, f32 = L.MuonState(p, exact=True), L.MuonState(q)
    L.muon_step(exact, p, b, lr=0.01)
    L.muon_step(f32, q, b, lr=0.01)
    L.check()
    for n in exact.names:
        assert torch.equal(exact.master[n], q[n]) and torch.equal(p[n], q[n].to(torch.bfloat16))
