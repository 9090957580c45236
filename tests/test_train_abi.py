"""Host-side checks of the router's losses and the update of stacked weights, no
GPU: the header's calls are bound, bad arguments are refused before any launch,
and the oracle is pinned by hand-worked values and differences."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import combine_moe_route_histogram_amd as M
from oracle import train_oracle as TO

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_train.h")
P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    return M.load()


def _declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return {n: p.count(",") + 1 for n, p in re.findall(r"\b(moe_[a-z_]+)\s*\(([^)]*)\)\s*;", src)}


def test_header_calls_are_bound(lib):
    calls = _declared()
    assert sorted(calls) == ["moe_balance", "moe_balance_bwd", "moe_balance_workspace_bytes", "moe_muon",
                             "moe_muon_workspace_bytes", "moe_orthogonalize"]
    for name, n in calls.items():
        assert hasattr(lib, name) and callable(getattr(M, name)) and name in M.__all__
        assert len(M._SIGS[name][1]) == n, name


def test_struct_sizes(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no host compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "moe_train.h"\n#include <stdio.h>\n'
                   'int main(void) { printf("%zu %zu", sizeof(moe_newton), sizeof(moe_muon_params)); return 0; }\n')
    subprocess.run([cc, "-I", os.path.dirname(HEADER), str(src), "-o", str(tmp_path / "t")], check=True)
    out = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout
    assert out == f"{ctypes.sizeof(M.Newton)} {ctypes.sizeof(M.MuonParams)}"


# ---------------------------------------------------------------- refusals

def _dims(**kw):
    return M.Dims(**{**dict(T=16, H=128, E=8, K=2, I=256, n_shared=0, dtype=M.BF16), **kw})


def _balance(lib, d, seq_len=16, ws=P, ws_bytes=1 << 40, **over):
    names = ("logits", "topk_idx", "mask", "counts", "tokens", "probs", "loss")
    return lib.moe_balance(ctypes.byref(d), seq_len, *[over.get(n, P) for n in names], ws, ws_bytes, None)


def _balance_bwd(lib, d, seq_len=16, **over):
    names = ("logits", "mask", "counts", "tokens", "dloss", "dtopk_w", "topk_w", "topk_idx", "dlogits")
    return lib.moe_balance_bwd(ctypes.byref(d), seq_len, *[over.get(n, P) for n in names], None)


@pytest.mark.parametrize("kw,status", [(dict(T=0), 1), (dict(E=257), 2), (dict(K=9), 2), (dict(K=0), 2), (dict(H=4), 2),
                                       (dict(T=(1 << 28) + 1), 2)])
def test_balance_bad_dims(lib, kw, status):
    d = _dims(**kw)
    assert _balance(lib, d, 1) == status and _balance_bwd(lib, d, 1) == status
    assert lib.moe_balance_workspace_bytes(ctypes.byref(d), 1) == 0


@pytest.mark.parametrize("seq_len", [0, -1, 17, -2 ** 31])
def test_balance_bad_seq_len(lib, seq_len):
    d = _dims()
    assert _balance(lib, d, seq_len) == 1 and "seq_len" in M.moe_last_error()
    assert _balance_bwd(lib, d, seq_len) == 1 and "seq_len" in M.moe_last_error()
    assert lib.moe_balance_workspace_bytes(ctypes.byref(d), seq_len) == 0


def test_balance_pointers_and_workspace(lib):
    d = _dims(T=100000)
    need = lib.moe_balance_workspace_bytes(ctypes.byref(d), 100000)
    assert need > 0 and need % 256 == 0
    for n in ("logits", "topk_idx", "counts", "tokens", "probs", "loss"):
        assert _balance(lib, d, 100000, **{n: None}) == 1 and n in M.moe_last_error()
        assert _balance(lib, d, 100000, **{n: ctypes.c_void_p(4100)}) == 1 and "aligned" in M.moe_last_error()
    for n in ("logits", "counts", "tokens", "dloss", "dtopk_w", "topk_w", "topk_idx", "dlogits"):
        assert _balance_bwd(lib, d, **{n: None}) == 1 and n in M.moe_last_error()
        assert _balance_bwd(lib, d, **{n: ctypes.c_void_p(4104)}) == 1 and "aligned" in M.moe_last_error()
    assert _balance(lib, d, 100000, ws_bytes=need - 1) == 3
    assert _balance(lib, d, 100000, ws=None) == 3
    assert _balance(lib, d, 100000, ws=ctypes.c_void_p(4096 + 16)) == 3


def _ortho(lib, G=2, R=8, C=16, dtype=1, n=None, g=P, out=P, ws=P, ws_bytes=1 << 50):
    return lib.moe_orthogonalize(G, R, C, dtype, n, g, out, ws, ws_bytes, None)


def _muon(lib, G=2, R=8, C=16, dtype=1, n=None, params=M.MuonParams(1e-3, 0.9, 0.0, 1.0, 1), lr=None, grad=P, mom=P,
          master=P, w=P, ws=P, ws_bytes=1 << 50):
    return lib.moe_muon(G, R, C, dtype, n, params and ctypes.byref(params), lr, grad, mom, master, w, ws, ws_bytes, None)


@pytest.mark.parametrize("G,R,C,dtype,status", [
    (0, 8, 8, 1, 1), (-1, 8, 8, 1, 1), (1, 0, 8, 1, 2), (1, 8, 0, 0, 2), (1, (1 << 20) + 1, 8, 0, 2),
    (1, 8, (1 << 20) + 1, 1, 2), (1, 8, 8, 2, 2), (1, 8, 8, -1, 2), (1, 1 << 20, 1 << 20, 1, 2), (2 ** 31 - 1, 1 << 20, 8, 1, 2),
])
def test_stack_bad_sizes(lib, G, R, C, dtype, status):
    w = P if dtype == 1 else None
    assert _ortho(lib, G, R, C, dtype) == status and M.moe_last_error() != ""
    assert _muon(lib, G, R, C, dtype, w=w) == status
    assert lib.moe_muon_workspace_bytes(G, R, C, dtype) == 0


def test_stack_of_too_many_matrices(lib):
    """The number of a matrix is counted up by parts of the stack, in 31 bits."""
    assert lib.moe_muon_workspace_bytes(1 << 30, 1, 1, 1) > 0
    for G in ((1 << 30) + 1, 2 ** 31 - 1):
        assert lib.moe_muon_workspace_bytes(G, 1, 1, 1) == 0
        assert _ortho(lib, G, 1, 1) == 2 and _muon(lib, G, 1, 1) == 2


def test_stack_pointers_and_workspace(lib):
    for n in ("g", "out"):
        assert _ortho(lib, **{n: None}) == 1 and n in M.moe_last_error()
        assert _ortho(lib, **{n: ctypes.c_void_p(4100)}) == 1 and "aligned" in M.moe_last_error()
    for n in ("grad", "mom", "master", "w"):
        assert _muon(lib, **{n: None}) == 1 and n in M.moe_last_error()
        assert _muon(lib, **{n: ctypes.c_void_p(4100)}) == 1 and "aligned" in M.moe_last_error()
    assert _muon(lib, dtype=0) == 1 and "w must be NULL" in M.moe_last_error()
    assert _muon(lib, params=None) == 1 and "params" in M.moe_last_error()
    assert _muon(lib, lr=ctypes.c_void_p(4098)) == 1 and "lr" in M.moe_last_error()
    need = lib.moe_muon_workspace_bytes(2, 8, 16, 1)
    assert need > 0 and need % 256 == 0
    for call in (_ortho, _muon):
        assert call(lib, ws_bytes=need - 1) == 3 and call(lib, ws=None) == 3
        assert call(lib, ws=ctypes.c_void_p(4096 + 128)) == 3


def test_iteration_is_checked(lib):
    n = M.Newton()
    for steps in (0, -1, 17):
        n.steps = steps
        assert _ortho(lib, n=ctypes.byref(n)) == 1 and "steps" in M.moe_last_error()
    n = M.Newton([(1, 2, 3)] * 2)
    for bad in (float("nan"), float("inf"), -32.5):
        n.coef[1][2] = bad
        assert _muon(lib, n=ctypes.byref(n)) == 1 and "coefficients" in M.moe_last_error()
    with pytest.raises(ValueError):
        M.Newton([])
    with pytest.raises(ValueError):
        M.Newton([(1, 2, 3)] * 17)


def test_workspace_is_of_a_part_of_the_stack(lib):
    """Many matrices are worked on part by part."""
    few, many = (lib.moe_muon_workspace_bytes(G, 1024, 1024, 1) for G in (256, 100000))
    assert many <= 2 * few


def test_binding_refuses_what_ctypes_would_cut():
    t = torch.zeros(4)
    for G, R, C in ((2 ** 32 + 1, 8, 8), (1, 2 ** 32 + 8, 8), (1, 8, 2 ** 33)):
        assert M.moe_muon_workspace_bytes(G, R, C, 1) == 0
        with pytest.raises(ValueError):
            M.moe_orthogonalize(G, R, C, t, t, t)
        with pytest.raises(ValueError):
            M.moe_muon(G, R, C, t, t, t, None, t, lr=0.1)
    d = _dims()
    assert M.moe_balance_workspace_bytes(d, 2 ** 32 + 4) == 0
    with pytest.raises(ValueError):
        M.moe_balance(d, 2 ** 32 + 4, t, t, None, t, t, t, t, t)


def test_binding_names_the_wrong_tensor(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = torch.zeros(256)
    with pytest.raises(TypeError):
        M.moe_orthogonalize(1, 8, 8, t, t.half(), t)
    with pytest.raises(TypeError):
        M.moe_muon(1, 8, 8, t, t, t, 5, t, lr=0.1)
    with pytest.raises(ValueError, match="g must be a GPU tensor"):
        M.moe_orthogonalize(1, 8, 8, t, t, t)
    with pytest.raises(ValueError, match="logits must be a GPU tensor"):
        M.moe_balance(_dims(), 16, t, t, None, t, t, t, t, None)


# ---------------------------------------------------------------- the oracle

def test_even_load_has_a_balance_of_one():
    """Equal logits, picks spread evenly: p = 1/E, c = K n / E, so the loss is E/(K n^2) E (K n/E)(n/E) = 1."""
    E, K, T = 4, 2, 8
    idx = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    got = TO.balance(np.zeros((T, E)), idx, None, T, E, K)
    assert got["loss"] == pytest.approx([1.0, np.log(4) ** 2])
    assert got["counts"].tolist() == [[4, 4, 4, 4]] and got["tokens"].tolist() == [8, 8, 1]


def test_balance_by_hand():
    """Two tokens of two experts, one sequence each, second one padding."""
    got = TO.balance(np.array([[np.log(3.0), 0.0], [5.0, 7.0]]), np.array([[0], [1]]), [1, 0], 1, 2, 1)
    assert got["probs"] == pytest.approx(np.array([[0.75, 0.25], [0, 0]]))
    assert got["loss"] == pytest.approx([2 * 0.75, np.log(4.0) ** 2])
    assert got["tokens"].tolist() == [1, 0, 1, 1]


def test_gradient_is_the_losses_difference():
    g = np.random.default_rng(3)
    T, E, K, n = 11, 5, 2, 4
    l = g.standard_normal((T, E))
    idx = np.argsort(-l, 1)[:, :K]
    mask = g.random(T) < 0.7
    dloss = np.array([0.3, 0.7])
    ref = TO.balance(l, idx, mask, n, E, K)
    d = TO.balance_bwd(l, mask, n, E, K, ref["counts"], ref["tokens"], dloss)
    for t in range(T):
        for e in range(E):
            lo, hi = l.copy(), l.copy()
            lo[t, e] -= 1e-5
            hi[t, e] += 1e-5
            diff = (TO.balance(hi, idx, mask, n, E, K)["loss"] - TO.balance(lo, idx, mask, n, E, K)["loss"]) / 2e-5
            assert d[t, e] == pytest.approx(float((dloss * diff).sum()), abs=1e-8)


def test_iteration_of_a_diagonal_matrix():
    """Singular values move by s <- a s + b s^3 + c s^5, each on its own."""
    s = np.array([3.0, 4.0])
    x = s / 5
    for a, b, c in TO.COEF:
        x = a * x + b * x ** 3 + c * x ** 5
    got = TO.newton(np.array([[3.0, 0, 0], [0, 4.0, 0]]))
    assert got[:, :2] == pytest.approx(np.diag(x))
    assert TO.newton(np.array([[3.0, 0, 0], [0, 4.0, 0]]).T) == pytest.approx(got.T)


def test_model_of_the_arithmetic():
    """Two fp16 parts are as good as float32; one is 1e-3 off, low ranks included."""
    g = np.random.default_rng(5)
    for u in (g.standard_normal((48, 80)), g.standard_normal((80, 6)) @ g.standard_normal((6, 48))):
        ref = TO.newton(u)
        err = lambda v: np.linalg.norm(v - ref) / np.linalg.norm(ref)
        assert err(TO.newton_model(u, True)) < 1e-4 and err(TO.newton_model(u, False)) < 4e-3


def test_exact_is_a_flag_of_either_type(lib):
    assert M.EXACT & (M.F32 | M.BF16) == 0
    need = {dt: lib.moe_muon_workspace_bytes(64, 256, 512, dt) for dt in (0, 1, M.EXACT, 1 | M.EXACT)}
    assert need[1 | M.EXACT] == need[M.EXACT] == need[0] > need[1] > 0
    assert _ortho(lib, 64, 256, 512, 1 | M.EXACT, ws_bytes=need[1]) == 3       # the exact form's workspace
    for bad in (2 | M.EXACT, 1 | 2 * M.EXACT, -M.EXACT):
        assert _ortho(lib, dtype=bad) == 2 and _muon(lib, dtype=bad) == 2
        assert lib.moe_muon_workspace_bytes(2, 8, 16, bad) == 0
    assert _muon(lib, dtype=1 | M.EXACT, w=None) == 1 and "w" in M.moe_last_error()
    assert _muon(lib, dtype=M.EXACT) == 1 and "w must be NULL" in M.moe_last_error()
