"""Host-side checks of the few-token layer and the 4-bit weight calls, no GPU:
bad arguments are refused before any launch, sizes follow the documented rules,
and the MXFP4 oracle is pinned by hand-worked values."""
import ctypes

import numpy as np
import pytest

import combine_moe_route_histogram_amd as M
from oracle import decode_oracle as D


@pytest.fixture(scope="module")
def lib():
    return M.load()


P = ctypes.c_void_p(4096)


def _dims(**kw):
    base = dict(T=16, H=128, E=8, K=2, I=256, n_shared=0, dtype=M.BF16)
    base.update(kw)
    return M.Dims(**base)


def _decode(lib, name, d, ws=P, ws_bytes=1 << 40, **over):
    names = ("logits", "x", "w1", "w3", "w2", "ws1", "ws3", "ws2", "n_tokens", "topk_idx", "topk_w", "out")
    args = [over.get(n, None if n == "n_tokens" else P) for n in names]
    return getattr(lib, name)(ctypes.byref(d), *args, ws, ws_bytes, None)


@pytest.mark.parametrize("name", ["moe_decode", "moe_decode_mx"])
@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(T=257), 2), (dict(E=257), 2), (dict(K=9), 2), (dict(H=100), 2), (dict(I=12), 2),
    (dict(H=(1 << 20) + 8), 2), (dict(I=(1 << 20) + 32), 2), (dict(n_shared=9), 2), (dict(dtype=3), 2),
    (dict(n_shared=1, I_shared=128), 2),
])
def test_bad_dims_are_refused(lib, name, kw, status):
    d = _dims(**kw)
    assert lib.moe_decode_workspace_bytes(ctypes.byref(d)) == 0
    assert _decode(lib, name, d) == status
    assert M.moe_last_error() != ""


def test_mx_layer_needs_multiples_of_the_group(lib):
    for kw in (dict(H=136), dict(I=264)):
        d = _dims(**kw)
        assert lib.moe_decode_workspace_bytes(ctypes.byref(d)) > 0      # the plain layer takes them
        assert _decode(lib, "moe_decode_mx", d) == 2 and "multiples of 32" in M.moe_last_error()


@pytest.mark.parametrize("name", ["moe_decode", "moe_decode_mx"])
def test_null_misaligned_and_workspace(lib, name):
    d = _dims(n_shared=1)
    need = lib.moe_decode_workspace_bytes(ctypes.byref(d))
    assert need > 0 and need % 256 == 0
    for arg in ("logits", "x", "w1", "w3", "w2", "ws1", "ws3", "ws2", "topk_idx", "topk_w", "out"):
        assert _decode(lib, name, d, **{arg: None}) == 1 and arg in M.moe_last_error()
        assert _decode(lib, name, d, **{arg: ctypes.c_void_p(4100)}) == 1 and "aligned" in M.moe_last_error()
    assert _decode(lib, name, d, n_tokens=ctypes.c_void_p(4098)) == 1 and "n_tokens" in M.moe_last_error()
    assert _decode(lib, name, d, ws_bytes=need - 1) == 3
    assert _decode(lib, name, d, ws=None) == 3
    assert _decode(lib, name, d, ws=ctypes.c_void_p(4096 + 16)) == 3


def test_workspace_covers_the_largest_dims(lib):
    small = lib.moe_decode_workspace_bytes(ctypes.byref(_dims(T=1)))
    large = lib.moe_decode_workspace_bytes(ctypes.byref(_dims(T=256, E=256, K=256, H=4096, I=14336, n_shared=8)))
    rows = 256 * 256 + 8 * 256
    assert small < 1 << 20 and large > rows * (14336 + 4096) * 4


@pytest.mark.parametrize("G,K,N,dtype,status", [
    (0, 32, 8, 1, 1), (1, 0, 8, 1, 2), (1, 40, 8, 1, 2), (1, 32, 4, 1, 2), (1, 32, 0, 1, 2), (1, 32, -8, 1, 2),
    (1, 32, 8, 2, 2), (1 << 30, 1 << 20, 1 << 20, 0, 2),
])
def test_mx_bad_sizes_are_refused(lib, G, K, N, dtype, status):
    assert lib.moe_mx_quantize(G, K, N, dtype, P, P, None) == status
    assert lib.moe_mx_dequantize(G, K, N, dtype, P, P, None) == status
    if dtype in (0, 1):
        assert M.moe_mx_bytes(G, K, N) == 0


def test_mx_pointers_are_checked(lib):
    for fn, names in ((lib.moe_mx_quantize, ("w", "mx")), (lib.moe_mx_dequantize, ("mx", "w"))):
        assert fn(1, 32, 8, 1, None, P, None) == 1 and names[0] in M.moe_last_error()
        assert fn(1, 32, 8, 1, P, None, None) == 1 and names[1] in M.moe_last_error()
        assert fn(1, 32, 8, 1, P, ctypes.c_void_p(4104), None) == 1 and "aligned" in M.moe_last_error()


def test_mx_bytes():
    assert M.moe_mx_bytes(1, 32, 8) == 8 * 17
    assert M.moe_mx_bytes(64, 2048, 1408) == 64 * 2048 * 1408 // 32 * 17


def test_a_tensor_of_another_device_is_refused(monkeypatch):
    """One process drives one GPU: a tensor of another one is named, not launched on.  (Tensors of
    two devices cannot be had here: a CPU tensor that says it is on a GPU stands for each.)"""
    import torch

    class On(torch.Tensor):
        def get_device(self):
            return self.index

        @property
        def device(self):
            return torch.device("cuda", self.index)

        @property
        def is_cuda(self):
            return True

    def on(index):
        t = torch.zeros(4).as_subclass(On)
        t.index = index
        return t
    called = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(M, "_stream", lambda stream: None)
    monkeypatch.setattr(M, "_call", lambda name, *args: called.append((name, args)))
    f32 = torch.float32
    M._launch("moe_decode", None, (7,), ((on(0), "x", f32, 4), (None, "ws1", f32, 4)), (9,))
    assert len(called) == 1 and called[0][1][0] == 7 and called[0][1][2:] == (None, 9, None)
    with pytest.raises(ValueError, match="out is on cuda:1, the call runs on cuda:0"):
        M._launch("moe_decode", None, (), ((on(0), "x", f32, 4), (on(1), "out", f32, 4)), ())
    with pytest.raises(ValueError, match="x has 4 elements, needs 5"):
        M._launch("moe_decode", None, (), ((on(0), "x", f32, 5),), ())
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        M._launch("moe_decode", None, (), ((torch.zeros(4), "x", f32, 4),), ())
    with pytest.raises(TypeError, match="x must be"):
        M._launch("moe_decode", None, (), ((on(0), "x", torch.int32, 4),), ())
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        M._launch("moe_decode", None, (), (([1.0], "x", f32, 1),), ())
    assert len(called) == 1


def test_mx_oracle_hand_worked():
    """Largest magnitude 5 -> scale 2^(2-2) = 1.  2.5 lies between 2 (code 4) and 3 (code 5): even
    code; 0.25 between 0 and .5: 0; 5 between 4 (code 6) and 6 (code 7): 4; 7 saturates."""
    w = np.zeros((1, 32, 2))
    w[0, :6, 0] = [5.0, 2.5, -0.25, 1.75, -3.5, 0.75]
    w[0, :2, 1] = [7.99, -8.0 * 2 ** -20]
    code, s = D.mx_quantize(w)
    assert s[0, 0].tolist() == [0, 0]
    assert code[0, 0, :6, 0].tolist() == [6, 4, 8, 4, 14, 2]
    assert D.mx_values(code, s)[0, :6, 0].tolist() == [4.0, 2.0, -0.0, 2.0, -4.0, 1.0]
    assert code[0, 0, 0, 1] == 7
    packed = D.mx_pack(code, s)
    assert packed.size == 2 * 17 and packed[0] == 6 | 4 << 4 and packed[-2:].tolist() == [127, 127]


def test_mx_oracle_zero_group_and_tiny():
    w = np.zeros((1, 32, 3), np.float32)
    w[0, 0, 1] = 2.0 ** -126
    w[0, 0, 2] = 2.0 ** -140
    code, s = D.mx_quantize(w)
    assert s[0, 0].tolist() == [-126, -126, -126]
    assert code[0, 0, 0].tolist() == [0, 2, 0]
