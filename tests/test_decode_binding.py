"""The Python binding of the few-token layer and the 4-bit weight calls, no GPU:
arguments that the C calls never see are refused by name."""
import pytest
import torch

import combine_moe_route_histogram_amd as M


@pytest.mark.parametrize("w", [[1.0] * 256, 1.0, "w"])
def test_mx_weights_that_are_no_tensor(w):
    mx = torch.zeros(136, dtype=torch.uint8)
    with pytest.raises(TypeError, match="w must be a torch.Tensor"):
        M.moe_mx_quantize(1, 32, 8, w, mx)
    with pytest.raises(TypeError, match="w must be a torch.Tensor"):
        M.moe_mx_dequantize(1, 32, 8, mx, w)


@pytest.mark.parametrize("sizes", [(1 + 2 ** 32, 32, 8), (1 - 2 ** 32, 32, 8), (1, 32 + 2 ** 32, 8), (1, 32, 8 - 2 ** 32),
                                   (2 ** 31, 32, 8)])
def test_mx_sizes_beyond_32_bits(sizes, monkeypatch):
    """A size whose low 32 bits are a good one: the call must not go out with those (the tensors
    were held against the whole size: a negative one asks for no element)."""
    monkeypatch.setattr(M, "_launch", lambda *a: pytest.fail("launched"))
    w, mx = torch.zeros(256), torch.zeros(136, dtype=torch.uint8)
    assert M.moe_mx_bytes(*sizes) == 0
    with pytest.raises(ValueError, match="must fit into 32 bits"):
        M.moe_mx_quantize(*sizes, w, mx)
    with pytest.raises(ValueError, match="must fit into 32 bits"):
        M.moe_mx_dequantize(*sizes, mx, w)


def test_current_stream_without_the_private_call(monkeypatch):
    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(M, "_raw_stream", None)
    assert M._stream(None) == 77
    monkeypatch.setattr(M, "_raw_stream", lambda device: 78 + device)
    assert M._stream(None) == 78 and M._stream(5) == 5
