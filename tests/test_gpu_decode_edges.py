"""The layer for a few tokens at the edges of its contract: the largest finite
numbers, scale bytes of packed weights that the packing calls do not write, and
rows of logits without a finite one."""
import numpy as np
import pytest
import torch

import combine_moe_route_histogram_amd as M
from combine_moe_route_histogram_amd import layer as L
from oracle import decode_oracle as D

pytestmark = pytest.mark.gpu

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _decode(d, p):
    b = L.DecodeBuffers(d)
    b.ws.fill_(0xA5)
    L.decode(b, p)
    torch.cuda.synchronize()
    return b


# ---------------------------------------------------------------- the largest numbers

# 24-bit significands (of 2^104) around the last half step below the float32 maximum: there a
# rounding to bf16 gives infinity (from 0xFF8000 on, a tie to the even side)
SIGNIFICANDS = [0xFF0000, 0xFF7FFF, 0xFF8000, 0xFF8001, 0xFFC000, 0xFFFF00, 0xFFFFFE, 0xFFFFFF]


@pytest.mark.parametrize("dtype,mx", [("bf16", False), ("bf16", True), ("f32", False), ("f32", True)],
                         ids=["bf16", "bf16-mx", "f32", "f32-mx"])
@pytest.mark.parametrize("T", [1, 7, 9, 16, 17, 40, 64])
def test_h_up_to_the_largest_float(T, dtype, mx):
    """A finite h gives a finite row.  Column c of h is v_c: x holds powers of two, W3 picks the
    binary digits of v_c / 64 among them, and silu(64) is 64, so every sum is exact; out[c] is
    v_c 2^-100, to the 16 bits that h keeps as two bf16 parts and the rounding of out (2^-8; f32:
    a few additions)."""
    H = I = 32
    print(f"case largest h T={T} {dtype} mx={mx}", flush=True)
    x, w1, w3, w2 = np.zeros((T, H)), np.zeros((1, H, I)), np.zeros((1, H, I)), np.zeros((1, I, H))
    x[:, 0], w1[0, 0, :] = 64.0, 1.0
    x[:, 1:25] = 2.0 ** (98 + np.arange(24))
    v = np.zeros(I)
    for c in range(I):
        m, sign = SIGNIFICANDS[c % 8], 1 - 2 * (c // 8 % 2)
        v[c] = sign * m * 2.0 ** 104
        w3[0, 1:25, c] = [sign * (m >> i & 1) for i in range(24)]
        w2[0, c, c] = 2.0 ** -100
    put = lambda a: torch.from_numpy(a).to(DTYPE[dtype]).cuda()
    p = dict(logits=torch.zeros(T, 1, device="cuda"), x=put(x), w1=put(w1), w3=put(w3), w2=put(w2))
    b = _decode(L.make_dims(T, H, 1, 1, I, 0, dtype), L.quantize_weights(p) if mx else p)
    want = v * 2.0 ** -100
    tol = 2.0 ** -8 + 2.0 ** -15 if dtype == "bf16" else 4 * 2.0 ** -23
    assert (np.abs(b.out.double().cpu().numpy() - want) <= tol * np.abs(want)).all()


@pytest.mark.parametrize("T", [1, 9, 16, 17, 40])
def test_x_up_to_the_largest_float_on_packed_weights(T):
    """float32 rows meet 4-bit weights as three bf16 parts: h = silu(1) x 2^-100, out = h."""
    H = I = 32
    print(f"case largest x T={T}", flush=True)
    v = np.array([SIGNIFICANDS[t % 8] * (1 - 2 * (t // 8 % 2)) * 2.0 ** 104 for t in range(T)])
    x, w1, w3 = np.zeros((T, H)), np.zeros((1, H, I)), np.zeros((1, H, I))
    x[:, 0], w1[0, 0], x[:, 1], w3[0, 1] = 1.0, 1.0, v, 2.0 ** -100
    put = lambda a: torch.from_numpy(a).float().cuda()
    p = L.quantize_weights(dict(logits=torch.zeros(T, 1, device="cuda"), x=put(x), w1=put(w1), w3=put(w3),
                                w2=put(np.eye(I)[None])))
    b = _decode(L.make_dims(T, H, 1, 1, I, 0, "f32"), p)
    want = v[:, None] * 2.0 ** -100 / (1 + np.exp(-1.0))
    # exp and the division 2^-20 of it, a few additions
    assert (np.abs(b.out.double().cpu().numpy() - want) <= (2.0 ** -20 + 8 * 2.0 ** -23) * np.abs(want)).all()
