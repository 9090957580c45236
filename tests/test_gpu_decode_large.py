"""The layer for a few tokens and the 4-bit weight calls on matrices whose
offsets pass 32 bits, in bytes and in elements."""
import pytest
import torch

import combine_moe_route_histogram_amd as M
from combine_moe_route_histogram_amd import layer as L
from test_gpu_decode_kernels import _reference

pytestmark = pytest.mark.gpu

K, N = 4096, 16384      # 2^26 weights a matrix


def _mx_group(mx, G, g):
    """Group g of a packed set, as a packed set of its own."""
    one = K * N // 32
    return torch.cat([mx[16 * one * g:16 * one * (g + 1)], mx[16 * one * G + one * g:16 * one * G + one * (g + 1)]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_packing_beyond_32_bit_offsets(dtype):
    """70 matrices, 4.7e9 weights: groups around 2^31 and 2^32 elements have the bytes and values
    that they have alone."""
    G = 70
    gen = torch.Generator(device="cuda").manual_seed(6)
    w = torch.empty(G, K, N, dtype=dtype, device="cuda")
    for g in range(G):
        w[g] = torch.randn(K, N, generator=gen, device="cuda") * 0.02
    assert w.numel() > 2 ** 32
    mx = torch.empty(M.moe_mx_bytes(G, K, N), dtype=torch.uint8, device="cuda")
    M.moe_mx_quantize(G, K, N, w, mx)
    back = torch.empty_like(w)
    M.moe_mx_dequantize(G, K, N, mx, back)
    one = torch.empty(M.moe_mx_bytes(1, K, N), dtype=torch.uint8, device="cuda")
    alone = torch.empty(K, N, dtype=dtype, device="cuda")
    for g in (0, 31, 32, 63, 64, G - 1):
        M.moe_mx_quantize(1, K, N, w[g], one)
        assert torch.equal(_mx_group(mx, G, g), one), g
        M.moe_mx_dequantize(1, K, N, one, alone)
        assert torch.equal(back[g], alone), g


@pytest.mark.parametrize("T", [2, 12, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,mx", [(130, True), (70, False)], ids=["mx", "plain"])
def test_last_expert_beyond_32_bit_offsets(E, mx, dtype, T):
    """Weights of more than 2^32 bytes (plain: elements) a matrix set; every token picks the last expert."""
    print(f"case large E={E} T={T} {dtype} mx={mx}", flush=True)
    H, I = K, N
    act = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(7)
    p, last = {}, {}
    for name, shape in (("w1", (H, I)), ("w3", (H, I)), ("w2", (I, H))):
        last[name] = (torch.randn(*shape, generator=gen, device="cuda") * 0.02).to(act)
        if mx:      # the groups before the last are never read as its own: they hold NaN
            one = H * I // 32
            packed = torch.empty(17 * one, dtype=torch.uint8, device="cuda")
            M.moe_mx_quantize(1, *shape, last[name], packed)
            p[name] = torch.full((17 * one * E,), 255, dtype=torch.uint8, device="cuda")
            p[name][16 * one * (E - 1):16 * one * E] = packed[:16 * one]
            p[name][16 * one * E + one * (E - 1):] = packed[16 * one:]
            last[name] = torch.empty(*shape, device="cuda")
            M.moe_mx_dequantize(1, *shape, packed, last[name])
            assert p[name].numel() > 2 ** 32
        else:
            p[name] = torch.full((E, *shape), float("nan"), dtype=act, device="cuda")
            p[name][E - 1] = last[name]
            assert p[name].numel() > 2 ** 32
    p["x"] = torch.randn(T, H, generator=gen, device="cuda").to(act)
    p["logits"] = torch.zeros(T, E, device="cuda")
    p["logits"][:, E - 1] = 1.0
    b = L.DecodeBuffers(L.make_dims(T, H, E, 1, I, 0, dtype))
    b.ws.fill_(0xA5)
    L.decode(b, p)
    _, _, want, bound = _reference(p, lambda name, e: last[name].double(), (T, H, E, 1, I, 0), act)
    assert (b.topk_idx == E - 1).all() and (b.topk_w == 1).all()
    assert ((b.out.double() - want).abs() <= bound).all()
