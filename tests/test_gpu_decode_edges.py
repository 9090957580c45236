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


# ---------------------------------------------------------------- scale bytes

def _every_scale(N=8):
    """All 16 codes (shifted by the column) under every scale byte: packed, and float64 values."""
    code = np.resize(np.arange(16, dtype=np.uint8), 32)[None, None, :, None] + np.arange(N, dtype=np.uint8)
    code = np.broadcast_to(code & 15, (1, 256, 32, N)).copy()
    s = np.broadcast_to((np.arange(256) - 127).reshape(1, 256, 1), (1, 256, N)).astype(np.int64)
    return D.mx_pack(code, s), D.mx_values(code, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dequantize_every_scale_byte(dtype):
    """Byte b is 2^(b-127) from 0 to 254; a value beyond the type's range is infinity, 255 is NaN."""
    packed, want = _every_scale()
    back = torch.empty(1, 256 * 32, 8, dtype=DTYPE[dtype], device="cuda")
    M.moe_mx_dequantize(1, 256 * 32, 8, torch.from_numpy(packed).cuda(), back)
    got = back.double().cpu().numpy()
    assert np.isnan(got[0, 255 * 32:]).all()
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)[0, :255 * 32]
    assert np.array_equal(got[0, :255 * 32], want)


def _packed_layer(rng, E, H, I, top, scale):
    """Packed weights with codes up to magnitude `top` in the matrices that `scale` gives a byte:
    (device tensors, float64 values)."""
    p, values = {}, {}
    for name, K, N in (("w1", H, I), ("w3", H, I), ("w2", I, H)):
        code = (rng.integers(0, top + 1, (E, K // 32, 32, N)) + 8 * rng.integers(0, 2, (E, K // 32, 32, N))).astype(np.uint8)
        s = np.full((E, K // 32, N), scale[name] - 127, np.int64)
        p[name], values[name] = torch.from_numpy(D.mx_pack(code, s)).cuda(), D.mx_values(code, s)
    return p, values


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 7, 9, 17, 40])
@pytest.mark.parametrize("byte,top", [(0, 7), (1, 7), (253, 5), (254, 3)])
def test_decode_mx_smallest_and_largest_scales(T, byte, top, dtype):
    """Weights under the scale bytes at both ends, as far as float32 holds their values (byte 253:
    codes up to 3, 254: up to 1.5), in the first product and in the second."""
    H, I = 96, 160
    print(f"case scale byte {byte} T={T} {dtype}", flush=True)
    rng = np.random.default_rng(17)
    far = 100 if byte < 127 else -100      # brings the products back into the middle of the range
    for scale, x_exp in ((dict(w1=124, w3=127 + far, w2=byte), 0), (dict(w1=124 - far, w3=byte, w2=127), far)):
        p, values = _packed_layer(rng, 1, H, I, top, scale)
        inp = {"logits": np.zeros((T, 1), np.float32)}
        x = torch.from_numpy(rng.standard_normal((T, H)) * 2.0 ** x_exp).to(DTYPE[dtype])
        inp["x"] = x.view(torch.int16).numpy().view(np.uint16) if dtype == "bf16" else x.numpy()
        b = _decode(L.make_dims(T, H, 1, 1, I, 0, dtype), dict(p, x=x.cuda(), logits=torch.zeros(T, 1, device="cuda")))
        ref = D.decode(inp, 1, dtype, values)
        assert (np.abs(b.out.double().cpu().numpy() - ref["out"]) <= ref["bound"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 7, 9, 17, 40])
@pytest.mark.parametrize("byte,code", [(253, 7), (254, 12), (255, 0), (255, 3)])
def test_decode_mx_values_beyond_the_range_stay_in_their_column(T, byte, code, dtype):
    """An infinite or NaN weight of the second product makes its column of the rows that meet it
    infinite or NaN, and changes nothing else."""
    H, I, E = 96, 160, 2
    print(f"case byte {byte} code {code} T={T} {dtype}", flush=True)
    rng = np.random.default_rng(18)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(DTYPE[dtype]).cuda()
    logits = torch.zeros(T, E, device="cuda")
    logits[::2, 1] = 1.0                    # the even rows pick expert 1
    p, _ = _packed_layer(rng, E, H, I, 7, dict(w1=124, w3=124, w2=124))
    p.update(x=x, logits=logits)
    clean = _decode(L.make_dims(T, H, E, 1, I, 0, dtype), p).out
    w2 = p["w2"].clone()
    groups, col = I // 32 * H, 33           # group 2 of expert 1's column 33
    at = groups + 2 * H + col
    w2[16 * at:16 * at + 16] = code * 17
    w2[16 * E * groups + at] = byte
    out = _decode(L.make_dims(T, H, E, 1, I, 0, dtype), dict(p, w2=w2)).out
    hit = torch.zeros(T, H, dtype=torch.bool, device="cuda")
    hit[::2, col] = True
    assert torch.equal(out[~hit], clean[~hit]) and not out[hit].isfinite().any()
    if byte == 255:
        assert out[hit].isnan().all()


# ---------------------------------------------------------------- logits without a finite one

ROUTES = [  # T, E, K, Ns: picks in the product's blocks, in a launch of their own, in one block
    (4, 8, 2, 0), (4, 100, 60, 1), (7, 8, 2, 1), (40, 64, 6, 0), (20, 100, 70, 0), (64, 64, 33, 1), (16, 256, 130, 0)]


@pytest.mark.parametrize("mx", [False, True], ids=["plain", "mx"])
@pytest.mark.parametrize("T,E,K,Ns", ROUTES)
def test_rows_whose_mask_leaves_nothing(T, E, K, Ns, mx):
    """All -inf: experts 0..K-1 and NaN weights, as with moe_route; +inf: NaN weights; the type's
    lowest value in every place: equal weights.  The other rows keep their bits."""
    print(f"case masked rows T={T} E={E} K={K} Ns={Ns} mx={mx}", flush=True)
    H = I = 32
    g = torch.Generator(device="cuda").manual_seed(T + E)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")
    p = dict(logits=draw(T, E), x=draw(T, H), w1=draw(E, H, I), w3=draw(E, H, I), w2=draw(E, I, H))
    if Ns:
        p.update(ws1=draw(Ns, H, I), ws3=draw(Ns, H, I), ws2=draw(Ns, I, H))
    q = L.quantize_weights(p) if mx else p
    d = L.make_dims(T, H, E, K, I, Ns, "f32")
    clean = _decode(d, q)
    logits = p["logits"].clone()
    logits[0] = float("-inf")
    logits[1, E - 1] = float("inf")
    logits[2] = torch.finfo(torch.float32).min
    b = _decode(d, dict(q, logits=logits))
    route = L.Buffers(d, backward=False)
    L.route(route, dict(p, logits=logits))
    torch.cuda.synchronize()
    assert torch.equal(b.topk_idx, route.topk_idx)
    assert torch.equal(b.topk_w.nan_to_num(2.0), route.topk_w.nan_to_num(2.0))
    first = torch.arange(K, dtype=torch.int32, device="cuda")
    assert torch.equal(b.topk_idx[0], first) and torch.equal(b.topk_idx[2], first) and b.topk_idx[1, 0] == E - 1
    assert b.topk_w[:2].isnan().all() and b.out[:2].isnan().all()
    # K equal exponentials: their sum is exact, so only the division rounds
    assert (b.topk_w[2].double() * K - 1).abs().max() <= 2.0 ** -23 and b.out[2].isfinite().all()
    for name in ("out", "topk_idx", "topk_w"):
        assert torch.equal(getattr(b, name)[3:], getattr(clean, name)[3:]), name


# ---------------------------------------------------------------- streams and graphs

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_packing_replays_eager_bits(dtype):
    """Packing and unpacking captured into one graph: replays see new weights, with eager work and
    synchronizations between them."""
    G, K, N = 3, 96, 1000
    g = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randn(G, K, N, generator=g, device="cuda").to(DTYPE[dtype])
    make = lambda: (torch.empty(M.moe_mx_bytes(G, K, N), dtype=torch.uint8, device="cuda"), torch.empty_like(w))

    def both(mx, back):
        M.moe_mx_quantize(G, K, N, w, mx)
        M.moe_mx_dequantize(G, K, N, mx, back)
    mx, back = make()
    both(mx, back)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(mx, back)
    for rep in range(4):
        w.copy_(torch.randn(G, K, N, generator=g, device="cuda") * 10.0 ** (rep - 2))
        eager = make()
        both(*eager)
        mx.zero_()
        back.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(mx, eager[0]) and torch.equal(back, eager[1]), rep


@pytest.mark.parametrize("T", [1, 40])
def test_streams_by_handle_and_current(T):
    """A stream given as torch's object, as its raw handle, and as the current one."""
    H, I, E = 64, 96, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")
    p = dict(logits=draw(T, E), x=draw(T, H), w1=draw(E, H, I), w3=draw(E, H, I), w2=draw(E, I, H))
    d = L.make_dims(T, H, E, 2, I, 0, "f32")
    want = _decode(d, p).out
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, None):
        b = L.DecodeBuffers(d)
        torch.cuda.synchronize()
        with torch.cuda.stream(side if stream is None else torch.cuda.current_stream()):
            L.decode(b, p, stream=stream)
        side.synchronize()
        assert torch.equal(b.out, want)
