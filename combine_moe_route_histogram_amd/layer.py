"""Buffers and call sequences of one MoE layer step over the C ABI.

torch is used only to allocate device memory; every computation is one of the
library's entry points, called in the order of the layer (UniEP article,
section 1.1 and Figure 1): route -> dispatch -> expert FFN -> combine, then the
mirror image for the backward.
"""
from __future__ import annotations

import torch

from . import (BF16, EXACT, F32, Dims, moe_balance, moe_balance_bwd, moe_balance_workspace_bytes, moe_combine,
               moe_combine_bwd, moe_decode, moe_decode_mx, moe_decode_workspace_bytes, moe_dispatch,
               moe_dispatch_bwd, moe_dispatch_ffn, moe_expert_ffn_bwd, moe_expert_ffn_bwd_data,
               moe_expert_ffn_bwd_weight, moe_expert_ffn_down, moe_expert_ffn_up, moe_ffn_combine,
               moe_muon, moe_muon_workspace_bytes, moe_mx_bytes, moe_mx_quantize, moe_route,
               moe_route_bwd, moe_sync_status, moe_workspace_bytes)


def make_dims(T, H, E, K, I, n_shared=0, dtype="bf16", I_shared=None) -> Dims:
    return Dims(T=T, H=H, E=E, K=K, I=I, n_shared=n_shared, I_shared=I_shared,
                dtype=BF16 if dtype == "bf16" else F32)


class Buffers:
    """Every intermediate and output of one forward + backward step."""

    def __init__(self, d: Dims, device="cuda", backward=True):
        dt, T, H, E, K, I, Ns = d.torch_dtype, d.T, d.H, d.E, d.K, d.I, d.n_shared
        R, RA = d.R, d.RA
        z = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device=device)
        i32, f32 = torch.int32, torch.float32
        self.d = d
        self.ws = z(max(moe_workspace_bytes(d), 256), dtype=torch.uint8)
        self.topk_idx = z(T, K, dtype=i32)
        self.topk_w = z(T, K, dtype=f32)
        self.counts = z(E, dtype=i32)
        self.offsets = z(E + 1, dtype=i32)
        self.slot = z(T, K, dtype=i32)
        self.slot_src = z(R, dtype=i32)
        self.x_perm = z(R, H)
        self.ab = z(RA, 2 * I)
        self.h = z(RA, I)
        self.y = z(RA, H)
        self.out = z(T, H)
        if backward:
            self.dy = z(R, H)
            self.dtopk_w = z(T, K, dtype=f32)
            self.dab = z(RA, 2 * I)
            self.dx_rows = z(RA, H)
            self.dx = z(T, H)
            self.dlogits = z(T, E, dtype=f32)
            self.dw1 = z(E, H, I, dtype=f32)
            self.dw3 = z(E, H, I, dtype=f32)
            self.dw2 = z(E, I, H, dtype=f32)
            self.dws1 = z(Ns, H, I, dtype=f32) if Ns else None
            self.dws3 = z(Ns, H, I, dtype=f32) if Ns else None
            self.dws2 = z(Ns, I, H, dtype=f32) if Ns else None


def route(b: Buffers, p: dict, stream=None):
    moe_route(b.d, p["logits"], b.topk_idx, b.topk_w, b.counts, b.offsets, b.slot, b.slot_src,
              b.ws, stream)


def forward(b: Buffers, p: dict, fused: bool = False, stream=None):
    """route -> dispatch -> expert FFN -> combine.  p holds the device inputs."""
    d = b.d
    route(b, p, stream)
    if fused:
        moe_dispatch_ffn(d, p["x"], b.slot_src, b.slot, b.offsets, p["w1"], p["w3"], p.get("ws1"),
                         p.get("ws3"), b.x_perm, b.ab, b.h, b.ws, stream)
        moe_ffn_combine(d, b.h, b.offsets, p["w2"], p.get("ws2"), b.slot, b.topk_w, b.y, b.out,
                        b.ws, stream)
    else:
        moe_dispatch(d, p["x"], b.slot, b.x_perm, stream)
        moe_expert_ffn_up(d, b.x_perm, p["x"], b.offsets, p["w1"], p["w3"], p.get("ws1"),
                          p.get("ws3"), b.ab, b.h, b.ws, stream)
        moe_expert_ffn_down(d, b.h, b.offsets, p["w2"], p.get("ws2"), b.y, b.ws, stream)
        moe_combine(d, b.y, b.slot, b.topk_w, b.out, stream)


def backward(b: Buffers, p: dict, fused: bool = False, stream=None, losses=None):
    """combine_bwd -> FFN input grads (B) -> FFN weight grads (W) -> dispatch_bwd -> route_bwd.
    fused: B and W in one launch, W filling the gaps of B (moe_expert_ffn_bwd).
    losses: BalanceBuffers of this step's logits (balance); p["dloss"], the gradients of its two
    losses, then go into dlogits along with route_bwd's, with the mask that balance was given."""
    d = b.d
    moe_combine_bwd(d, p["dout"], b.y, b.slot, b.topk_w, b.dy, b.dtopk_w, stream)
    if fused:
        moe_expert_ffn_bwd(d, b.dy, p.get("dout"), b.offsets, p["w1"], p["w3"], p["w2"],
                           p.get("ws1"), p.get("ws3"), p.get("ws2"), b.ab, b.x_perm, p["x"], b.h,
                           b.dab, b.dx_rows, b.dw1, b.dw3, b.dw2, b.dws1, b.dws3, b.dws2, b.ws,
                           stream)
    else:
        moe_expert_ffn_bwd_data(d, b.dy, p.get("dout"), b.offsets, p["w1"], p["w3"], p["w2"],
                                p.get("ws1"), p.get("ws3"), p.get("ws2"), b.ab, b.dab, b.dx_rows,
                                b.ws, stream)
        moe_expert_ffn_bwd_weight(d, b.x_perm, p["x"], b.h, b.dy, p.get("dout"), b.dab, b.offsets,
                                  b.dw1, b.dw3, b.dw2, b.dws1, b.dws3, b.dws2, b.ws, stream)
    moe_dispatch_bwd(d, b.dx_rows, b.slot, b.dx, stream)
    if losses is None:
        moe_route_bwd(d, b.dtopk_w, b.topk_w, b.topk_idx, b.dlogits, stream)
    else:
        moe_balance_bwd(d, losses.seq_len, p["logits"], losses.mask, losses.counts, losses.tokens, p["dloss"],
                        b.dtopk_w, b.topk_w, b.topk_idx, b.dlogits, stream)


def check(stream=None):
    """Wait for the step's work and raise MoeError (MOE_ETIMEOUT) if a bounded
    wait inside a persistent kernel gave up, which leaves invalid results."""
    moe_sync_status(stream)


class DecodeBuffers:
    """Outputs and workspace of the layer for a few tokens (at most 256)."""

    def __init__(self, d: Dims, device="cuda"):
        self.d = d
        self.ws = torch.empty(max(moe_decode_workspace_bytes(d), 256), dtype=torch.uint8, device=device)
        self.topk_idx = torch.empty(d.T, d.K, dtype=torch.int32, device=device)
        self.topk_w = torch.empty(d.T, d.K, dtype=torch.float32, device=device)
        self.out = torch.empty(d.T, d.H, dtype=d.torch_dtype, device=device)


def decode(b: DecodeBuffers, p: dict, stream=None):
    """The whole layer for a few tokens, logits to out.  p holds the device
    inputs as for forward(); its weights are plain matrices or packed ones
    (quantize_weights).  p["n_tokens"], if there, is the device int32 count of
    the rows in use: the rows behind it have no effect and are not written."""
    call = moe_decode_mx if p["w1"].dtype == torch.uint8 else moe_decode
    call(b.d, p["logits"], p["x"], p["w1"], p["w3"], p["w2"], p.get("ws1"), p.get("ws3"), p.get("ws2"),
         p.get("n_tokens"), b.topk_idx, b.topk_w, b.out, b.ws, stream)


def quantize_weights(p: dict) -> dict:
    """A copy of p with its weight matrices packed to 4 bits (moe_mx_quantize), on the current
    stream: the packed tensors are allocated here, so memory and work must be of one stream."""
    q = dict(p)
    for name in ("w1", "w3", "w2", "ws1", "ws3", "ws2"):
        w = p.get(name)
        if w is not None:
            G, K, N = w.shape
            q[name] = torch.empty(moe_mx_bytes(G, K, N), dtype=torch.uint8, device=w.device)
            moe_mx_quantize(G, K, N, w, q[name])
    return q


class BalanceBuffers:
    """Outputs and workspace of the router's losses; seq_len None: the batch is one sequence."""

    def __init__(self, d: Dims, seq_len=None, device="cuda"):
        self.d = d
        self.seq_len = n = d.T if seq_len is None else seq_len
        z = lambda *s, dtype: torch.empty(*s, dtype=dtype, device=device)
        self.ws = z(max(moe_balance_workspace_bytes(d, n), 256), dtype=torch.uint8)
        if n < 1:
            raise ValueError(f"seq_len must be at least 1 (got {n})")
        S = -(-d.T // n)
        self.counts = z(S, d.E, dtype=torch.int32)      # picks of each expert in each sequence
        self.tokens = z(S + 2, dtype=torch.int32)       # of each sequence; all; sequences with any
        self.probs = z(S, d.E, dtype=torch.float32)     # sums of softmax(logits)
        self.loss = z(2, dtype=torch.float32)           # load balance; squared log-sum-exp
        self.mask = None                                # of the losses, for their gradient


def balance(l: BalanceBuffers, logits, topk_idx, mask=None, stream=None):
    """The router's losses and per-expert counts of routed tokens (mask: 0 for padding)."""
    l.mask = mask
    moe_balance(l.d, l.seq_len, logits, topk_idx, mask, l.counts, l.tokens, l.probs, l.loss, l.ws, stream)


WEIGHTS = ("w1", "w3", "w2", "ws1", "ws3", "ws2")


class MuonState:
    """Momentum, float32 weights and the shared workspace of the optimizer for the weights in p (made on
    the current stream).  float32 weights are updated in place, bf16 ones are copies of `master`.  exact: bf16
    weights, too, are updated by products as exact as float32's, in about 2.5 times the time."""

    def __init__(self, p: dict, exact: bool = False):
        self.exact = exact
        self.names = [n for n in WEIGHTS if p.get(n) is not None]
        self.mom = {n: torch.zeros(p[n].shape, dtype=torch.float32, device=p[n].device) for n in self.names}
        self.master = {n: p[n].float() for n in self.names}      # float32 weights: p[n] itself
        need = 256
        for n in self.names:
            dtype = (BF16 if p[n].dtype == torch.bfloat16 else F32) | (EXACT if exact else 0)
            need = max(need, moe_muon_workspace_bytes(*p[n].shape, dtype))
        self.ws = torch.empty(need, dtype=torch.uint8, device=p[self.names[0]].device)


def muon_step(m: MuonState, p: dict, b: Buffers, lr, momentum=0.95, weight_decay=0.0, nesterov=True, coef=None,
              stream=None):
    """One step of every weight in p from the gradients that backward() left in b.  The orthogonalized
    update of a matrix [R, C] is scaled by 0.2 sqrt(max(R, C)): entries of 0.2 on average."""
    for n in m.names:
        w = p[n]
        G, R, C = w.shape
        moe_muon(G, R, C, getattr(b, "d" + n), m.mom[n], m.master[n], w if w.dtype == torch.bfloat16 else None, m.ws,
                 lr=lr, momentum=momentum, weight_decay=weight_decay, scale=0.2 * max(R, C) ** 0.5, nesterov=nesterov,
                 coef=coef, stream=stream, exact=m.exact)
