"""Synthetic speculative-verification driver: draft chunks of n tokens through a
stack of BlockFFN layers.

Pages: "BlockFFN: Towards End-Side Acceleration-Friendly Mixture-of-Experts
with Chunk-Level Activation Sparsity", Abstract (chunk-level sparsity is what
lets speculative decoding verify several drafted tokens at the cost of one
union), and "BlockFFN: Sparse Mixture-of-Experts Optimized for End-Device
Deployment", Full BlockFFN Layer with Combined Losses (a layer is the expert
sum, then the residual and LayerNorm).

A verification step takes the hidden states of n drafted tokens and runs every
layer on them: one ``forward`` per layer (the union of the chunk's experts,
gates either injected per layer or from the layer's router, optional expert
biases, and the closing LayerNorm(y + h), which the single-chunk kernel applies
in its last step), all issued on one stream with no host synchronisation (each
kernel is a programmatic dependent of the one before it).  There is no draft model and no
language-model head: how many tokens a step accepts is a synthetic input (see
``workloads.accept_lengths``), so the driver measures the verifier's cost per
drafted and per accepted token.  Only orchestration lives here; every step of
the arithmetic runs in the library's kernels.

A layer may also route by top-k (``TopK``: its logits are an 8-bit product with
``W_r``) and hold its experts in 8 bits (int8 ``W_in`` and ``W_out`` with their channel
scales, as ``quantize_int8`` lays them out): then its step is ``int8_linear``,
``route_topk`` and ``forward_int8``.  Either can go with the other form of its
counterpart.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

from .api import Workspace, forward, forward_int8, int8_linear, route, route_topk


@dataclass
class TopK:
    """How a layer chooses its experts (see ``route_topk``)."""
    k: int
    scores: str = "softmax"
    bias: Optional[torch.Tensor] = None      # [E] fp32, added to the scores for the choice only
    n_group: int = 1
    topk_group: Optional[int] = None
    renormalize: bool = True
    scale: float = 1.0


@dataclass
class Layer:
    W_in: torch.Tensor                       # [E, d_e, d_h]
    W_out: torch.Tensor                      # [E, d_h, d_e]
    ln_gamma: torch.Tensor                   # [d_h] fp32
    ln_beta: torch.Tensor                    # [d_h] fp32
    gates: Optional[torch.Tensor] = None     # [n, E] fp32 injected gates, or the router below
    W_r: Optional[torch.Tensor] = None       # [E, d_h]
    b_r: Optional[torch.Tensor] = None       # [E] fp32
    gamma: Optional[torch.Tensor] = None     # [E] fp32
    eps: float = 2.0 ** -23                  # router RMSNorm epsilon
    ln_eps: float = 1e-5                     # LayerNorm epsilon
    b_in: Optional[torch.Tensor] = None      # [E, d_e] fp32 expert fc1 biases
    b_out: Optional[torch.Tensor] = None     # [E, d_h] fp32 expert fc2 biases
    # 8-bit experts: W_in and W_out are int8, these are their channel scales
    s_in: Optional[torch.Tensor] = None      # [E, d_e] fp32
    s_out: Optional[torch.Tensor] = None     # [E, d_h] fp32
    # top-k routing: W_r [E, d_h] is int8 with the channel scales s_r, b_r its bias
    topk: Optional[TopK] = None
    s_r: Optional[torch.Tensor] = None       # [E] fp32

    @property
    def int8(self) -> bool:
        return self.W_in.dtype == torch.int8


class Verifier:
    """Runs n-token draft chunks through ``layers``; owns one workspace per layer
    and the activation buffers, so a step allocates nothing (it can be captured
    in a CUDA graph)."""

    def __init__(self, layers: Sequence[Layer], n: int, dtype: torch.dtype = torch.bfloat16,
                 device=None):
        if not layers:
            raise ValueError("at least one layer")
        self.layers: List[Layer] = list(layers)
        self.n = n
        E, d_e, d_h = self.layers[0].W_in.shape
        self.d_h = d_h
        device = device or self.layers[0].W_in.device
        for L in self.layers:
            if L.int8 and (L.s_in is None or L.s_out is None):
                raise ValueError("8-bit experts need their scales s_in and s_out")
            if L.topk is not None and (L.gates is not None or L.W_r is None or L.s_r is None):
                raise ValueError("a top-k layer needs an int8 W_r with its scales s_r, and no gates")
        self.ws = [self._workspace(L, dtype, device) for L in self.layers]
        # what a layer's routing writes on the way, where ``forward`` does not route itself
        self.routing = [self._routing_buffers(L, device) for L in self.layers]
        self.h = [torch.empty((n, d_h), dtype=dtype, device=device) for _ in range(2)]

    def _workspace(self, L: Layer, dtype: torch.dtype, device) -> Workspace:
        E, d_e, d_h = L.W_in.shape
        if L.int8:
            return Workspace.for_forward_int8(self.n, d_h, E, d_e, device)
        return Workspace.for_shapes(self.n, d_h, E, d_e, self.n, dtype, L.gates is None and L.topk is None, device,
                                    with_bias=L.b_out is not None)

    def _routing_buffers(self, L: Layer, device):
        E, f32 = L.W_in.shape[0], torch.float32
        buf = lambda cols, dtype: torch.empty((self.n, cols), dtype=dtype, device=device)  # noqa: E731
        if L.topk is not None:   # the product's scratch, logits, gates, ids, weights
            return (Workspace.for_int8_linear(self.n, L.W_r.shape[1], E, device), buf(E, f32), buf(E, f32),
                    buf(L.topk.k, torch.int32), buf(L.topk.k, f32))
        return buf(E, f32) if L.int8 and L.gates is None else None

    def _gates(self, i: int, L: Layer, h: torch.Tensor) -> Optional[torch.Tensor]:
        """The layer's gates, or None where ``forward`` runs the layer's router itself."""
        if L.topk is not None:
            ws, logits, *out = self.routing[i]
            int8_linear(h, L.W_r, L.s_r, bias=L.b_r, y=logits, workspace=ws)
            c = L.topk
            return route_topk(logits, c.k, scores=c.scores, bias=c.bias, n_group=c.n_group, topk_group=c.topk_group,
                              renormalize=c.renormalize, scale=c.scale, out=out)[0]
        if L.gates is None and L.int8:
            return route(h, L.W_r, L.gamma, L.eps, b_r=L.b_r, out=self.routing[i])
        return L.gates

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """Hidden states [n, d_h] of the chunk after every layer (a buffer of the
        verifier's, overwritten by the next step)."""
        h = x
        for i, L in enumerate(self.layers):
            # the layer's output goes to the buffer its input is not in
            kw = dict(y=self.h[i % 2], workspace=self.ws[i], b_in=L.b_in, b_out=L.b_out,
                      ln_weight=L.ln_gamma, ln_bias=L.ln_beta, ln_eps=L.ln_eps)
            gates = self._gates(i, L, h)
            if L.int8:
                h = forward_int8(h, gates, L.W_in, L.s_in, L.W_out, L.s_out, **kw)
            elif gates is not None:
                h = forward(h, L.W_in, L.W_out, self.n, gates=gates, **kw)
            else:
                h = forward(h, L.W_in, L.W_out, self.n, W_r=L.W_r, b_r=L.b_r, gamma=L.gamma, eps=L.eps, **kw)
        return h


def run(verifier: Verifier, drafts: Sequence[torch.Tensor], accepted: Sequence[int],
        graph: bool = True) -> dict:
    """Verify len(accepted) steps, step k on drafts[k % len(drafts)], timed on the
    device.  ``accepted[k]`` is the synthetic number of tokens step k yields.
    Returns the time per step and the drafted / accepted tokens per second."""
    steps = len(accepted)
    stream = torch.cuda.current_stream()
    for k in range(min(3, steps)):
        verifier.step(drafts[k % len(drafts)])
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    if graph:
        # one graph over one pass of the drafts, replayed
        per = len(drafts)
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(stream)
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                for d in drafts:
                    verifier.step(d)
        torch.cuda.synchronize()
        reps = max(1, steps // per)
        steps = reps * per
        e0.record(stream)
        for _ in range(reps):
            g.replay()
        e1.record(stream)
    else:
        e0.record(stream)
        for k in range(steps):
            verifier.step(drafts[k % len(drafts)])
        e1.record(stream)
    e1.synchronize()
    ms = e0.elapsed_time(e1)
    acc = int(sum(int(a) for a in list(accepted)[:steps]))
    return {"steps": steps, "us_per_step": ms * 1e3 / steps,
            "drafted_tokens_per_s": steps * verifier.n / (ms * 1e-3),
            "accepted_tokens_per_s": acc / (ms * 1e-3), "mean_accepted": acc / steps,
            "layers": len(verifier.layers)}
