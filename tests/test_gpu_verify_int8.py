"""GPU: the verification driver's layers with top-k routing and 8-bit experts."""
import pytest
import torch

from gpu_common import require_cuda

pytestmark = pytest.mark.gpu


def layers_of(bffn, d_h, E, d_e, n):
    """One layer of each kind: top-k + 8-bit experts, top-k + bf16 experts, ReLU router + 8-bit
    experts, injected gates + 8-bit experts."""
    from chunk_sparse_moe_b200.verify import Layer, TopK
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    ln = dict(ln_gamma=torch.ones(d_h, device="cuda"), ln_beta=torch.zeros(d_h, device="cuda"))
    W_in, W_out, W_r = r(E, d_e, d_h) / d_h ** 0.5, r(E, d_h, d_e) / d_e ** 0.5, r(E, d_h) / d_h ** 0.5
    (qi, si), (qo, so), (qr, sr) = (bffn.quantize_int8(w) for w in (W_in, W_out, W_r))
    eight = dict(W_in=qi, W_out=qo, s_in=si, s_out=so)
    topk = dict(W_r=qr, s_r=sr, b_r=0.1 * r(E),
                topk=TopK(4, scores="sigmoid", bias=0.1 * r(E), n_group=4, topk_group=2, scale=1.5))
    gates = torch.where(torch.rand(n, E, generator=gen).cuda() < 0.3, r(n, E), 0.0)
    return [Layer(**eight, **topk, **ln, b_in=0.1 * r(E, d_e), b_out=0.1 * r(E, d_h)),
            Layer(W_in=W_in.bfloat16(), W_out=W_out.bfloat16(), **topk, **ln),
            Layer(**eight, W_r=W_r.bfloat16(), gamma=torch.ones(E, device="cuda"), **ln),
            Layer(**eight, gates=gates, **ln)]


def by_hand(bffn, L, h, n):
    opts = dict(b_in=L.b_in, b_out=L.b_out, ln_weight=L.ln_gamma, ln_bias=L.ln_beta, ln_eps=L.ln_eps)
    gates = L.gates
    if L.topk is not None:
        c = L.topk
        logits = bffn.int8_linear(h, L.W_r, L.s_r, bias=L.b_r, out_dtype=torch.float32)
        gates, _, _ = bffn.route_topk(logits, c.k, scores=c.scores, bias=c.bias, n_group=c.n_group,
                                      topk_group=c.topk_group, renormalize=c.renormalize, scale=c.scale)
    elif gates is None:
        gates = bffn.route(h, L.W_r, L.gamma, L.eps)
    torch.cuda.synchronize()
    if L.int8:
        h = bffn.forward_int8(h, gates, L.W_in, L.s_in, L.W_out, L.s_out, **opts)
    else:
        h = bffn.forward(h, L.W_in, L.W_out, n, gates=gates, **opts)
    torch.cuda.synchronize()
    return h


@pytest.mark.parametrize("n", [1, 8, 32])
def test_steps_equal_the_calls_made_one_by_one(n):
    bffn = require_cuda()
    from chunk_sparse_moe_b200.verify import Verifier
    layers = layers_of(bffn, 512, 32, 128, n)
    v = Verifier(layers, n)
    for seed in (1, 2):
        x = torch.randn(n, 512, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        h = x
        for L in layers:
            h = by_hand(bffn, L, h, n)
        assert torch.isfinite(h.float()).all() and torch.equal(v.step(x), h)
    for ws in v.ws + [r[0] for r in v.routing if isinstance(r, tuple)]:
        assert bffn.device_status(ws) == (0, 0)


def test_run_as_a_graph():
    """The captured run leaves what the last draft's step leaves."""
    bffn = require_cuda()
    from chunk_sparse_moe_b200.verify import Verifier, run
    n = 16
    v = Verifier(layers_of(bffn, 256, 16, 128, n), n)
    drafts = [torch.randn(n, 256, device="cuda").bfloat16() for _ in range(3)]
    got = run(v, drafts, [4] * 6)
    assert got["steps"] == 6 and got["layers"] == 4 and got["us_per_step"] > 0
    last = v.h[1].clone()
    assert torch.equal(v.step(drafts[-1]), last)


def test_incomplete_layers_are_refused():
    bffn = require_cuda()
    from dataclasses import replace
    from chunk_sparse_moe_b200.verify import Verifier
    layers = layers_of(bffn, 256, 16, 128, 8)
    for bad in (replace(layers[3], s_in=None), replace(layers[1], s_r=None),
                replace(layers[1], gates=torch.zeros(8, 16, device="cuda"))):
        with pytest.raises(ValueError):
            Verifier([bad], 8)
