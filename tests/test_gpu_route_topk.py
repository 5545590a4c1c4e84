"""GPU: top-k routing and its gradient against the plain 64-bit forms."""
import numpy as np
import pytest
import torch

import topk_reference as ref
from gpu_common import require_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                       # half a step of fp32
# weights: expf off by 2 steps and its argument by half a step of |z| <= 16 (relative 16 U),
# up to 13 additions, a division, the scale
W_TOL = (2 * 2 + 16 + 13 + 2 + 1) * U
INF = float("inf")


def logits_of(T, E, dtype, seed, spread=1.5):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy((spread * rng.standard_normal((T, E))).astype(np.float32)).to(dtype)
    return z


def check(bffn, z, k, **kw):
    """Route on the GPU and compare with the reference; z a CPU tensor."""
    bias = kw.get("bias")
    gates, ids, w = bffn.route_topk(z.cuda(), k, **{**kw, "bias": None if bias is None else bias.cuda()})
    rg, ri, rw = ref.route(z.double().numpy(), k, kw.get("scores", "softmax"),
                           None if bias is None else bias.double().numpy(), kw.get("n_group", 1),
                           kw.get("topk_group"), kw.get("renormalize", True), kw.get("scale", 1.0))
    gates, ids, w = gates.double().cpu().numpy(), ids.cpu().numpy(), w.double().cpu().numpy()
    assert np.array_equal(ids, ri)
    assert np.all(np.abs(w - rw) <= W_TOL * np.abs(rw) + 1e-37)
    assert np.all(np.abs(gates - rg) <= W_TOL * np.abs(rg) + 1e-37)
    return gates, ids, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,renorm", [(1, 1, 1, True), (1, 256, 8, True), (5, 7, 7, False), (130, 64, 6, True),
                                          (33, 40, 1, False), (17, 96, 32, True), (9, 160, 5, False),
                                          (64, 16, 2, True), (3, 224, 3, False), (130, 255, 8, True)])
def test_no_bias(T, E, k, renorm, scores, dtype):
    bffn = require_cuda()
    check(bffn, logits_of(T, E, dtype, T + E), k, scores=scores, renormalize=renorm, scale=1.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,g", [(1, 256, 8, 8, 4), (257, 256, 8, 8, 4), (40, 64, 4, 4, 2), (31, 60, 5, 6, 3),
                                       (20, 100, 3, 50, 7), (12, 12, 3, 12, 5), (50, 128, 6, 1, 1),
                                       (8, 256, 4, 256, 9), (33, 160, 6, 8, 8), (65, 32, 2, 2, 1),
                                       (19, 192, 8, 16, 5), (11, 250, 6, 2, 1)])
def test_bias_and_groups(T, E, k, G, g, scores, dtype):
    bffn = require_cuda()
    rng = np.random.default_rng(E + G)
    bias = torch.from_numpy((0.2 * rng.standard_normal(E)).astype(np.float32))
    z = logits_of(T, E, dtype, T * E + G)
    check(bffn, z, k, scores=scores, bias=bias, n_group=G, topk_group=g, renormalize=True, scale=2.5)
    check(bffn, z, k, scores=scores, n_group=G, topk_group=g, renormalize=False)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_masks_and_extremes(scores):
    """Rows with nothing to choose, too little, only lowest values, NaN and infinities."""
    bffn = require_cuda()
    E, low = 64, float(torch.finfo(torch.float32).min)
    z = logits_of(12, E, torch.float32, 3)
    z[0] = -INF
    z[1, 3:] = -INF                       # three experts for k = 5
    z[2] = low                            # uniform
    z[3, 10:] = low
    z[4, ::2] = float("nan")
    z[5, 7] = INF
    z[6, 3] = -90.0
    z[7] = -200.0 + z[7] / 2              # every sigmoid underflows in fp32: the ratios do not
    z[8, 1:] = -INF
    z[9] = 0.0                            # all tie
    z[10] = torch.where(torch.arange(E) % 3 == 0, z[10], torch.tensor(-INF))
    for renorm in (True, False):
        if not renorm:
            z[7] = 0.5                    # (unscaled, those scores are below the smallest number)
        gates, ids, w = check(bffn, z, 5, scores=scores, renormalize=renorm)
        assert np.all(ids[0] == -1) and not np.any(gates[0]) and list(ids[9]) == [0, 1, 2, 3, 4]
    bias = torch.zeros(E)
    bias[5], bias[6], bias[7] = -INF, float("nan"), 3.0
    check(bffn, z, 5, scores=scores, bias=bias)
    check(bffn, z, 5, scores=scores, bias=bias, n_group=8, topk_group=3)


@pytest.mark.parametrize("n_group,topk_group", [(1, 1), (8, 3)])
def test_near_ties_are_decided_exactly(n_group, topk_group):
    """Biases that make scores equal up to the last bits: the order of the exact values."""
    bffn = require_cuda()
    rng = np.random.default_rng(9)
    T, E = 200, 64
    z = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    z[:] = z[0]                            # one set of scores ...
    s = 1 / (1 + np.exp(-z[0].double().numpy()))
    bias = torch.from_numpy((1.0 - s).astype(np.float32))   # ... every s + b is 1 within half a step
    z[1:] += torch.from_numpy((1e-7 * rng.standard_normal((T - 1, E))).astype(np.float32))
    check(bffn, z, 8, scores="sigmoid", bias=bias, n_group=n_group, topk_group=topk_group)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (130, 64, 6), (5, 7, 7), (33, 40, 1), (9, 160, 32), (66, 255, 4)])
def test_backward(T, E, k, renorm, scores, dtype):
    bffn = require_cuda()
    rng = np.random.default_rng(T + E + k)
    z = logits_of(T, E, dtype, T + 3 * E)
    z[T // 2] = -INF
    if E > 8:
        z[T // 3, 5:] = -INF
    zd = z.cuda()
    _, ids, _ = bffn.route_topk(zd, k, scores=scores, renormalize=renorm, scale=2.0)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    got = bffn.route_topk_backward(zd, ids, dw.cuda(), scores=scores, renormalize=renorm, scale=2.0)
    assert got.dtype == dtype
    want, size = ref.backward(z.double().numpy(), ids.cpu().numpy(), dw.numpy(), scores, renorm, 2.0)
    # every term as the weights, twice (its score and the mean), then the type's rounding
    tol = 3 * W_TOL * size + torch.finfo(dtype).eps / 2 * np.abs(want) * 1.01 + 1e-37
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


def test_backward_of_repeated_and_bad_ids():
    """An expert listed twice counts twice; ids outside the experts have no gradient."""
    bffn = require_cuda()
    z = logits_of(4, 20, torch.float32, 1)
    ids = torch.tensor([[3, 3, 5], [3, 3, 3], [-1, 7, 20], [1 << 30, -5, 0]], dtype=torch.int32)
    dw = torch.tensor([[1.0, 2, -1], [0.5, 0.25, 1], [9, 1, 9], [9, 9, 2]])
    for scores in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = bffn.route_topk_backward(z.cuda(), ids.cuda(), dw.cuda(), scores=scores, renormalize=renorm)
            want, size = ref.backward(z.double().numpy(), ids.numpy(), dw.numpy(), scores, renorm)
            assert np.all(np.abs(got.double().cpu().numpy() - want) <= 3 * W_TOL * size + U * np.abs(want) + 1e-37)


def test_backward_against_differences():
    """Against differences of the routed weights themselves (fp32 forward, step 2^-5: error of order
    step^2 and U / step)."""
    bffn = require_cuda()
    T, E, k, h = 4, 24, 4, 2.0 ** -5
    z = logits_of(T, E, torch.float32, 8)
    z += 0.15 * torch.argsort(torch.argsort(z, 1), 1)   # neighbours 0.15 apart or more: no choice flips
    for scores in ("softmax", "sigmoid"):
        _, ids, _ = bffn.route_topk(z.cuda(), k, scores=scores)
        dw = torch.linspace(-1, 1, T * k).view(T, k)
        got = bffn.route_topk_backward(z.cuda(), ids, dw.cuda(), scores=scores).cpu()
        for e in range(E):
            d = torch.zeros(T, E)
            d[:, e] = h
            out = []
            for zz in (z + d, z - d):
                _, i2, w = bffn.route_topk(zz.cuda(), k, scores=scores)
                # the same experts, perhaps in another order
                assert torch.equal(i2.sort(1).values, ids.sort(1).values)
                w = w.gather(1, i2.argsort(1)).gather(1, ids.argsort(1).argsort(1))
                out.append((w.cpu() * dw).sum(1))
            diff = (out[0] - out[1]) / (2 * h)
            assert torch.all((diff - got[:, e]).abs() < h * h + 16 * U / h)


def test_out_buffers_empty_and_streams():
    bffn = require_cuda()
    z = logits_of(6, 32, torch.float32, 2).cuda()
    want = bffn.route_topk(z, 4)
    out = tuple(torch.full_like(t, 7) for t in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = bffn.route_topk(z, 4, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert all(g is o for g, o in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(got, want))
    g, i, w = bffn.route_topk(z[:0], 4)
    assert g.shape == (0, 32) and i.shape == (0, 4) and w.shape == (0, 4)
    assert bffn.route_topk_backward(z[:0], i, w).shape == (0, 32)


def test_refusals():
    bffn = require_cuda()
    z = logits_of(4, 32, torch.float32, 2).cuda()
    for kw in (dict(k=0), dict(k=33), dict(k=9, n_group=8, topk_group=2), dict(k=2, n_group=5),
               dict(k=2, n_group=4, topk_group=5), dict(k=2, n_group=4, topk_group=0), dict(k=2, scale=INF)):
        with pytest.raises((bffn.BlockFFNError, RuntimeError)):
            bffn.route_topk(z, **kw)
    with pytest.raises(ValueError):
        bffn.route_topk(z, 2, scores="relu")
    with pytest.raises(ValueError):
        bffn.route_topk(z, 2, bias=torch.zeros(31, device="cuda"))
    with pytest.raises(TypeError):
        bffn.route_topk(z, 2, bias=torch.zeros(32, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        bffn.route_topk(z.half(), 2)
    with pytest.raises(ValueError):
        bffn.route_topk(z.t(), 2)
    with pytest.raises(ValueError):
        bffn.route_topk(z, 2, bias=torch.zeros(32))
    _, ids, w = bffn.route_topk(z, 2)
    with pytest.raises(TypeError):
        bffn.route_topk_backward(z, ids.long(), w)
    with pytest.raises(ValueError):
        bffn.route_topk_backward(z, ids, w[:, :1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_zeros_of_either_sign_tie(scores, dtype):
    """-0 and +0 are one logit: the lowest index goes first, also at the border of the choice."""
    bffn = require_cuda()
    E = 40
    z = logits_of(8, E, dtype, 4)
    z[0] = torch.where(torch.arange(E) % 2 == 0, -0.0, 0.0)
    z[1] = -0.0
    z[2] = torch.where(torch.arange(E) < 30, -0.0, 0.0)
    z[3] = torch.where(z[3] > 0.5, torch.tensor(0.0, dtype=dtype), -z[3].abs() * (torch.arange(E) % 3 > 0))
    z[4, :5], z[4, 5:] = -0.0, -1.0
    z[5] = -z[5].abs()
    z[5, ::7] = torch.tensor([0.0, -0.0, 0.0, -0.0, -0.0, 0.0])
    assert torch.signbit(z[3]).logical_and(z[3] == 0).any() and (z[3] == 0).sum() > 6
    for kw in (dict(), dict(bias=torch.zeros(E)), dict(bias=-torch.zeros(E), n_group=5, topk_group=2)):
        _, ids, _ = check(bffn, z, 6, scores=scores, **kw)
        if not kw:
            assert all(list(r) == [0, 1, 2, 3, 4, 5] for r in ids[:3])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_of_ids_that_cannot_be_chosen(renorm, scores, dtype):
    """Ids whose logit is NaN or -inf have no weight: no gradient from them, whatever their d_weights hold, and
    the others' as if they were not listed."""
    bffn = require_cuda()
    E, k = 40, 5
    z = logits_of(6, E, dtype, 6)
    ids = torch.tensor([[3, 7, 9, 11, 2]] * 6, dtype=torch.int32)
    dw = torch.from_numpy(np.random.default_rng(1).standard_normal((6, k)).astype(np.float32))
    z[0, 7], z[1, 3], z[1, 2] = float("nan"), float("nan"), -INF
    z[2, 9], dw[2, 2] = float("nan"), float("nan")
    z[3, 11], dw[3, 3] = -INF, INF
    z[4] = float("nan")
    z[5, 30:] = float("nan")               # (not among the ids)
    got = bffn.route_topk_backward(z.cuda(), ids.cuda(), dw.cuda(), scores=scores, renormalize=renorm, scale=2.0)
    want, size = ref.backward(z.double().numpy(), ids.numpy(), dw.numpy(), scores, renorm, 2.0)
    assert np.all(np.isfinite(want)) and not np.any(want[4]) and np.any(want[0])
    tol = 3 * W_TOL * size + torch.finfo(dtype).eps / 2 * np.abs(want) * 1.01 + 1e-37
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("E,G,g", [(64, 8, 3), (60, 6, 2), (256, 32, 9)])
def test_groups_whose_two_best_cancel(E, G, g):
    """Biases of a few hundred of either sign: a group's value is the small difference of two large scores, whose
    fp32 rounding (1.5e-5 at 200) is far above the gaps between groups.  The choice is that of 64 bits."""
    bffn = require_cuda()
    rng = np.random.default_rng(E)
    T, per = 300, E // G
    z = torch.from_numpy((0.02 * rng.standard_normal((T, E))).astype(np.float32))
    bias = torch.full((E,), -1000.0)
    size = torch.from_numpy(rng.integers(150, 400, G).astype(np.float32))
    for i in range(G):                     # its two best: +size and -size, and the scores
        bias[i * per + int(rng.integers(0, per // 2))] = size[i]
        bias[i * per + int(rng.integers(per // 2, per))] = -size[i]
    for scores in ("softmax", "sigmoid"):
        check(bffn, z, 3, scores=scores, bias=bias, n_group=G, topk_group=g)
        # and one group alone that cancels, far above the others' border or next to it
        one = 0.2 * torch.from_numpy(rng.standard_normal(E).astype(np.float32))
        one[:per] = bias[:per]
        check(bffn, z, 3, scores=scores, bias=one, n_group=G, topk_group=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(300, 256, 8), (300, 60, 6), (7, 32, 3)])
def test_plain_softmax_weights_do_not_depend_on_how_they_are_chosen(T, E, k, dtype):
    """A bias of zeros and groups that hold the chosen experts anyway change no bit of the weights."""
    bffn = require_cuda()
    z = logits_of(T, E, dtype, T + E, spread=4.0).cuda()
    want = bffn.route_topk(z, k, renormalize=False, scale=1.5)
    zero = torch.zeros(E, device="cuda")
    for kw in (dict(bias=zero), dict(bias=zero, n_group=2, topk_group=2)):
        got = bffn.route_topk(z, k, renormalize=False, scale=1.5, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    gates, ids, w = bffn.route_topk(z, k, renormalize=False, scale=1.5, n_group=4, topk_group=2)
    full = bffn.route_topk(z, min(32, E), renormalize=False, scale=1.5)[0]
    # the same experts' weights among the min(32, E) largest, where they are there
    listed = full.gather(1, ids.long())
    assert (listed != 0).float().mean() > 0.5 and torch.all((listed == 0) | (listed == w))
