"""GPU: the expert sum in 8-bit integers against the same formula in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_common import require_cuda

pytestmark = pytest.mark.gpu

EPS = torch.finfo(torch.bfloat16).eps / 2


def quantized(v):
    amax = np.abs(v).max(-1, keepdims=True)
    q = np.where(amax > 0, np.rint(v * 127 / np.where(amax > 0, amax, 1)), 0)
    return q, amax[..., 0] / 127


def reference(x, g, W_in, s_in, W_out, s_out, b_in=None, b_out=None):
    """(y, how far fp32 steps and a rounding of h to the other side of a border may move it), fp64."""
    T, d_h = x.shape
    E = W_in.shape[0]
    y, tol = np.zeros((T, d_h)), np.zeros((T, d_h))
    xq, sx = quantized(x)
    for e in range(E):
        t = np.nonzero(g[:, e] != 0)[0]
        if not len(t):
            continue
        z = (xq[t] @ W_in[e].T.astype(np.float64)) * sx[t, None] * s_in[e]
        if b_in is not None:
            z = z + b_in[e]
        h = z / (1 + np.exp(-z))
        hq, hs = quantized(h)
        w = W_out[e].T.astype(np.float64)
        o = (hq @ w) * hs[:, None] * s_out[e]
        if b_out is not None:
            o = o + b_out[e]
        ge = g[t, e, None]
        y[t] += ge * o
        # values of h within 1e-4 of a step of the border between two whole numbers (fp32 z and Swish:
        # some 2^-20 of |h|, at most 127 steps) may go to the other side: a step of hs each
        near = np.abs(np.abs(h / np.where(hs[:, None] > 0, hs[:, None], 1) - hq) - 0.5) < 127 * 2.0 ** -20 * 4
        flip = (near.astype(np.float64) @ np.abs(w)) * hs[:, None] * s_out[e]
        tol[t] += np.abs(ge) * (flip + 2.0 ** -20 * (np.abs(hq) @ np.abs(w) * hs[:, None] * s_out[e] + np.abs(o)))
    return y, tol


def make(T, d_h, E, d_e, seed, active, biases=False):
    """Inputs as numpy; ``active``: probability, or 'topk4', of a gate."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, d_h)).astype(np.float32)).to(torch.bfloat16)
    W_in = rng.integers(-127, 128, (E, d_e, d_h)).astype(np.int8)
    W_out = rng.integers(-127, 128, (E, d_h, d_e)).astype(np.int8)
    s_in = ((0.5 + rng.random((E, d_e))) / 73 / np.sqrt(d_h)).astype(np.float32)
    s_out = ((0.5 + rng.random((E, d_h))) / 73 / np.sqrt(d_e)).astype(np.float32)
    if active == "topk4":
        on = np.zeros((T, E), bool)
        np.put_along_axis(on, rng.random((T, E)).argsort(1)[:, :4], True, 1)
    else:
        on = rng.random((T, E)) < active
    g = np.where(on, rng.standard_normal((T, E)), 0).astype(np.float32)
    b = (rng.standard_normal((E, d_e)).astype(np.float32) * 0.1,
         rng.standard_normal((E, d_h)).astype(np.float32) * 0.1) if biases else (None, None)
    return x, g, W_in, s_in, W_out, s_out, b[0], b[1]


def call(bffn, d, **kw):
    c = [None if a is None else (a if torch.is_tensor(a) else torch.from_numpy(a)).cuda() for a in d]
    return bffn.forward_int8(*c[:6], b_in=c[6], b_out=c[7], **kw)


def compare(y, d, rows=None):
    want, tol = reference(d[0].double().numpy(), *[None if a is None else a.astype(np.float64) for a in d[1:]])
    got = y.double().cpu().numpy()
    if rows is not None:
        want, tol, got = want[rows], tol[rows], got[rows]
    assert np.all(np.abs(got - want) <= tol + 1.01 * EPS * (np.abs(want) + tol) + 1e-30)
    none = ~np.any((d[1] if rows is None else d[1][rows]) != 0, axis=1)
    if d[7] is None:
        assert not got[none].any()


CASES = [(1, 256, 16, 128, "topk4"), (1, 2048, 64, 128, "topk4"), (2, 128, 1, 128, 1.0), (7, 384, 5, 256, 0.5),
         (16, 1024, 32, 512, 0.3), (32, 2048, 64, 128, 0.2), (32, 256, 256, 128, "topk4"), (33, 512, 8, 384, 0.5),
         (50, 4096, 16, 128, "topk4"), (64, 512, 8, 512, 1.0), (100, 640, 24, 256, 0.1), (130, 256, 16, 128, 0.6),
         (257, 512, 40, 128, "topk4"), (300, 256, 4, 512, 1.0), (1000, 256, 16, 384, 0.25), (1100, 384, 12, 128, 0.5),
         (1500, 256, 6, 256, 0.9), (2051, 256, 32, 128, "topk4"), (600, 128, 200, 128, 0.02), (40, 1152, 16, 128, 0.0)]


@pytest.mark.parametrize("T,d_h,E,d_e,active", CASES)
def test_forward_int8(T, d_h, E, d_e, active):
    bffn = require_cuda()
    for biases in (False, True):
        d = make(T, d_h, E, d_e, T + d_h + E, active, biases)
        ws = bffn.Workspace.for_forward_int8(T, d_h, E, d_e)
        y = call(bffn, d, workspace=ws)
        assert bffn.device_status(ws) == (0, 0)
        compare(y, d)


def test_same_bits_shared_workspace_and_rows_behind():
    """Two rounds of calls of different shapes through one workspace give the same bits; rows behind the
    last token stay as they were."""
    bffn = require_cuda()
    shapes = CASES[:14]
    ws = bffn.Workspace(max(bffn.Workspace.for_forward_int8(*s[:4]).nbytes for s in shapes))
    first = []
    for turn in range(2):
        for n, s in enumerate(shapes):
            d = make(*s[:4], n, s[4])
            whole = torch.full((s[0] + 2, s[1]), 3.0, device="cuda", dtype=torch.bfloat16)
            call(bffn, d, workspace=ws, y=whole[: s[0]])
            assert torch.all(whole[s[0]:] == 3)
            if turn == 0:
                first.append(whole)
            else:
                assert torch.equal(whole, first[n])
    assert bffn.device_status(ws) == (0, 0)


def test_slices_of_a_long_input():
    """More than 8192 tokens: slices through the same scratch, each row as if called alone."""
    bffn = require_cuda()
    T = 8192 + 77
    d = make(T, 128, 4, 128, 1, 0.4)
    y = call(bffn, d)
    rows = np.r_[0:40, 8180:8192 + 77]
    part = [d[0][rows], d[1][rows], *d[2:]]
    compare(y[rows], part)
    lone = call(bffn, [d[0][8192:], d[1][8192:], *d[2:]])
    assert torch.equal(lone, y[8192:])


def test_layernorm_and_in_place():
    bffn = require_cuda()
    T, d_h = 40, 512
    d = make(T, d_h, 8, 128, 3, 0.5, True)
    lw, lb = torch.rand(d_h).cuda(), torch.rand(d_h).cuda()
    y = call(bffn, d)
    want = bffn.residual_layernorm(y, d[0].cuda(), lw, lb)
    assert torch.equal(call(bffn, d, ln_weight=lw, ln_bias=lb), want)
    # y may be x itself without a LayerNorm: the tokens have been rounded before y is written
    x = d[0].cuda()
    c = [torch.from_numpy(a).cuda() for a in d[1:]]
    bffn.forward_int8(x, *c[:5], b_in=c[5], b_out=c[6], y=x)
    assert torch.equal(x, y)


def test_infinite_tokens_and_gates_stay_in_their_rows():
    bffn = require_cuda()
    d = make(70, 256, 8, 128, 5, 0.5)
    clean = call(bffn, d)
    x, g = d[0].clone(), d[1].copy()
    x[3, 5], x[40, 7] = float("inf"), float("nan")
    g[3, 0] = g[40, 0] = 1.0
    g[60, 2] = np.nan
    y = call(bffn, [x, g, *d[2:]])
    bad = [3, 40, 60]
    assert torch.isnan(y[bad].float()).all()
    rest = [t for t in range(70) if t not in bad]
    assert torch.equal(y[rest], clean[rest])


def test_stream_and_graph():
    """On its own stream, and captured with the router before it and replayed on other tokens."""
    bffn = require_cuda()
    T, d_h, E, d_e = 32, 512, 32, 128
    d = make(T, d_h, E, d_e, 6, 0.5)
    c = [torch.from_numpy(a).cuda() for a in d[2:6]]
    x = d[0].cuda()
    z = torch.randn(T, E, device="cuda")
    ws = bffn.Workspace.for_forward_int8(T, d_h, E, d_e)
    out = bffn.route_topk(z, 4)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        bffn.forward_int8(x, out[0], *c, y=y, workspace=ws)
        with torch.cuda.graph(g, stream=side):
            bffn.route_topk(z, 4, out=out)
            bffn.forward_int8(x, out[0], *c, y=y, workspace=ws)
    torch.cuda.synchronize()
    for seed in (1, 2):
        torch.manual_seed(seed)
        z.normal_()
        x.normal_()
        g.replay()
        torch.cuda.synchronize()
        gates = bffn.route_topk(z, 4)[0]
        assert torch.equal(y, bffn.forward_int8(x, gates, *c))
    assert bffn.device_status(ws) == (0, 0)


def test_layer_in_8_bits_end_to_end():
    """The operators as a layer uses them: weights rounded once, logits from the 8-bit product, top-k
    gates, 8-bit experts.  Near the same layer with unrounded weights: 8 bits are good for about 1 part in
    100 of a random sum (a step is amax / 127, its error a third of that at most: relative
    amax / (127 sqrt(12)) / rms per factor, 1 % with amax near 4 rms, and there are four)."""
    bffn = require_cuda()
    T, d_h, E, d_e, k = 96, 1024, 32, 128, 4
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen)
    x = r(T, d_h).bfloat16()
    W_r, W_in, W_out = r(E, d_h) / d_h ** 0.5, r(E, d_e, d_h) / d_h ** 0.5, r(E, d_h, d_e) / d_e ** 0.5
    (qr, sr), (qi, si), (qo, so) = (bffn.quantize_int8(w.cuda()) for w in (W_r, W_in, W_out))
    logits = bffn.int8_linear(x.cuda(), qr, sr, out_dtype=torch.float32)
    gates, ids, w = bffn.route_topk(logits, k)
    y = bffn.forward_int8(x.cuda(), gates, qi, si, qo, so).double().cpu()
    want_logits = x.double() @ W_r.double().T
    assert torch.linalg.norm(logits.double().cpu() - want_logits) < 0.03 * torch.linalg.norm(want_logits)
    want = torch.zeros(T, d_h, dtype=torch.float64)
    g = gates.double().cpu()
    for e in range(E):
        z = x.double() @ W_in[e].double().T
        want += g[:, e, None] * ((z * torch.sigmoid(z)) @ W_out[e].double().T)
    assert torch.linalg.norm(y - want) < 0.05 * torch.linalg.norm(want)
    # and the union form of the framework on the same gates and the weights that the 8 bits stand for
    deq = [(q.float() * s[..., None]).bfloat16() for q, s in ((qi, si), (qo, so))]
    y16 = bffn.forward(x.cuda(), *deq, 32, gates=gates).double().cpu()
    assert torch.linalg.norm(y - y16) < 0.05 * torch.linalg.norm(y16)


def test_empty_and_refusals():
    bffn = require_cuda()
    d = make(4, 256, 4, 128, 1, 0.5)
    c = [d[0].cuda()] + [torch.from_numpy(a).cuda() for a in d[1:6]]
    assert bffn.forward_int8(c[0][:0], c[1][:0], *c[2:]).shape == (0, 256)
    with pytest.raises(bffn.BlockFFNError):
        bffn.forward_int8(c[0].float(), *c[1:])
    with pytest.raises(bffn.BlockFFNError):
        bffn.forward_int8(*c, workspace=bffn.Workspace(256))
    with pytest.raises(bffn.BlockFFNError):       # d_e 64
        bffn.forward_int8(c[0], c[1], c[2][:, :64].contiguous(), c[3][:, :64].contiguous(),
                          c[4][:, :, :64].contiguous(), c[5])
    with pytest.raises(TypeError):
        bffn.forward_int8(c[0], c[1].bfloat16(), *c[2:])
    with pytest.raises(TypeError):
        bffn.forward_int8(c[0], c[1], c[2].float(), *c[3:])
    for i, bad in ((1, c[1][:3]), (3, c[3][:, :5]), (4, c[4][:3]), (5, c[5].t())):
        with pytest.raises(ValueError):
            bffn.forward_int8(*[bad if j == i else v for j, v in enumerate(c)])
    with pytest.raises(ValueError):
        bffn.forward_int8(*c, b_in=torch.zeros(4, 1, device="cuda"))


def test_workspaces_of_the_two_forms_are_kept_apart():
    """A workspace that the bf16 forward has used is refused by the 8-bit calls, and the other way round:
    recorded in its status word, outputs left as they were, usable again after a reset."""
    bffn = require_cuda()
    T, d_h, E, d_e = 8, 256, 8, 128
    d = make(T, d_h, E, d_e, 2, 0.5)
    c = [d[0].cuda()] + [torch.from_numpy(a).cuda() for a in d[1:6]]
    W = torch.randint(-127, 128, (64, d_h), device="cuda", dtype=torch.int8)
    s_w = torch.rand(64, device="cuda")
    size = max(bffn.Workspace.for_forward_int8(T, d_h, E, d_e).nbytes, bffn.Workspace.for_int8_linear(T, d_h, 64).nbytes,
               bffn.workspace_bytes(T, d_h, E, d_e, 32, torch.bfloat16, False))
    wide = [(c[2].float() * c[3][..., None]).bfloat16(), (c[4].float() * c[5][..., None]).bfloat16()]
    calls = {"forward": lambda ws, y: bffn.forward(c[0], *wide, 32, gates=c[1], y=y, workspace=ws),
             "forward_int8": lambda ws, y: bffn.forward_int8(*c, y=y, workspace=ws),
             "int8_linear": lambda ws, y: bffn.int8_linear(c[0], W, s_w, y=y[:, :64].contiguous(), workspace=ws)}
    for first, second in (("forward", "forward_int8"), ("forward", "int8_linear"), ("forward_int8", "forward"),
                          ("int8_linear", "forward")):
        ws = bffn.Workspace(size)
        y = torch.empty_like(c[0])
        good = calls[second](bffn.Workspace(size), y.clone())
        calls[first](ws, y.clone())
        assert bffn.device_status(ws) == (0, 0)
        left = calls[second](ws, torch.full_like(y, 9.0))
        assert bffn.device_status(ws) == (5, 10) and torch.all(left == 9)
        ws.reset()
        assert torch.equal(calls[second](ws, y.clone()), good) and bffn.device_status(ws) == (0, 0)


def test_first_calls_inside_a_capture():
    """A process whose first call of each operator is a captured one: nothing that a first call looks up
    breaks the capture."""
    import os
    import subprocess
    import sys
    code = """
import torch, chunk_sparse_moe_b200 as bffn
x = torch.randn(32, 256, device='cuda').bfloat16(); z = torch.randn(32, 8, device='cuda')
W = torch.randint(-127, 128, (64, 256), device='cuda', dtype=torch.int8); s = torch.rand(64, device='cuda')
qi = torch.randint(-127, 128, (8, 128, 256), device='cuda', dtype=torch.int8); si = torch.rand(8, 128, device='cuda') / 1e3
qo = torch.randint(-127, 128, (8, 256, 128), device='cuda', dtype=torch.int8); so = torch.rand(8, 256, device='cuda') / 1e3
w1, w2 = bffn.Workspace(1 << 22), bffn.Workspace(1 << 22)
def step():
    y = bffn.int8_linear(x, W, s, workspace=w1)
    g, i, w = bffn.route_topk(z, 2)
    d = bffn.route_topk_backward(z, i, w)
    return y, g, d, bffn.forward_int8(x, g, qi, si, qo, so, workspace=w2)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
assert bffn.device_status(w1) == (0, 0) and bffn.device_status(w2) == (0, 0)
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_refused_call_reads_no_tables():
    """A refused call goes by none of the tables in its workspace, whatever they hold: nothing is computed,
    the outputs stay, and a reset makes the workspace usable."""
    bffn = require_cuda()
    for T, d_h, E, d_e in ((5, 256, 8, 128), (64, 256, 64, 256), (700, 256, 16, 128)):
        d = make(T, d_h, E, d_e, 3, 0.3)
        c = [d[0].cuda()] + [torch.from_numpy(a).cuda() for a in d[1:6]]
        size = max(bffn.Workspace.for_forward_int8(T, d_h, E, d_e).nbytes,
                   bffn.workspace_bytes(T, d_h, E, d_e, 32, torch.bfloat16, False))
        ws = bffn.Workspace(size)
        good = bffn.forward_int8(*c, workspace=ws)
        ws.reset()
        wide = [(c[2].float() * c[3][..., None]).bfloat16(), (c[4].float() * c[5][..., None]).bfloat16()]
        bffn.forward(c[0], *wide, 32, gates=c[1], workspace=ws)   # (the workspace is this call's now)
        assert bffn.device_status(ws) == (0, 0)
        gen = torch.Generator(device="cuda").manual_seed(T)
        tables = ws.buf.view(torch.uint8)[256:]   # (behind the control block)
        tables.random_(0, 256, generator=gen)
        y = bffn.forward_int8(*c, y=torch.full_like(c[0], 9.0), workspace=ws)
        assert bffn.device_status(ws) == (5, 10) and torch.all(y == 9)
        ws.reset()
        assert torch.equal(bffn.forward_int8(*c, workspace=ws), good)


@pytest.mark.parametrize("shift", [0.0, -20.0, -60.0, -86.0])
@pytest.mark.parametrize("T", [20, 2048])
def test_h_is_rounded_as_the_formula_says(T, shift):
    """The 8-bit h themselves, read through a W_out of ones on the diagonal, at values of z from everyday ones to
    those where Swish is next to nothing.  The steps of z are IEEE fp32 and repeated here; then expf is off by 2
    steps (4 U) at most, 1 + e and the quotient by U each, the row's largest value likewise, and 127 h and its quotient
    by that value by U each: 127 (6 + 6 + 2) U of a step, and everything further from a border between two whole
    numbers has to be on its side."""
    bffn = require_cuda()
    d_h = d_e = 128
    E, U = 4, 2.0 ** -24
    rng = np.random.default_rng(int(-shift) + T)
    x = torch.from_numpy(rng.standard_normal((T, d_h)).astype(np.float32)).to(torch.bfloat16)
    W_in = rng.integers(-127, 128, (E, d_e, d_h)).astype(np.int8)
    s_in = ((0.5 + rng.random((E, d_e))) / 73 / np.sqrt(d_h) * (0.3 if shift else 1.0)).astype(np.float32)
    b_in = (shift + 0.1 * rng.standard_normal((E, d_e))).astype(np.float32)
    W_out = np.broadcast_to(np.eye(d_h, d_e, dtype=np.int8), (E, d_h, d_e)).copy()
    s_out = np.ones((E, d_h), np.float32)
    pick = rng.integers(0, E, T)
    g = np.zeros((T, E), np.float32)
    g[np.arange(T), pick] = 1
    y = call(bffn, (x, g, W_in, s_in, W_out, s_out, b_in, None)).double().cpu().numpy()
    # z in fp32, as the formula reads
    xq, _ = quantized(x.double().numpy())
    sx = (np.abs(x.float().numpy()).max(1) / np.float32(127)).astype(np.float32)
    v = np.einsum("tk,tjk->tj", xq, W_in[pick].astype(np.float64)).astype(np.float32)   # (below 2^24: exact)
    z = (v * s_in[pick]) * sx[:, None] + b_in[pick]
    assert z.dtype == np.float32 and np.abs(v).max() < 2 ** 24
    h = z.astype(np.float64) / (1 + np.exp(-z.astype(np.float64)))
    amax = np.abs(h).max(1, keepdims=True)
    # (below z = -88.7 exp(-z) passes the range of fp32 and h is 0; amax below 2^-120 counts as a row of zeros)
    assert z.min() > -88.7 and np.all(amax > 1.01 * 2.0 ** -120)
    # y = hq amax / 127, rounded to bf16: off by 127 * 2^-9 = a quarter of a step at most
    hq = np.rint(y * 127 / amax)
    assert np.all(np.abs(hq) <= 127) and np.all(np.abs(np.abs(hq).max(1)) == 127)
    assert np.all(np.abs(hq - 127 * h / amax) <= 0.5 + 127 * 14.1 * U)


REFUSED = [(1, 256, 16, 128), (32, 2048, 64, 128), (200, 512, 8, 256), (2000, 256, 16, 128), (8192 + 40, 128, 4, 128)]


@pytest.mark.parametrize("T,d_h,E,d_e", REFUSED)
def test_calls_after_an_error_leave_y(T, d_h, E, d_e):
    """A workspace that holds an earlier error: every form of the last step (clusters that share a tile, one block,
    several tiles, slices) leaves y as it is, call after call."""
    bffn = require_cuda()
    d = make(T, d_h, E, d_e, 5, 0.3)
    c = [d[0].cuda()] + [torch.from_numpy(a).cuda() for a in d[1:6]]
    ws = bffn.Workspace.for_forward_int8(T, d_h, E, d_e)
    good = bffn.forward_int8(*c, workspace=ws)             # (its tables and h stay behind)
    torch.cuda.synchronize()
    ws.buf[:8] = torch.tensor([4, 0, 0, 0, 6, 0, 0, 0], dtype=torch.uint8)   # a wait that ran out
    y = torch.full_like(good, 9.0)
    for _ in range(20):
        bffn.forward_int8(*c, y=y, workspace=ws)
    assert bffn.device_status(ws) == (4, 6) and torch.all(y == 9)
    ws.reset()
    assert torch.equal(bffn.forward_int8(*c, workspace=ws), good) and bffn.device_status(ws) == (0, 0)


@pytest.mark.parametrize("d_h", [256, 8320])
def test_layernorm_after_an_error_leaves_y(d_h):
    """A refused call with a LayerNorm rewrites no row of y (rows in registers, and longer ones)."""
    bffn = require_cuda()
    T, E, d_e = 40, 4, 128
    d = make(T, d_h, E, d_e, 5, 0.5)
    c = [d[0].cuda()] + [torch.from_numpy(a).cuda() for a in d[1:6]]
    ln = dict(ln_weight=torch.rand(d_h).cuda(), ln_bias=torch.rand(d_h).cuda())
    ws = bffn.Workspace.for_forward_int8(T, d_h, E, d_e)
    good = bffn.forward_int8(*c, workspace=ws, **ln)
    assert torch.equal(good, bffn.residual_layernorm(bffn.forward_int8(*c), c[0], ln["ln_weight"], ln["ln_bias"]))
    torch.cuda.synchronize()
    y = torch.full_like(good, 9.0)
    for key in (False, True):
        ws.reset()
        if key:
            ws.buf[24] = 1                                # (the key of another form's shapes)
        else:
            ws.buf[:8] = torch.tensor([4, 0, 0, 0, 6, 0, 0, 0], dtype=torch.uint8)
        bffn.forward_int8(*c, y=y, workspace=ws, **ln)
        assert bffn.device_status(ws) == ((5, 10) if key else (4, 6)) and torch.all(y == 9)
    ws.reset()
    assert torch.equal(bffn.forward_int8(*c, workspace=ws, **ln), good)


@pytest.mark.parametrize("T,d_h,E,d_e", [(256, 128, 256, 128), (600, 128, 256, 128)])
def test_every_gate_on_with_256_experts(T, d_h, E, d_e):
    """The fullest list of work that a block of the last step can have: 256 tokens of all 256 experts."""
    bffn = require_cuda()
    d = make(T, d_h, E, d_e, 8, 1.0)
    ws = bffn.Workspace.for_forward_int8(T, d_h, E, d_e)
    y = call(bffn, d, workspace=ws)
    assert bffn.device_status(ws) == (0, 0)
    compare(y, d)


@pytest.mark.parametrize("T,d_h,E,d_e,biases", [(700, 512, 64, 128, True), (3000, 256, 64, 128, False)])
def test_long_input_with_gates_of_a_relu_router(T, d_h, E, d_e, biases):
    """About a fifth of the experts a token, neighbours alike, some tokens with none."""
    bffn = require_cuda()
    rng = np.random.default_rng(T)
    d = list(make(T, d_h, E, d_e, T, 0.0, biases))
    runs = np.repeat(rng.random(((T + 7) // 8, E)) < 0.22, 8, 0)[:T]
    on = runs & (rng.random((T, E)) < 0.9) & (rng.random((T, 1)) >= 0.05)
    d[1] = np.where(on, np.abs(rng.standard_normal((T, E))), 0).astype(np.float32)
    assert not on.any(1).all()
    ws = bffn.Workspace.for_forward_int8(T, d_h, E, d_e)
    y = call(bffn, d, workspace=ws)
    assert bffn.device_status(ws) == (0, 0)
    compare(y, d)


@pytest.mark.parametrize("T", [4, 700])
def test_calls_at_once_on_two_streams(T):
    """The three steps of a layer on two streams at once, each with its own workspaces: the bits of a call alone."""
    bffn = require_cuda()
    d_h, E, d_e = 512, 32, 128
    sets = []
    for seed in (1, 2):
        d = make(T, d_h, E, d_e, seed, 0.2)
        c = [d[0].cuda()] + [torch.from_numpy(a).cuda() for a in d[1:6]]
        W = torch.from_numpy(np.random.default_rng(seed).integers(-127, 128, (E, d_h)).astype(np.int8)).cuda()
        ws = (bffn.Workspace.for_int8_linear(T, d_h, E), bffn.Workspace.for_forward_int8(T, d_h, E, d_e))
        sets.append((c, W, torch.rand(E).cuda() / 500, ws, torch.cuda.Stream()))

    def layer(c, W, s, ws):
        gates, ids, w = bffn.route_topk(bffn.int8_linear(c[0], W, s, out_dtype=torch.float32, workspace=ws[0]), 4)
        return ids, w, bffn.forward_int8(c[0], gates, *c[2:], workspace=ws[1])

    want = [layer(*s[:4]) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(40):
        for i, s in enumerate(sets):
            with torch.cuda.stream(s[4]):
                got[i].append(layer(*s[:4]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))
        assert all(bffn.device_status(ws) == (0, 0) for ws in sets[i][3])
