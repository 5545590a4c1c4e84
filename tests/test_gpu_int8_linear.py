"""GPU: rows in 8 bits and the 8-bit linear layer against exact integers in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_common import require_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def quantized(v):
    """(whole numbers, scale) of the rows of fp64 values."""
    amax = np.abs(v).max(-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(amax >= 2.0 ** -120, np.rint(v * 127 / amax), 0)
    return q, np.where(amax >= 2.0 ** -120, amax / 127, 0)[..., 0]


def values(shape, dtype, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal(shape) * (1 + 3 * (rng.random(shape[-1:]) < 0.05)) * spread
    return torch.from_numpy(v.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 1), (3, 17), (5, 128), (2, 3, 2048), (4, 4096), (2, 9000), (3, 8192), (7, 10001)])
def test_quantize(shape, dtype):
    bffn = require_cuda()
    w = values(shape, dtype, sum(shape))
    w.view(-1, shape[-1])[-1] = 0
    q, s = bffn.quantize_int8(w.cuda())
    rq, rs = quantized(w.double().numpy())
    assert np.array_equal(q.cpu().numpy().astype(np.int64), rq)
    assert np.all(np.abs(s.double().cpu().numpy() - rs) <= U * rs)


def test_quantize_borders_and_extremes():
    """Values next to the border of two whole numbers and exact halves; tiny rows; infinities, NaN."""
    bffn = require_cuda()
    K = 512
    w = torch.zeros(6, K)
    k = torch.arange(K - 1, dtype=torch.float64)
    half = ((k % 254) - 127 + 0.5) / 127 * 0.7310
    w[0, 1:] = half.float()
    w[1, 1:] = torch.nextafter(half.float(), torch.tensor(2.0))
    w[0, 0] = w[1, 0] = 0.7310
    w[2, 1:] = ((k % 254) - 127 + 0.5).float()
    w[2, 0] = 127.0                                  # exact halves go to the even number
    w[3, 5] = 1e-39                                  # too small to divide by
    w[4, 3], w[4, 5] = float("inf"), 1.0
    w[5, 3], w[5, 5] = float("nan"), 1.0
    q, s = bffn.quantize_int8(w.cuda())
    rq, rs = quantized(w[:4].double().numpy())
    assert np.array_equal(q[:4].cpu().numpy().astype(np.int64), rq)
    assert np.all(np.abs(s[:4].double().cpu().numpy() - rs) <= U * rs) and float(s[3]) == 0
    assert torch.isnan(s[4:]).all() and not q[4:].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("top", [3e38, 4.0, 1.0, 3.75, 2.0 ** -119, 2.0 ** -60])
def test_quantize_ranges(top, dtype):
    """Rows from the largest values to the smallest, many of them halves between two whole numbers."""
    bffn = require_cuda()
    rng = np.random.default_rng(7)
    w = torch.from_numpy((rng.integers(-256, 257, (8, 2048)) / 256).astype(np.float32))
    w[:, 0] = 1.0
    w = (w.double() * top).to(dtype)
    q, s = bffn.quantize_int8(w.cuda())
    rq, rs = quantized(w.double().numpy())
    assert np.array_equal(q.cpu().numpy().astype(np.int64), rq)
    assert np.all(np.abs(s.double().cpu().numpy() - rs) <= U * rs + 2.0 ** -150)


def check(bffn, x, W, s_w, bias, out_dtype, **kw):
    d = lambda t: None if t is None else t.cuda()
    y = bffn.int8_linear(d(x), d(W), d(s_w), bias=d(bias), out_dtype=out_dtype, **kw)
    q, s = quantized(x.double().numpy())
    acc = q @ W.double().numpy().T                    # exact: every sum below 2^53
    big = acc * s[:, None] * s_w.double().numpy()
    want = big if bias is None else big + bias.double().numpy()
    # int32 -> fp32, the token scale, two products, the sum; then the output type
    tol = 5 * U * np.abs(big) + torch.finfo(y.dtype).eps / 2 * np.abs(want) * 1.001 + 1e-37
    got = y.double().cpu().numpy()
    assert got.shape == want.shape and np.all(np.abs(got - want) <= tol)
    return y


SHAPES = [(1, 4096, 4096), (1, 16, 1), (2, 128, 127), (32, 2048, 8192), (17, 2064, 1007), (333, 2064, 1007),
          (64, 4096, 256), (100, 48, 130), (129, 256, 512), (300, 1024, 3000), (700, 512, 2050), (1000, 8192, 129),
          (16, 12288, 300), (257, 144, 4100), (2048, 1024, 4096), (4096, 256, 5000), (3001, 272, 2700),
          (8200, 128, 1100)]


@pytest.mark.parametrize("T,K,O", SHAPES)
def test_linear(T, K, O):
    bffn = require_cuda()
    rng = np.random.default_rng(T + K + O)
    W = torch.from_numpy(rng.integers(-127, 128, (O, K)).astype(np.int8))
    s_w = torch.from_numpy((0.01 + rng.random(O)).astype(np.float32))
    bias = torch.from_numpy(rng.standard_normal(O).astype(np.float32))
    for dtype, b, out in ((torch.bfloat16, None, None), (torch.float32, bias, None),
                          (torch.bfloat16, bias, torch.float32), (torch.float32, None, torch.bfloat16)):
        check(bffn, values((T, K), dtype, T * 3 + K), W, s_w, b, out)


def test_linear_largest_sums():
    """Every product at its largest, K at its limit: the int32 sums do not wrap."""
    bffn = require_cuda()
    K = 131056
    x = torch.ones(3, K)
    x[1] = -1
    W = torch.full((2, K), 127, dtype=torch.int8)
    W[1] = -128
    check(bffn, x, W, torch.ones(2), None, torch.float32)


def test_linear_repeats_bits_and_shares_a_workspace():
    """Calls of different shapes through one workspace, twice: the same bits, no error recorded."""
    bffn = require_cuda()
    rng = np.random.default_rng(4)
    ws = bffn.Workspace(max(bffn.Workspace.for_int8_linear(T, K, O).nbytes for T, K, O in SHAPES))
    first = []
    for turn in range(2):
        for n, (T, K, O) in enumerate(SHAPES):
            W = torch.from_numpy(np.random.default_rng(n).integers(-127, 128, (O, K)).astype(np.int8)).cuda()
            s_w = torch.full((O,), 0.01, device="cuda")
            y = bffn.int8_linear(values((T, K), torch.bfloat16, n).cuda(), W, s_w, workspace=ws)
            if turn == 0:
                first.append(y.clone())
            else:
                assert torch.equal(y, first[n])
    assert bffn.device_status(ws) == (0, 0)


def test_linear_rows_with_infinity_zero_rows_and_padding():
    bffn = require_cuda()
    T, K, O = 37, 256, 200
    x = values((T, K), torch.bfloat16, 1)
    x[3] = 0
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    W = torch.from_numpy(np.random.default_rng(2).integers(-127, 128, (O, K)).astype(np.int8)).cuda()
    s_w = torch.rand(O).cuda()
    # rows behind the last token stay as they are
    whole = torch.full((T + 3, O), 5.0, device="cuda", dtype=torch.bfloat16)
    y = bffn.int8_linear(x.cuda(), W, s_w, y=whole[:T])
    assert torch.all(whole[T:] == 5) and not y[3].any()
    assert torch.isnan(y[5:7]).all()
    rest = [t for t in range(T) if t not in (5, 6)]
    assert torch.isfinite(y[rest].float()).all()
    assert torch.equal(y[rest], bffn.int8_linear(x[rest].cuda().contiguous(), W, s_w))


def test_linear_graph_and_stream():
    """Captured once, replayed on changed inputs; and on a stream of its own."""
    bffn = require_cuda()
    T, K, O = 32, 1024, 640
    W = torch.from_numpy(np.random.default_rng(3).integers(-127, 128, (O, K)).astype(np.int8)).cuda()
    s_w = torch.rand(O).cuda()
    x = values((T, K), torch.bfloat16, 1).cuda()
    ws = bffn.Workspace.for_int8_linear(T, K, O)
    y = torch.empty(T, O, dtype=torch.bfloat16, device="cuda")
    bffn.int8_linear(x, W, s_w, y=y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bffn.int8_linear(x, W, s_w, y=y, workspace=ws)
    for seed in (5, 6):
        x.copy_(values((T, K), torch.bfloat16, seed))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, bffn.int8_linear(x, W, s_w))
    assert bffn.device_status(ws) == (0, 0)


@pytest.mark.parametrize("T", [1, 64, 600])
def test_linear_reads_what_the_kernel_before_it_wrote(T):
    """Weights, scales and tokens written by the kernels right before the call (it loads its first weight
    tiles early)."""
    bffn = require_cuda()
    K, O = 2048, 1024
    rng = np.random.default_rng(8)
    sets = [(torch.from_numpy(rng.integers(-127, 128, (O, K)).astype(np.int8)).cuda(), torch.rand(O).cuda(),
             values((T, K), torch.bfloat16, i).cuda()) for i in range(3)]
    want = [bffn.int8_linear(x, W, s) for W, s, x in sets]
    W, s, x = (torch.empty_like(t) for t in sets[0])
    ws = bffn.Workspace.for_int8_linear(T, K, O)
    got = []
    torch.cuda.synchronize()
    for turn in range(30):
        for dst, src in zip((x, s, W), (sets[turn % 3][2], sets[turn % 3][1], sets[turn % 3][0])):
            dst.copy_(src)
        got.append(bffn.int8_linear(x, W, s, workspace=ws))
    for turn in range(30):
        assert torch.equal(got[turn], want[turn % 3])


def test_linear_empty_and_refusals():
    bffn = require_cuda()
    W = torch.zeros(8, 64, dtype=torch.int8, device="cuda")
    s_w = torch.ones(8, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    assert bffn.int8_linear(x[:0], W, s_w).shape == (0, 8)
    assert bffn.quantize_int8(x[:0])[0].shape == (0, 64)
    with pytest.raises(bffn.BlockFFNError):
        bffn.int8_linear(torch.zeros(4, 40, device="cuda"), torch.zeros(8, 40, dtype=torch.int8, device="cuda"), s_w)
    with pytest.raises(bffn.BlockFFNError):
        bffn.int8_linear(x, W, s_w, workspace=bffn.Workspace(256))
    with pytest.raises(TypeError):
        bffn.int8_linear(x, W.float(), s_w)
    with pytest.raises(TypeError):
        bffn.int8_linear(x.half(), W, s_w)
    with pytest.raises(ValueError):
        bffn.int8_linear(x, W, s_w[:7])
    with pytest.raises(ValueError):
        bffn.int8_linear(x, W[:, :32], s_w)
    with pytest.raises(ValueError):
        bffn.int8_linear(x, W.cpu(), s_w)
    with pytest.raises(ValueError):
        bffn.int8_linear(x, W, s_w, y=torch.zeros(4, 7, device="cuda"))
    with pytest.raises(ValueError):
        bffn.quantize_int8(torch.zeros(4, 64, device="cuda").t())


@pytest.mark.parametrize("T,K,O", [(8, 256, 64), (1, 4096, 4096), (17, 2064, 1007), (700, 512, 2050), (4096, 128, 1100),
                                   (8200, 128, 1100), (2048, 1024, 4096)])
def test_refused_calls_leave_y(T, K, O):
    """In a workspace that holds an earlier error, or that a bf16 forward uses, nothing is computed whatever form
    the product takes: one block a tile, clusters that split K, several tiles a block, pairs of blocks."""
    bffn = require_cuda()
    x = values((T, K), torch.bfloat16, 1).cuda()
    W = torch.from_numpy(np.random.default_rng(2).integers(-127, 128, (O, K)).astype(np.int8)).cuda()
    s_w = torch.rand(O).cuda()
    ws = bffn.Workspace.for_int8_linear(T, K, O)
    good = bffn.int8_linear(x, W, s_w, workspace=ws)       # (q and the scales of this call stay behind)
    torch.cuda.synchronize()
    ws.buf[:8] = torch.tensor([4, 0, 0, 0, 6, 0, 0, 0], dtype=torch.uint8)   # a wait that ran out
    y = torch.full_like(good, 9.0)
    for _ in range(20):
        bffn.int8_linear(x, W, s_w, y=y, workspace=ws)
    assert bffn.device_status(ws) == (4, 6) and torch.all(y == 9)
    ws.reset()
    ws.buf[24] = 1                                        # (the key of another form's shapes)
    for _ in range(20):
        bffn.int8_linear(x, W, s_w, y=y, workspace=ws)
    assert bffn.device_status(ws) == (5, 10) and torch.all(y == 9)
    ws.reset()
    assert torch.equal(bffn.int8_linear(x, W, s_w, workspace=ws), good) and bffn.device_status(ws) == (0, 0)
