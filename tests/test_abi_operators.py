"""Host-side refusals of the top-k router and the 8-bit products: made before any CUDA
call, so they run on a machine without a GPU."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from chunk_sparse_moe_b200 import build
    build.build()
    from chunk_sparse_moe_b200 import _lib
    return _lib


ROUTE = dict(logits=16, dt=0, bias=None, T=4, E=32, k=2, scores=0, n_group=1, topk_group=1, renorm=1, scale=1.0,
             gates=16, ids=16, weights=16, stream=None)


@pytest.mark.parametrize("change", [
    dict(dt=2), dict(scores=2), dict(scores=-1), dict(T=-1), dict(E=0), dict(E=257), dict(k=0), dict(k=33),
    dict(E=16, k=17), dict(n_group=0), dict(n_group=5), dict(n_group=4, topk_group=0), dict(n_group=4, topk_group=5),
    dict(n_group=8, topk_group=1, k=5), dict(scale=float("inf")), dict(scale=float("nan")), dict(logits=None),
    dict(ids=None), dict(weights=None), dict(logits=18), dict(ids=24), dict(weights=20), dict(bias=20), dict(gates=8)])
def test_route_topk_refuses(lib, change):
    assert lib.lib.blockffn_route_topk(*{**ROUTE, **change}.values()) == lib.ERR_INVALID_ARG
    assert lib.lib.blockffn_last_error_message()


BACK = dict(logits=16, dt=0, ids=16, d_weights=16, T=4, E=32, k=2, scores=0, renorm=1, scale=1.0, d_logits=16,
            stream=None)


@pytest.mark.parametrize("change", [
    dict(dt=7), dict(scores=3), dict(T=-2), dict(E=0), dict(E=300), dict(k=0), dict(k=33), dict(E=4, k=5),
    dict(scale=float("nan")), dict(logits=None), dict(ids=None), dict(d_weights=None), dict(d_logits=None),
    dict(logits=17), dict(ids=20), dict(d_weights=24), dict(d_logits=28)])
def test_route_topk_backward_refuses(lib, change):
    assert lib.lib.blockffn_route_topk_backward(*{**BACK, **change}.values()) == lib.ERR_INVALID_ARG


def test_quantize_refuses(lib):
    f = lib.lib.blockffn_quantize_int8
    for bad in ((16, 4, 0, 0, 16, 16), (16, -1, 8, 0, 16, 16), (16, 4, 8, 5, 16, 16), (16, 4, 1 << 27, 0, 16, 16),
                (None, 4, 8, 0, 16, 16), (16, 4, 8, 0, None, 16), (16, 4, 8, 0, 16, None), (18, 4, 8, 0, 16, 16),
                (16, 4, 8, 0, 17, 16), (16, 4, 8, 0, 16, 20)):
        assert f(*bad, None) == lib.ERR_INVALID_ARG


LINEAR = dict(x=16, dt=1, W=16, s_w=16, bias=None, T=4, K=64, O=32, y_dt=1, y=16, ws=256, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dt=2), 1), (dict(y_dt=-1), 1), (dict(T=-1), 1), (dict(K=0), 1), (dict(O=0), 1), (dict(K=72), 2),
    (dict(K=131072), 2), (dict(T=2 ** 31 - 1, O=2 ** 31 - 1), 2), (dict(x=None), 1), (dict(W=None), 1),
    (dict(s_w=None), 1), (dict(y=None), 1), (dict(ws=None), 1), (dict(x=18), 1), (dict(W=24), 1), (dict(s_w=20), 1),
    (dict(bias=20), 1), (dict(y=8), 1), (dict(ws=264), 1), (dict(ws_bytes=300), 5)])
def test_int8_linear_refuses(lib, change, status):
    assert lib.lib.blockffn_int8_linear(*{**LINEAR, **change}.values()) == status
    assert lib.lib.blockffn_last_error_message()


def test_int8_linear_workspace_size(lib):
    f = lib.lib.blockffn_int8_linear_workspace_bytes
    assert f(4, 72, 32) == 0 and f(-1, 64, 32) == 0 and f(4, 64, 0) == 0
    assert f(1000, 4096, 1) >= 1000 * 4096 + 1000 * 4 + 256


def test_no_rows_are_no_ops(lib):
    L = lib.lib
    none = {k: None for k in ("logits", "gates", "ids", "weights")}
    assert L.blockffn_route_topk(*{**ROUTE, **none, "T": 0}.values()) == lib.OK
    none = {k: None for k in ("logits", "ids", "d_weights", "d_logits")}
    assert L.blockffn_route_topk_backward(*{**BACK, **none, "T": 0}.values()) == lib.OK
    assert L.blockffn_quantize_int8(None, 0, 8, 0, None, None, None) == lib.OK
    assert L.blockffn_int8_linear(*{**LINEAR, "x": None, "y": None, "ws": None, "T": 0}.values()) == lib.OK


FORWARD = dict(x=16, gates=16, W_in=16, s_in=16, W_out=16, s_out=16, T=4, d_h=256, E=8, d_e=128, dt=1, opts=None,
               y=16, ws=256, ws_bytes=1 << 24, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dt=5), 1), (dict(dt=0), 2), (dict(T=-1), 1), (dict(d_h=0), 1), (dict(d_h=200), 2), (dict(d_h=1 << 17), 2),
    (dict(E=0), 1), (dict(E=257), 1), (dict(d_e=64), 2), (dict(d_e=640), 2), (dict(x=None), 1), (dict(gates=None), 1),
    (dict(W_in=None), 1), (dict(s_in=None), 1), (dict(W_out=None), 1), (dict(s_out=None), 1), (dict(y=None), 1),
    (dict(ws=None), 1), (dict(x=20), 1), (dict(gates=20), 1), (dict(W_in=24), 1), (dict(s_out=8), 1),
    (dict(ws_bytes=1024), 5)])
def test_forward_int8_refuses(lib, change, status):
    assert lib.lib.blockffn_forward_int8(*{**FORWARD, **change}.values()) == status
    assert lib.lib.blockffn_last_error_message()


def test_forward_int8_options_and_sizes(lib):
    import ctypes
    L = lib.lib
    for o in (lib.LayerOpts(20, None, None, None, 0.0), lib.LayerOpts(None, 24, None, None, 0.0),
              lib.LayerOpts(None, None, 16, 20, 1e-5), lib.LayerOpts(None, None, 16, None, -1.0)):
        assert L.blockffn_forward_int8(*{**FORWARD, "opts": ctypes.byref(o)}.values()) == lib.ERR_INVALID_ARG
    f = L.blockffn_forward_int8_workspace_bytes
    assert f(4, 200, 8, 128) == 0 and f(4, 256, 300, 128) == 0
    # bounded by the slice: a long input needs no more than one of 8192 tokens
    assert f(100000, 256, 8, 128) == f(8192, 256, 8, 128) > f(100, 256, 8, 128) > 0
    assert L.blockffn_forward_int8(*{**FORWARD, "T": 0, "x": None, "y": None, "ws": None}.values()) == lib.OK


@pytest.mark.parametrize("y", [1 << 20, (1 << 20) + 64, (1 << 20) - 1024])
def test_forward_int8_refuses_a_y_over_x_with_a_layernorm(lib, y):
    """The LayerNorm reads x after y has been written, so the two may not share memory then."""
    import ctypes
    o = lib.LayerOpts(None, None, 16, None, 1e-5)
    call = {**FORWARD, "x": 1 << 20, "y": y, "opts": ctypes.byref(o)}   # (4 x 256 bf16: 2048 bytes)
    assert lib.lib.blockffn_forward_int8(*call.values()) == lib.ERR_INVALID_ARG
    assert b"LayerNorm" in lib.lib.blockffn_last_error_message()
