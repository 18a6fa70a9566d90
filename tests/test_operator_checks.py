"""Refusals of the dense product, the expert-order moves and the router's
gradient, through the C ABI and the binding (CPU: every call here returns
before a kernel could launch)."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def milo():
    import int3_gemm_rank_b200 as m
    m.lib()
    return m


@pytest.fixture
def cpu(milo, monkeypatch):
    """Lets CPU tensors through the CUDA check, and stops at the launch."""
    monkeypatch.setattr(milo, "_cuda", lambda t, name: None)

    def launched(dev, name, *args):
        raise AssertionError(f"{name} was not refused")

    monkeypatch.setattr(milo, "_launch", launched)
    return milo


F = C.c_void_p(0x10000)
ODD = C.c_void_p(0x10001)
HALF = C.c_void_p(0x10008)


def test_moves_refuse_bad_sizes_and_types(milo):
    L = milo.lib()
    ok = (F, 1, 4, 2, 64, F, F)
    for args, want in (
            ((F, 3, 4, 2, 64), milo.MILO_ERR_INVALID_ARG),               # dtype
            ((F, 1, -1, 2, 64), milo.MILO_ERR_INVALID_ARG),              # T
            ((F, 1, 4, 2, 0), milo.MILO_ERR_INVALID_ARG),                # H
            ((F, 1, 4, 0, 64), milo.MILO_ERR_UNSUPPORTED_SHAPE),         # k
            ((F, 1, 4, 17, 64), milo.MILO_ERR_UNSUPPORTED_SHAPE),
            ((F, 1, 4, 2, (1 << 24) + 1), milo.MILO_ERR_UNSUPPORTED_SHAPE),
            ((F, 1, 0x3FFFFFFF, 2, 64), milo.MILO_ERR_UNSUPPORTED_SHAPE),   # T*k
            ((F, 1, 1 << 20, 2, 1 << 20), milo.MILO_ERR_UNSUPPORTED_SHAPE),   # T*H
            ((None, 1, 4, 2, 64), milo.MILO_ERR_INVALID_ARG),
            ((ODD, 1, 4, 2, 64), milo.MILO_ERR_INVALID_ARG)):
        assert L.milo_dispatch(*args, F, F, F, 1, None, None) == want, args
        assert L.milo_combine(*args, F, F, None, F, 1, None, None) == want, args
        assert L.milo_dispatch_backward(*args, F, F, F, F, 1, F, None, None) == want, args
        assert L.milo_combine_backward(*args, F, F, F, F, 1, F, None, None) == want, args
    assert L.milo_dispatch(*ok, F, 7, None, None) == milo.MILO_ERR_INVALID_ARG
    assert L.milo_dispatch(*ok[:5], None, F, F, 1, None, None) == milo.MILO_ERR_INVALID_ARG
    assert L.milo_combine(*ok, ODD, F, 1, None, None) == milo.MILO_ERR_INVALID_ARG
    # a weight gradient needs the weights and the other rows
    for w, rows in ((None, F), (F, None)):
        assert L.milo_dispatch_backward(F, 1, 4, 2, 64, F, w, rows, F, 1, F, None, None) == milo.MILO_ERR_INVALID_ARG
        assert L.milo_combine_backward(F, 1, 4, 2, 64, F, w, rows, F, 1, F, None, None) == milo.MILO_ERR_INVALID_ARG
    # no tokens: nothing to do, nothing looked at
    assert L.milo_dispatch(None, 1, 0, 2, 64, None, None, None, 1, None, None) == milo.MILO_OK
    assert L.milo_combine_backward(None, 1, 0, 2, 64, None, None, None, None, 1, None, None, None) == milo.MILO_OK


def test_route_backward_refuses(milo):
    L = milo.lib()
    for args, want in (((-1, 8, 2, 0, F, 0), milo.MILO_ERR_INVALID_ARG),
                       ((4, 257, 2, 0, F, 0), milo.MILO_ERR_UNSUPPORTED_SHAPE),
                       ((4, 8, 9, 0, F, 0), milo.MILO_ERR_UNSUPPORTED_SHAPE),
                       ((4, 8, 2, 2, F, 0), milo.MILO_ERR_INVALID_ARG),
                       ((4, 8, 2, 0, F, 5), milo.MILO_ERR_INVALID_ARG),
                       ((4, 8, 2, 0, None, 0), milo.MILO_ERR_INVALID_ARG)):
        assert L.milo_route_backward(F, F, F, F, *args, None, None) == want, args
    # the full softmax needs the logits
    assert L.milo_route_backward(None, F, F, F, 4, 8, 2, 0, F, 0, None, None) == milo.MILO_ERR_INVALID_ARG
    assert L.milo_route_backward(None, None, None, None, 0, 8, 2, 0, None, 0, None, None) == milo.MILO_OK


def _linear(L, x=F, W=F, dt=1, M=4, N=16, K=64, bias=None, res=None, act=0, y=F, ydt=1, z=None):
    return L.milo_dense_linear(x, W, dt, M, N, K, bias, res, act, y, ydt, z, None, None)


def _backward(L, dy=F, dydt=1, x=F, W=F, dt=1, M=4, N=16, K=64, act=0, z=None, dx=F, dW=F, db=F, ws=F, n=1 << 30):
    return L.milo_dense_linear_backward(dy, dydt, x, W, dt, M, N, K, act, z, dx, dW, db, ws, n, None, None)


def test_dense_linear_refuses(milo):
    L = milo.lib()
    bad, shape = milo.MILO_ERR_INVALID_ARG, milo.MILO_ERR_UNSUPPORTED_SHAPE
    for call in (_linear, _backward):
        for kw, want in ((dict(dt=2), bad), (dict(M=-1), bad), (dict(N=0), bad), (dict(K=0), bad), (dict(act=5), bad),
                         (dict(act=-1), bad), (dict(K=60), shape), (dict(K=(1 << 24) + 8), shape),
                         (dict(M=(1 << 24) + 1), shape), (dict(N=1 << 24, K=1 << 20), shape), (dict(x=None), bad),
                         (dict(W=None), bad), (dict(x=HALF), bad), (dict(W=HALF), bad)):
            assert call(L, **kw) == want, (call.__name__, kw)
    for kw in (dict(y=None), dict(y=ODD), dict(ydt=3), dict(bias=ODD), dict(res=ODD), dict(z=ODD)):
        assert _linear(L, **kw) == bad, kw
    for kw in (dict(dy=None), dict(dy=ODD), dict(dydt=3), dict(act=2), dict(z=ODD), dict(dx=HALF), dict(dW=HALF),
               dict(db=ODD), dict(ws=None)):
        assert _backward(L, **kw) == bad, kw
    assert _backward(L, ws=HALF) == milo.MILO_ERR_WORKSPACE
    need = C.c_size_t()
    assert L.milo_dense_linear_backward_workspace_bytes(4, 16, 64, C.byref(need)) == milo.MILO_OK
    assert _backward(L, n=need.value - 1) == milo.MILO_ERR_WORKSPACE
    assert L.milo_dense_linear_backward_workspace_bytes(4, 16, 64, None) == bad
    assert L.milo_dense_linear_backward_workspace_bytes(4, 16, 60, C.byref(need)) == shape
    # an empty batch forward, and no gradient wanted: nothing to do
    assert _linear(L, x=None, y=None, M=0) == milo.MILO_OK
    assert _backward(L, dx=None, dW=None, db=None) == milo.MILO_OK


def _route(T, k):
    return {"ids": torch.zeros((T, k), dtype=torch.int32), "w": torch.zeros((T, k)),
            "inv_perm": torch.zeros(T * k, dtype=torch.int32)}


def test_binding_checks_the_moves(cpu):
    r = _route(4, 2)
    x, xs = torch.zeros((4, 16), dtype=torch.bfloat16), torch.zeros((8, 16), dtype=torch.bfloat16)
    w = r["w"]
    for call in (lambda: cpu.milo_dispatch(x[:3], r), lambda: cpu.milo_dispatch(x[0], r),
                 lambda: cpu.milo_dispatch(x.int(), r), lambda: cpu.milo_dispatch(x, r, w[:3]),
                 lambda: cpu.milo_dispatch(x, r, w.half()), lambda: cpu.milo_dispatch(x, r, xs=xs[:7]),
                 lambda: cpu.milo_dispatch(x, r, out_dtype=torch.int32),
                 lambda: cpu.milo_dispatch(x, dict(r, inv_perm=r["inv_perm"][:7])),
                 lambda: cpu.milo_dispatch(x, dict(r, inv_perm=r["inv_perm"].long())),
                 lambda: cpu.milo_dispatch(x, dict(r, ids=r["ids"].reshape(-1))),
                 lambda: cpu.milo_dispatch(x, r, dev_status=torch.zeros(1)),
                 lambda: cpu.milo_combine(xs[:7], r), lambda: cpu.milo_combine(xs, r, w[:, :1]),
                 lambda: cpu.milo_combine(xs, r, w, x[:3]), lambda: cpu.milo_combine(xs, r, w, x.half(), out_dtype=torch.bfloat16),
                 lambda: cpu.milo_combine(xs, r, w, y=xs),
                 lambda: cpu.milo_dispatch_backward(xs, r, x.half(), w), lambda: cpu.milo_dispatch_backward(x, r),
                 lambda: cpu.milo_dispatch_backward(xs, r, dw=w), lambda: cpu.milo_dispatch_backward(xs, r, x, w, dw=w[:2]),
                 lambda: cpu.milo_combine_backward(x, r, xs[:, :8], w), lambda: cpu.milo_combine_backward(x, r, xs.float(), w),
                 lambda: cpu.milo_combine_backward(x, r, dw=w), lambda: cpu.milo_combine_backward(x, r, xs, w, dys=x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        cpu.milo_dispatch(None, r)
    for call in (lambda: cpu.milo_dispatch(x, r, w), lambda: cpu.milo_combine(xs, r, w, x)):
        with pytest.raises(AssertionError, match="not refused"):
            call()


def test_binding_checks_the_router_gradient(cpu):
    r, dw = _route(4, 2), torch.zeros((4, 2))
    for call in (lambda: cpu.milo_route_backward(r, dw[:3], True, 8), lambda: cpu.milo_route_backward(r, dw, False, 8),
                 lambda: cpu.milo_route_backward(r, dw, False, 8, torch.zeros((4, 7), dtype=torch.float16)),
                 lambda: cpu.milo_route_backward(r, dw, False, 8, torch.zeros((4, 8))),
                 lambda: cpu.milo_route_backward(dict(r, w=dw[:, :1]), dw, True, 8),
                 lambda: cpu.milo_route_backward(r, dw, True, 8, dlogits=torch.zeros((4, 9)))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        cpu.milo_route_backward(dict(r, w=None), dw, True, 8)


def test_binding_checks_the_dense_product(cpu):
    b16 = torch.bfloat16
    x, W, y = torch.zeros((4, 64), dtype=b16), torch.zeros((16, 64), dtype=b16), torch.zeros((4, 16), dtype=b16)
    bias = torch.zeros(16, dtype=b16)
    for call in (lambda: cpu.milo_dense_linear(x[:, :56], W), lambda: cpu.milo_dense_linear(x.half(), W),
                 lambda: cpu.milo_dense_linear(x.float(), W.float()), lambda: cpu.milo_dense_linear(x, W[0]),
                 lambda: cpu.milo_dense_linear(x, W, bias[:8]), lambda: cpu.milo_dense_linear(x, W, bias.float()),
                 lambda: cpu.milo_dense_linear(x, W, act="tanh"), lambda: cpu.milo_dense_linear(x, W, residual=y[:3]),
                 lambda: cpu.milo_dense_linear(x, W, residual=y, out_dtype=torch.float32),
                 lambda: cpu.milo_dense_linear(x, W, z=y.half()), lambda: cpu.milo_dense_linear(x, W, y=y.t()),
                 lambda: cpu.milo_dense_linear(x, W, out_dtype=torch.int8),
                 lambda: cpu.milo_dense_linear_backward(y[:3], x, W), lambda: cpu.milo_dense_linear_backward(y.double(), x, W),
                 lambda: cpu.milo_dense_linear_backward(y, x, W, "silu"),
                 lambda: cpu.milo_dense_linear_backward(y, x, W, "silu", y.half()),
                 lambda: cpu.milo_dense_linear_backward(y, x, W, need=("dy",)),
                 lambda: cpu.milo_dense_linear_backward(y, x, W, out={"dW": x})):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cpu.milo_dense_linear(x, W, bias, "gelu", y, z=y.clone()),
                 lambda: cpu.milo_dense_linear_backward(y, x, W, "silu", y)):
        with pytest.raises(AssertionError, match="not refused"):
            call()


def test_binding_needs_cuda_tensors(milo):
    with pytest.raises(ValueError, match="contiguous CUDA"):
        milo.milo_dense_linear(torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((16, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous CUDA"):
        milo.milo_dispatch(torch.zeros((4, 64), dtype=torch.bfloat16), _route(4, 2))


@pytest.mark.skipif(torch.cuda.is_available(), reason="the made-up pointers below must not reach a GPU")
def test_planning_of_extreme_sizes_returns(milo):
    """Without a GPU the calls get as far as the driver: the host planning of
    every size returns an error status, never a crash."""
    import random
    L, rng = milo.lib(), random.Random(1)
    edge = [1, 2, 7, 8, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 4096, 65536, 1 << 24]
    for i in range(600):
        M, N, K = (rng.choice(edge) if rng.random() < 0.7 else rng.randint(1, 1 << 24) for _ in range(3))
        K = max(8, K // 8 * 8)
        dt, act = rng.randint(0, 1), rng.randint(0, 4)
        ok = (milo.MILO_ERR_CUDA, milo.MILO_ERR_UNSUPPORTED_SHAPE)
        assert _linear(L, dt=dt, M=M, N=N, K=K, act=act, bias=F, ydt=rng.randint(0, 2)) in ok, (M, N, K)
        assert _backward(L, dt=dt, M=M, N=N, K=K, act=act, z=F, n=1 << 62) in ok, (M, N, K)
        T, k, H, E = rng.choice(edge), rng.randint(1, 16), rng.choice(edge), rng.randint(1, 256)
        w = rng.choice([None, F])
        assert L.milo_dispatch(F, dt, T, k, H, F, w, F, dt, None, None) in ok
        assert L.milo_combine(F, dt, T, k, H, F, w, rng.choice([None, F]), F, rng.randint(0, 2), None, None) in ok
        assert L.milo_dispatch_backward(F, dt, T, k, H, F, F, F, F, dt, F, None, None) in ok
        assert L.milo_combine_backward(F, dt, T, k, H, F, F, F, F, dt, F, None, None) in ok
        assert L.milo_route_backward(F, F, F, F, T, E, min(k, E), dt, F, 2, None, None) in ok
