"""milo_dense_linear and its gradients on the GPU against the plain 64-bit
implementation, within its derived bounds: token counts from one up, widths
that fill no tile, every activation and type; captured, on other streams, and
chained with the router and the expert-order moves."""
import numpy as np
import pytest

import operator_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def milo():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int3_gemm_rank_b200 as m
    m.lib()
    return m


def n64(t):
    return t.detach().double().cpu().numpy()


def rand(rng, shape, dt, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * std).to(DT[dt]).cuda()


def check(got, want, bound, what):
    err = np.abs(n64(got) - want)
    assert got.shape == want.shape and (err <= bound).all(), f"{what}: {(err - bound).max():.3e} above the bound"


# M around every tile edge; N of one column, below and above a tile, odd; K of
# one 16-byte piece, below, at and past a stage, many stages
SIZES = [(1, 1, 8), (1, 4096, 512), (2, 130, 72), (7, 64, 2048), (16, 16, 64), (17, 1411, 264), (33, 72, 1032),
         (64, 256, 4096), (65, 65, 136), (128, 128, 128), (129, 257, 200), (200, 8, 4160), (255, 520, 64),
         (256, 1000, 320), (300, 64, 2048), (513, 384, 1096), (1000, 1030, 136), (1025, 2056, 72)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dt,out,act,bias,res,z", [("bf16", "bf16", "silu", True, True, True),
                                                   ("f16", "f16", "none", False, False, False),
                                                   ("bf16", "f32", "gelu", True, False, False),
                                                   ("f16", "bf16", "gelu_tanh", False, True, True),
                                                   ("bf16", "f16", "relu", True, True, False)])
def test_forward(milo, M, N, K, dt, out, act, bias, res, z):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    x, W = rand(rng, (M, K), dt), rand(rng, (N, K), dt, K ** -0.5)
    b = rand(rng, (N,), dt) if bias else None
    r = rand(rng, (M, N), out) if res else None
    zt = torch.full((M, N), float("nan"), dtype=DT[dt], device="cuda") if z else None
    st = milo.new_status()
    y = milo.milo_dense_linear(x, W, b, act, r, out_dtype=DT[out], z=zt, dev_status=st)
    yr, yb, zr, zb = R.linear(n64(x), n64(W), n64(b) if bias else None, act, n64(r) if res else None, dt, out)
    check(y, yr, yb, "y")
    if z:
        check(zt, zr, zb, "z")
    assert y.dtype == DT[out] and int(st.item()) == 0


@pytest.mark.parametrize("M,N,K", [s for s in SIZES if s != (64, 256, 4096)])
@pytest.mark.parametrize("dt,dyt,act", [("bf16", "bf16", "silu"), ("f16", "f16", "none"), ("bf16", "f32", "gelu"),
                                        ("f16", "bf16", "gelu_tanh"), ("bf16", "f16", "none"), ("f16", "f16", "relu")])
def test_backward(milo, M, N, K, dt, dyt, act):
    rng = np.random.default_rng(M * 5 + N + K)
    x, W = rand(rng, (M, K), dt), rand(rng, (N, K), dt, K ** -0.5)
    dy = rand(rng, (M, N), dyt, N ** -0.5)
    z = rand(rng, (M, N), dt, 2.0) if act != "none" else None
    st = milo.new_status()
    g = milo.milo_dense_linear_backward(dy, x, W, act, z, dev_status=st)
    want = R.linear_backward(n64(dy), n64(x), n64(W), act, None if z is None else n64(z), dt, act == "none" and dyt == dt)
    assert list(g) == ["dx", "dW", "db"]
    for name in g:
        check(g[name], *want[name], name)
        assert g[name].dtype == DT[dt]
    assert int(st.item()) == 0
    # each gradient alone is the same, bit for bit
    for name in ("dx", "dW", "db"):
        assert torch.equal(milo.milo_dense_linear_backward(dy, x, W, act, z, need=(name,))[name], g[name]), name


@pytest.mark.parametrize("M,N,K", [(5, 9001, 520), (18, 6288, 1032), (100, 4100, 1096), (128, 8192, 264), (129, 8195, 264)])
@pytest.mark.parametrize("dt,dyt,act", [("bf16", "bf16", "none"), ("f16", "f16", "gelu")])
def test_backward_of_few_tokens_and_wide_layers(milo, M, N, K, dt, dyt, act):
    """Shapes whose two gradients want tiles of different kinds."""
    test_backward(milo, M, N, K, dt, dyt, act)


# tiles of pairs of CTAs (256 x 256), more tiles than fit at once, ragged on every side
LARGE = [(2600, 2312, 648), (1537, 5000, 264), (4100, 1032, 512)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("dt,out,act,res", [("bf16", "bf16", "gelu_tanh", True), ("f16", "f32", "none", False)])
def test_large_products(milo, M, N, K, dt, out, act, res):
    rng = np.random.default_rng(M + N + K)
    x, W = rand(rng, (M, K), dt), rand(rng, (N, K), dt, K ** -0.5)
    b, r = rand(rng, (N,), dt), rand(rng, (M, N), out) if res else None
    zt = torch.empty((M, N), dtype=DT[dt], device="cuda")
    st = milo.new_status()
    y = milo.milo_dense_linear(x, W, b, act, r, out_dtype=DT[out], z=zt, dev_status=st)
    yr, yb, zr, zb = R.linear(n64(x), n64(W), n64(b), act, n64(r) if res else None, dt, out)
    check(y, yr, yb, "y")
    check(zt, zr, zb, "z")
    dy = rand(rng, (M, N), dt, N ** -0.5)
    g = milo.milo_dense_linear_backward(dy, x, W, act, zt, dev_status=st)
    want = R.linear_backward(n64(dy), n64(x), n64(W), act, n64(zt), dt, act == "none")
    for name in g:
        check(g[name], *want[name], name)
        one = milo.milo_dense_linear_backward(dy, x, W, act, zt, need=(name,), dev_status=st)[name]
        assert torch.equal(one, g[name]), name
    assert int(st.item()) == 0


def test_calls_on_several_streams_at_once(milo):
    """Products of every kind (streamed, split over clusters, pairs of CTAs, both
    gradients) side by side on four streams give what they give alone."""
    rng = np.random.default_rng(10)
    work = []
    for M, N, K in ((1, 512, 4096), (40, 512, 2048), (700, 64, 2048), (512, 1024, 1024), (2300, 2312, 264)):
        x, W, dy = rand(rng, (M, K), "bf16"), rand(rng, (N, K), "bf16"), rand(rng, (M, N), "bf16")
        work.append((x, W, dy, milo.milo_dense_linear(x, W), milo.milo_dense_linear_backward(dy, x, W)))
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        with torch.cuda.stream(streams[i % 4]):
            x, W, dy, y, g = work[(i * 7) % len(work)]
            got.append((milo.milo_dense_linear(x, W), y))
            g2 = milo.milo_dense_linear_backward(dy, x, W)
            got += [(g2[n], g[n]) for n in g]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activations_far_out(milo, act):
    """Pre-activations from 2^-20 to 2^12 and zeros, through an identity weight:
    no NaN, and within the activation's bound."""
    v = np.concatenate([[0.0], 2.0 ** np.arange(-20.0, 13.0), np.linspace(0.1, 20, 31)])
    v = np.concatenate([v, -v])
    v = np.resize(v, (16, 64))
    x = torch.from_numpy(v).half().cuda()
    W = torch.eye(64, dtype=torch.float16, device="cuda")
    y = milo.milo_dense_linear(x, W, None, act, out_dtype=torch.float32)
    yr, yb, _, _ = R.linear(n64(x), n64(W), None, act, None, "f16", "f32")
    check(y, yr, yb, "y")
    dy = torch.ones((16, 64), dtype=torch.float16, device="cuda")
    g = milo.milo_dense_linear_backward(dy, x, W, act, x, need=("dx",))
    check(g["dx"], *R.linear_backward(n64(dy), n64(x), n64(W), act, n64(x), "f16", False)["dx"], "dx")


def test_in_place_residual_views_and_an_empty_batch(milo):
    rng = np.random.default_rng(4)
    x, W = rand(rng, (70, 128), "bf16"), rand(rng, (96, 128), "bf16", 0.1)
    y = rand(rng, (70, 96), "bf16")
    want = R.linear(n64(x), n64(W), None, "none", n64(y), "bf16", "bf16")
    assert milo.milo_dense_linear(x, W, residual=y, y=y) is y
    check(y, want[0], want[1], "in place")
    # rows taken from a larger tensor, results into an odd offset of a larger buffer
    buf = torch.zeros(40 * 96 + 1, dtype=torch.bfloat16, device="cuda")
    out = buf[1:].view(40, 96)
    milo.milo_dense_linear(x[30:], W[:96], y=out)
    yr, yb, _, _ = R.linear(n64(x[30:]), n64(W), None, "none", None, "bf16", "bf16")
    check(out, yr, yb, "unaligned y")
    assert float(buf[0]) == 0.0
    empty = x[:0]
    assert milo.milo_dense_linear(empty, W).shape == (0, 96)
    g = milo.milo_dense_linear_backward(torch.empty((0, 96), dtype=torch.bfloat16, device="cuda"), empty, W)
    assert g["dx"].shape == (0, 128) and not g["dW"].any() and not g["db"].any()


# a split sum, tiles of single CTAs, of pairs; each with rows of whole 16-byte
# pieces, of whole words, of odd elements
@pytest.mark.parametrize("M,N,K", [(300, 64, 2048), (300, 66, 2048), (301, 63, 2048), (20001, 120, 72), (20001, 122, 72),
                                   (20001, 121, 72), (2600, 2312, 264), (2600, 2310, 264), (2601, 2311, 264)])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f32")])
def test_residuals_in_place_in_every_form(milo, M, N, K, dt, out):
    rng = np.random.default_rng(M + N)
    x, W, b = rand(rng, (M, K), dt), rand(rng, (N, K), dt, K ** -0.5), rand(rng, (N,), dt)
    buf = rand(rng, (M + 40, N), out)            # rows behind the last stay as they are
    tail, r = buf[M:].clone(), buf[:M].clone()
    zt = torch.full((M + 40, N), 7.0, dtype=DT[dt], device="cuda")
    yr, yb, zr, zb = R.linear(n64(x), n64(W), n64(b), "silu", n64(r), dt, out)
    y = milo.milo_dense_linear(x, W, b, "silu", r, z=zt[:M])
    check(y, yr, yb, "y")
    check(zt[:M], zr, zb, "z")
    milo.milo_dense_linear(x, W, b, "silu", buf[:M], y=buf[:M])
    assert torch.equal(buf[:M], y) and torch.equal(buf[M:], tail) and bool((zt[M:] == 7.0).all())


@pytest.mark.parametrize("M,N", [(65, 63), (300, 66), (300, 64), (2601, 2311), (2600, 2312)])
def test_no_range_flag_from_outside_the_rows(milo, M, N):
    """Pre-activations at fp16's largest value and a residual that takes them
    back to zero: nothing is out of range, in no row or column of a ragged tile."""
    x, W = torch.zeros((M, 64), dtype=torch.float16, device="cuda"), torch.zeros((N, 64), dtype=torch.float16, device="cuda")
    b = torch.full((N,), 65504.0, dtype=torch.float16, device="cuda")
    r = torch.full((M, N), -65504.0, dtype=torch.float16, device="cuda")
    z, st = torch.empty_like(r), milo.new_status()
    y = milo.milo_dense_linear(x, W, b, "none", r, z=z, dev_status=st)
    assert not y.any() and bool((z == 65504.0).all()) and int(st.item()) == 0


@pytest.mark.parametrize("M,N,K", [(3, 24, 131072), (20, 40, 65536), (300, 40, 16384), (700, 130, 520)])
def test_long_sums_and_fp32_residuals(milo, M, N, K):
    rng = np.random.default_rng(K)
    x, W = rand(rng, (M, K), "f16"), rand(rng, (N, K), "f16", K ** -0.5)
    r, b = rand(rng, (M, N), "f32"), rand(rng, (N,), "f16")
    z = torch.empty((M, N), dtype=torch.float16, device="cuda")
    y = milo.milo_dense_linear(x, W, b, "silu", r, z=z)
    assert y.dtype == torch.float32              # the residual's type
    yr, yb, zr, zb = R.linear(n64(x), n64(W), n64(b), "silu", n64(r), "f16", "f32")
    check(y, yr, yb, "y")
    check(z, zr, zb, "z")


def test_outputs_past_32_bits(milo):
    """M * N above 2^31 elements: the last rows are where they belong."""
    M, N, K = 40000, 60000, 64
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    W = torch.randn((N, K), generator=gen, device="cuda").bfloat16()
    y = milo.milo_dense_linear(x, W)
    rows = [0, 1, M // 2, 35792, M - 1]
    want = x[rows].double() @ W.double().t()
    bound = R._rounded(n64(want), R._mma(K) * n64(x[rows].double().abs() @ W.double().abs().t()), "bf16")
    check(y[rows], n64(want), bound, "rows")
    g = milo.milo_dense_linear_backward(y, x, W, need=("db",))["db"]
    col = y[:, [0, N - 1]].double()
    err = (g[[0, N - 1]].double() - col.sum(0)).abs()
    assert (err <= 2.0 ** -8 * col.sum(0).abs() + M * 2.0 ** -24 * col.abs().sum(0) * 1.01).all()


def test_first_call_inside_a_capture():
    """A process whose first calls are captured: what the library sets up once
    (kernel attributes, occupancy) does not disturb the capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, int3_gemm_rank_b200 as milo
x = torch.randn(300, 512, device="cuda").bfloat16(); W = torch.randn(64, 512, device="cuda").bfloat16()
one = x[:2].clone()
inv = torch.arange(600, dtype=torch.int32, device="cuda")
r = {"ids": torch.zeros((300, 2), dtype=torch.int32, device="cuda"), "inv_perm": inv}
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = milo.milo_dense_linear(x, W); s = milo.milo_dense_linear(one, W)
    b = milo.milo_dense_linear_backward(y, x, W)
    xs = milo.milo_dispatch(x, r); c = milo.milo_combine(xs, r)
g.replay(); torch.cuda.synchronize()
assert torch.equal(y, milo.milo_dense_linear(x, W)) and torch.equal(s, milo.milo_dense_linear(one, W))
assert torch.equal(b["dW"], milo.milo_dense_linear_backward(y, x, W)["dW"])
assert torch.equal(c, (x.float() * 2).bfloat16())
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_nan_and_inf_stay_in_their_rows(milo):
    """A NaN or infinite row of x reaches its own output row only, at sizes with
    ragged tiles."""
    rng = np.random.default_rng(5)
    for M in (5, 200):
        x, W = rand(rng, (M, 72), "bf16"), rand(rng, (41, 72), "bf16")
        clean = milo.milo_dense_linear(x, W, out_dtype=torch.float32)
        x2 = x.clone()
        x2[3] = float("nan")
        x2[1, 5] = float("inf")
        y = milo.milo_dense_linear(x2, W, out_dtype=torch.float32)
        keep = [i for i in range(M) if i not in (1, 3)]
        assert torch.isnan(y[3]).all() and not torch.isfinite(y[1]).any()
        assert torch.equal(y[keep], clean[keep])


def test_fp16_overflow_is_flagged(milo):
    x = torch.full((3, 64), 100.0, dtype=torch.float16, device="cuda")
    W = torch.full((16, 64), 100.0, dtype=torch.float16, device="cuda")
    st = milo.new_status()
    assert torch.isinf(milo.milo_dense_linear(x, W, dev_status=st)).all()
    assert int(st.item()) == milo.MILO_DEV_FP16_RANGE
    st = milo.new_status()
    y = milo.milo_dense_linear(x, W, out_dtype=torch.float32, dev_status=st)
    assert (y == 640000.0).all() and int(st.item()) == 0


def test_results_do_not_depend_on_timing(milo):
    """The same bits on every call (split sums are joined in a fixed order)."""
    rng = np.random.default_rng(6)
    for M, N, K in ((1, 512, 4096), (300, 64, 2048), (40, 40, 8192), (2000, 24, 512)):
        x, W, dy = rand(rng, (M, K), "bf16"), rand(rng, (N, K), "bf16"), rand(rng, (M, N), "bf16")
        y = milo.milo_dense_linear(x, W, out_dtype=torch.float32)
        g = milo.milo_dense_linear_backward(dy, x, W)
        for _ in range(5):
            assert torch.equal(milo.milo_dense_linear(x, W, out_dtype=torch.float32), y)
            g2 = milo.milo_dense_linear_backward(dy, x, W)
            assert all(torch.equal(g[n], g2[n]) for n in g)


def test_captured_replayed_and_on_a_side_stream(milo):
    rng = np.random.default_rng(7)
    x, W, b = rand(rng, (48, 264), "bf16"), rand(rng, (136, 264), "bf16", 0.1), rand(rng, (136,), "bf16")
    dy = rand(rng, (48, 136), "bf16")

    def run():
        z = torch.empty((48, 136), dtype=torch.bfloat16, device="cuda")
        y = milo.milo_dense_linear(x, W, b, "gelu", z=z)
        g = milo.milo_dense_linear_backward(dy, x, W, "gelu", z)
        return [y, z, g["dx"], g["dW"], g["db"]]

    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graphs = []
    for _ in range(2):                       # two graphs, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    x.copy_(rand(rng, (48, 264), "bf16"))
    dy.copy_(rand(rng, (48, 136), "bf16"))
    want = [t.clone() for t in run()]
    for _ in range(2):
        for g, out in graphs:
            g.replay()
            assert all(torch.equal(a, c) for a, c in zip(out, want))


def test_moe_layer_with_16_bit_experts(milo):
    """A layer of 16-bit experts as it would be trained: router product,
    routing, dispatch, per expert up-projection with activation and
    down-projection, combine with the residual, and the whole way back.  Each
    step is held to its bound on the values it was given."""
    rng = np.random.default_rng(8)
    T, H, I, E, k = 150, 128, 192, 5, 2
    x = rand(rng, (T, H), "bf16")
    Wg = rand(rng, (E, H), "bf16", H ** -0.5)
    W1 = [rand(rng, (I, H), "bf16", H ** -0.5) for _ in range(E)]
    W2 = [rand(rng, (H, I), "bf16", I ** -0.5) for _ in range(E)]
    st = milo.new_status()
    logits = milo.milo_dense_linear(x, Wg, out_dtype=torch.float16, dev_status=st)
    r = milo.milo_route(logits, k, True, dev_status=st)
    xs = milo.milo_dispatch(x, r, dev_status=st)
    off = r["offsets"].tolist()
    ys, zs, hs = torch.empty((T * k, H), dtype=x.dtype, device="cuda"), [], []
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        z = torch.empty((off[e + 1] - off[e], I), dtype=x.dtype, device="cuda")
        h = milo.milo_dense_linear(xs[rows], W1[e], None, "silu", z=z, dev_status=st)
        milo.milo_dense_linear(h, W2[e], y=ys[rows], dev_status=st)
        want = R.linear(n64(h), n64(W2[e]), None, "none", None, "bf16", "bf16")
        check(ys[rows], want[0], want[1], "down")
        zs.append(z)
        hs.append(h)
    y = milo.milo_combine(ys, r, r["w"], x, dev_status=st)
    inv = n64(r["inv_perm"]).astype(int).reshape(T, k)
    check(y, *R.combine(n64(ys), inv, n64(r["w"]), n64(x), "bf16"), "y")

    dy = rand(rng, (T, H), "bf16")
    dys, dw = milo.milo_combine_backward(dy, r, ys, r["w"], dev_status=st)
    dxs = torch.empty_like(dys)
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        g2 = milo.milo_dense_linear_backward(dys[rows], hs[e], W2[e], need=("dx", "dW"), dev_status=st)
        g1 = milo.milo_dense_linear_backward(g2["dx"], xs[rows], W1[e], "silu", zs[e], need=("dx", "dW"),
                                             out={"dx": dxs[rows]}, dev_status=st)
        want = R.linear_backward(n64(g2["dx"]), n64(xs[rows]), n64(W1[e]), "silu", n64(zs[e]), "bf16", False)
        check(g1["dx"], *want["dx"], "dx")
        check(g1["dW"], *want["dW"], "dW1")
    dx, _ = milo.milo_dispatch_backward(dxs, r, dev_status=st)
    check(dx, *R.combine(n64(dxs), inv, None, None, "bf16"), "dx tokens")
    dl = milo.milo_route_backward(r, dw, True, E, dev_status=st)
    check(dl, *R.route_backward(n64(logits), n64(r["ids"]).astype(int), n64(r["w"]), n64(dw), E, True, "f16"), "dl")
    gg = milo.milo_dense_linear_backward(dl, x, Wg, need=("dx", "dW"), dev_status=st)
    want = R.linear_backward(n64(dl), n64(x), n64(Wg), "none", None, "bf16", False)
    check(gg["dW"], *want["dW"], "dWg")
    check(gg["dx"], *want["dx"], "dx router")
    assert int(st.item()) == 0
