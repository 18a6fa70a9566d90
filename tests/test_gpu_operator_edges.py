"""Edges of the 16-bit operators on the GPU that their main suites do not reach:
what a kernel leaves under way when it ends, flags of rows that do not exist,
far tails of the activations, calls beside the library's other kernels."""
import math

import numpy as np
import pytest

import operator_ref as R
from test_gpu_dense import check, milo, n64, rand      # noqa: F401 (milo is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_pairs_of_ctas_end_with_nothing_under_way(milo):
    """Pairs of CTAs (both products of a gradient, a product alone; fewer slices
    than stages, and more) whose SMs go at once to other kernels with barriers
    in the same places: every commit's arrival has landed before its CTA left,
    so no later kernel's barrier gets one too many."""
    rng = np.random.default_rng(21)
    pairs = []
    for M, N, K in ((2600, 2312, 72), (2600, 2312, 648), (4100, 1032, 136)):
        x, W, dy = rand(rng, (M, K), "bf16"), rand(rng, (N, K), "bf16", K ** -0.5), rand(rng, (M, N), "bf16")
        pairs.append((x, W, dy, milo.milo_dense_linear(x, W), milo.milo_dense_linear_backward(dy, x, W)))
    x, W = rand(rng, (300, 2048), "bf16"), rand(rng, (64, 2048), "bf16")          # a split sum
    x1, W1 = rand(rng, (40, 512), "bf16"), rand(rng, (2048, 512), "bf16")         # tokens as columns
    y, y1 = milo.milo_dense_linear(x, W), milo.milo_dense_linear(x1, W1)
    st = milo.new_status()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(24):
        with torch.cuda.stream(streams[i % 2]):
            a, b, dy, want, g = pairs[i % 3]
            got.append((milo.milo_dense_linear(a, b, dev_status=st), want))
            got.append((milo.milo_dense_linear(x, W, dev_status=st), y))
            g2 = milo.milo_dense_linear_backward(dy, a, b, dev_status=st)
            got += [(g2[n], g[n]) for n in g]
            got.append((milo.milo_dense_linear(x1, W1, dev_status=st), y1))
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert all(torch.equal(a, b) for a, b in got)


@pytest.mark.parametrize("H", [63, 331, 2051])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_at_both_ends_of_a_tensor_off_16_bytes(milo, H, dt):
    """Tensors whose first and last bytes lie inside a 16-byte piece: the rows
    there come in part element by element, into places of the ring that bulk
    copies fill before and after.  Without weights every element is a copy."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(22)
    T, k = 9001, 2
    # both ends of the expert rows among the first items of a warp
    ends = torch.tensor([0, T * k - 1], device="cuda")
    perm = torch.cat([ends, 1 + torch.randperm(T * k - 2, generator=gen, device="cuda")]).int()
    route = {"ids": torch.zeros((T, k), dtype=torch.int32, device="cuda"), "inv_perm": perm}

    def off(rows):                                 # rows at an odd element of a buffer
        return torch.randn(rows * H + 1, generator=gen, device="cuda").to(dt)[1:].view(rows, H)

    x, ys = off(T), off(T * k)
    p = perm.long()
    st = milo.new_status()
    for _ in range(3):
        xs = milo.milo_dispatch(x, route, dev_status=st)
        assert torch.equal(xs[p], x.repeat_interleave(k, 0))
        y = milo.milo_combine(ys, route, dev_status=st)
        assert torch.equal(y, (ys[p[0::2]].float() + ys[p[1::2]].float()).to(dt))
    assert int(st.item()) == 0


@pytest.mark.parametrize("M,N", [(17, 64), (65, 64), (65, 63), (300, 64), (300, 66), (301, 63), (2600, 2312), (2601, 2312),
                                 (2601, 2311), (20001, 120), (20001, 121)])
def test_no_range_flag_from_a_bias_above_fp16(milo, M, N):
    """bf16 operands, an fp16 output: a bias that fp16 does not hold, taken back
    into range by the residual in every row there is, flags nothing -- the rows
    that fill up a ragged block have the bias but no residual.  One row without
    the residual does flag."""
    x, W = torch.zeros((M, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((N, 64), dtype=torch.bfloat16, device="cuda")
    b = torch.full((N,), 1e5, dtype=torch.bfloat16, device="cuda")
    r = torch.full((M, N), -65000.0, dtype=torch.float16, device="cuda")
    st = milo.new_status()
    y = milo.milo_dense_linear(x, W, b, "none", r, dev_status=st)
    want = torch.tensor(float(b[0]) + float(r[0, 0])).half().item()
    assert bool((y == want).all()) and int(st.item()) == 0
    r[M - 1] = 0.0
    y = milo.milo_dense_linear(x, W, b, "none", r, dev_status=st)
    assert bool(torch.isinf(y[M - 1]).all()) and bool((y[:M - 1] == want).all())
    assert int(st.item()) == milo.MILO_DEV_FP16_RANGE


@pytest.mark.parametrize("M", [8, 200])
@pytest.mark.parametrize("dt,out", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_gelu_far_below_zero_relative_to_its_value(milo, M, dt, out):
    """gelu(z) = z erfc(-z / sqrt 2) / 2 and its slope from -3 down to where fp32 still
    holds them as normal numbers, relative to their values.  In fp32 the argument
    is off by 2^-23 (constant and product), which erfc multiplies by at most
    z^2 + 1; erfcf is within 4 steps of 2^-23, the two products 2^-24 each: (z^2 +
    6) 2^-23.  In the slope Phi + z phi, |z phi| >= 9 Phi here; exp is off by
    z^2 / 2 times 2^-23 from its argument, 2^-21 of its own with the products."""
    v = np.resize(-np.linspace(3.0, 12.0, 64), (M, 64)) * (1.0 + np.arange(M)[:, None] * 1e-4)
    x = torch.from_numpy(v).to(torch.bfloat16 if dt == "bf16" else torch.float16).cuda()
    W = torch.eye(64, dtype=x.dtype, device="cuda")
    z = n64(x)
    Phi = 0.5 * np.vectorize(math.erfc)(-z / math.sqrt(2.0))
    zphi = z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    y = milo.milo_dense_linear(x, W, None, "gelu", out_dtype={"bf16": torch.bfloat16, "f32": torch.float32}[out])
    rel = (z * z + 6.0) * 2.0 ** -23
    check(y, z * Phi, np.abs(z * Phi) * (rel + R.U[out] * (1.0 + rel)), "y")
    if dt == "bf16" and out == "bf16":
        dy = torch.ones((M, 64), dtype=torch.bfloat16, device="cuda")
        s = Phi + zphi
        err = rel * Phi + (z * z * 2.0 ** -24 + 2.0 ** -21) * np.abs(zphi)
        dx = milo.milo_dense_linear_backward(dy, x, W, "gelu", x, need=("dx",))["dx"]
        check(dx, s, err + R.U["bf16"] * (np.abs(s) + err), "dx")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", [8, 200])
def test_silu_and_gelu_tanh_relative_to_their_values(milo, act, M):
    """fp32 outputs from deep in the negative tail up: with v the exponential's
    argument, ex2 is within 2^-22.5, its argument (product and constant) 1.3 2^-24 |v|,
    the sum 2^-24, the reciprocal 2^-23, the product 2^-24: below (5 + |v|) 2^-23 for
    silu.  gelu_tanh's v has five roundings of 2^-24 at most of its own: (5 + 4 |v|)
    2^-23."""
    low = -80.0 if act == "silu" else -9.0
    v = np.resize(np.linspace(low, 9.0, 251), (M, 64))
    x = torch.from_numpy(v).bfloat16().cuda()
    W = torch.eye(64, dtype=x.dtype, device="cuda")
    z = n64(x)
    u = z if act == "silu" else math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3)
    want = z / (1.0 + np.exp(-u))
    y = milo.milo_dense_linear(x, W, None, act, out_dtype=torch.float32)
    rel = (5.0 + (1.0 if act == "silu" else 4.0) * np.abs(u)) * 2.0 ** -23
    check(y, want, np.abs(want) * (rel + R.U["f32"] * (1.0 + rel)), act)


@pytest.mark.parametrize("M", [8, 200])
def test_gelu_over_its_range_and_at_its_ends(milo, M):
    """Every few bf16 values of [-13, 13]: gelu(z) = max(z, 0) - |z| Phi(-|z|) and the
    slope's Phi and z phi.  Phi(-a) is within (a^2 + 9) 2^-23 of its value, relative
    to it: the exponential's argument a^2 / 2 times 2^-23, the exponential 2^-22.5,
    the reciprocal 2^-23 and its argument 2^-24, each at most 3.2 times (the slope of ln
    r over ln t, largest at 0), the fit and the Horner steps 2^-23, two products.
    Infinities give the limits, NaN stays NaN."""
    zs = torch.arange(0x3A00, 0x4150, 8 if M == 8 else 1, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)   # 4.9e-4 to 13
    zs = torch.cat([zs, -zs])
    v = zs.repeat(-(-M * 64 // len(zs)))[:M * 64]
    x = v.view(M, 64).cuda()
    W = torch.eye(64, dtype=x.dtype, device="cuda")
    z = n64(x)
    a = np.abs(z)
    q = 0.5 * np.vectorize(math.erfc)(a / math.sqrt(2.0))
    eq = q * (a * a + 9.0) * 2.0 ** -23 + 2.0 ** -126          # below the normal range flushed
    y = np.maximum(z, 0.0) - a * q
    got = milo.milo_dense_linear(x, W, None, "gelu", out_dtype=torch.float32)
    check(got, y, a * eq + 2.0 ** -24 * np.abs(y) + 2.0 ** -149, "y")
    dy = torch.ones_like(x)
    s = np.where(z > 0, 1.0 - q, q) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    # e (r - a / sqrt(2 pi)): as q, and the same for a phi; the 1 - of the upper half
    es = eq + a * np.exp(-0.5 * z * z) * 0.4 * (a * a + 9.0) * 2.0 ** -23 + 2.0 ** -24 + a * 2.0 ** -126
    dx = milo.milo_dense_linear_backward(dy, x, W, "gelu", x, need=("dx",))["dx"]
    check(dx, s, es + R.U["bf16"] * (np.abs(s) + es), "dx")

    ends = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 1e30, -1e30, 3e38], dtype=torch.bfloat16)
    b = ends.repeat(8).cuda()
    zero = torch.zeros((M, 64), dtype=torch.bfloat16, device="cuda")
    y = milo.milo_dense_linear(zero, W, b, "gelu", out_dtype=torch.float32)
    want = torch.tensor([math.inf, 0.0, math.nan, 0.0, 0.0, float(ends[5]), 0.0, float(ends[7])]).repeat(M, 8).cuda()
    assert torch.equal(torch.nan_to_num(y, nan=7.0, posinf=8.0), torch.nan_to_num(want, nan=7.0, posinf=8.0))
    db = milo.milo_dense_linear_backward(dy[:1], x[:1], W, "gelu", b.view(1, 64), need=("db",))["db"]
    want = torch.tensor([1.0, 0.0, math.nan, 0.5, 0.5, 1.0, 0.0, 1.0]).repeat(8).cuda()
    assert torch.equal(torch.nan_to_num(db.float(), nan=7.0), torch.nan_to_num(want, nan=7.0))


def test_small_products_beside_the_grouped_gemm(milo):
    """The grouped int3 GEMM on the tensor cores (all TMEM columns of its SMs) on
    two streams, small dense products (tokens as columns, split over clusters)
    and pairs of CTAs on two others: each as alone, no wait runs out."""
    import workloads as wl
    from parity_util import f16_dev
    rng = np.random.default_rng(23)
    P = [wl.make_projection("t_mix", "w", e, 512, 1024, rk) for e, rk in enumerate((16, 0, 32, 8))]
    lin = milo.GroupedLinear([milo.QWeight.quantize(f16_dev(p.W), f16_dev(p.U) if p.rank else None,
                                                    f16_dev(p.V) if p.rank else None) for p in P])
    T, k = 3000, 2
    x, logits = rand(rng, (T, 1024), "bf16"), rand(rng, (T, 4), "f16")
    st = milo.new_status()
    r = milo.milo_route(logits, k, True, dev_status=st)
    dense = [(rand(rng, (M, K), "bf16"), rand(rng, (N, K), "bf16", K ** -0.5))
             for M, N, K in ((20, 512, 4096), (64, 2816, 2048), (300, 64, 2048), (2600, 2312, 264))]
    milo.milo_set_gemm_path("tc")
    try:
        want = lin(x, r["offsets"], r["perm"], k=k, dev_status=st)
        ys = [milo.milo_dense_linear(a, b, dev_status=st) for a, b in dense]
        # a workspace of its own for each of the two streams
        linears = [lin, milo.GroupedLinear(lin.weights)]
        for g in linears:
            g(x, r["offsets"], r["perm"], k=k)
        streams = [torch.cuda.Stream() for _ in range(4)]
        torch.cuda.synchronize()
        got = []
        for i in range(20):
            for j in (0, 1):
                with torch.cuda.stream(streams[j]):
                    got.append((linears[j](x, r["offsets"], r["perm"], k=k, dev_status=st), want))
            for j in (2, 3):
                with torch.cuda.stream(streams[j]):
                    for (a, b), y in zip(dense, ys):
                        got.append((milo.milo_dense_linear(a, b, dev_status=st), y))
        torch.cuda.synchronize()
    finally:
        milo.milo_set_gemm_path("auto")
    assert int(st.item()) == 0 and all(torch.equal(a, b) for a, b in got)
