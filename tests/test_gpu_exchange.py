"""milo_dispatch, milo_combine, their gradients and milo_route_backward on the
GPU against the plain 64-bit implementation, within its derived bounds; as one
chain around milo_grouped_linear; captured, on other streams, and with rows
past 2^31 elements."""
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


def rand(rng, shape, dt):
    return torch.from_numpy(rng.standard_normal(shape)).to(DT[dt]).cuda()


def make_route(milo, rng, T, k, E, drop):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32).reshape(T, k)
    if drop == "some":
        ids[rng.random((T, k)) < 0.3] = -1
        if T > 1:
            ids[T // 2] = -1                 # a token with no expert at all
    elif drop == "all":
        ids[:] = E
    r = milo.milo_route(None, k, False, E=E, ids=torch.from_numpy(ids).cuda())
    r["w"] = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    return r


def check(got, want, bound, what):
    err = np.abs(n64(got) - want)
    assert got.shape == want.shape and (err <= bound).all(), f"{what}: {(err - bound).max():.3e} above the bound"


# H: one column, odd, even, 16-byte rows shorter and longer than a block's pass
CASES = [(1, 1, 1, 1, "none"), (1, 2, 4096, 8, "none"), (3, 3, 7, 5, "some"), (16, 2, 64, 8, "none"),
         (37, 6, 2051, 64, "some"), (50, 16, 264, 16, "some"), (9, 9, 514, 200, "none"), (5, 2, 40, 4, "all"),
         (130, 8, 1024, 256, "none"), (2, 4, 8200, 4, "some"), (1900, 2, 1032, 8, "some"), (1000, 3, 771, 8, "some")]


@pytest.mark.parametrize("T,k,H,E,drop", CASES)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
def test_moves_and_gradients(milo, T, k, H, E, drop, dt, out):
    rng = np.random.default_rng(T * 1000 + H)
    r = make_route(milo, rng, T, k, E, drop)
    inv = r["inv_perm"].cpu().numpy().reshape(T, k).astype(int)
    w = n64(r["w"])
    st = milo.new_status()
    x, rows = rand(rng, (T, H), dt), rand(rng, (T * k, H), dt)
    res = rand(rng, (T, H), out)
    live = np.zeros(T * k, bool)
    live[inv[inv >= 0]] = True
    rows[torch.from_numpy(~live).cuda()] = float("nan")       # rows no slot points to are not read
    rows64 = np.where(live[:, None], n64(rows), 0.0)
    kept = rand(rng, (T * k, H), out)                          # and not written

    for weights in (r["w"], None):
        wn = None if weights is None else w
        xs = milo.milo_dispatch(x, r, weights, xs=kept.clone(), dev_status=st)
        check(xs, *R.dispatch(n64(x), inv, wn, out, n64(kept)), "dispatch")
        for residual in (res, None):
            y = milo.milo_combine(rows, r, weights, residual, out_dtype=DT[out], dev_status=st)
            check(y, *R.combine(rows64, inv, wn, None if residual is None else n64(res), out), "combine")
        dx, dw = milo.milo_dispatch_backward(rows, r, x, weights, out_dtype=DT[out], dev_status=st)
        check(dx, *R.combine(rows64, inv, wn, None, out), "dx")
        dys, dw2 = milo.milo_combine_backward(x, r, rows, weights, dys=kept.clone(), dev_status=st)
        check(dys, *R.dispatch(n64(x), inv, wn, out, n64(kept)), "dys")
        if weights is None:
            assert dw is None and dw2 is None
        else:
            d, b = R.slot_dots(n64(x), rows64, inv)
            check(dw, d, b, "dispatch dw")
            check(dw2, d, b, "combine dw")
    # weights without their gradient
    dys, none = milo.milo_combine_backward(x, r, None, r["w"], dys=kept.clone(), dev_status=st)
    check(dys, *R.dispatch(n64(x), inv, w, out, n64(kept)), "dys alone")
    dx, none2 = milo.milo_dispatch_backward(rows, r, None, r["w"], out_dtype=DT[out], dev_status=st)
    check(dx, *R.combine(rows64, inv, w, None, out), "dx alone")
    assert none is None and none2 is None and int(st.item()) == 0


def test_unaligned_rows_and_residual_in_place(milo):
    """A base address off by one element takes the element path; y may be the
    residual's buffer."""
    rng = np.random.default_rng(7)
    T, k, H = 11, 3, 64
    r = make_route(milo, rng, T, k, 8, "none")
    inv = r["inv_perm"].cpu().numpy().reshape(T, k).astype(int)
    buf = rand(rng, (T * H + 1,), "bf16")
    x = buf[1:].view(T, H)
    assert x.data_ptr() % 16 == 2
    xs = milo.milo_dispatch(x, r)
    check(xs, *R.dispatch(n64(x), inv, None, "bf16", np.zeros((T * k, H))), "unaligned")
    y = rand(rng, (T, H), "bf16")
    want = R.combine(n64(xs), inv, n64(r["w"]), n64(y), "bf16")
    assert milo.milo_combine(xs, r, r["w"], y, y=y) is y
    check(y, *want, "in place")


@pytest.mark.parametrize("dt,out", [("bf16", "f32"), ("f32", "f32"), ("f32", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("H", [1, 3, 5, 8, 13, 263, 515])
@pytest.mark.parametrize("so,oo", [(0, 0), (1, 0), (0, 3), (5, 2)])
def test_rows_that_start_anywhere(milo, dt, out, H, so, oo):
    """Inputs and outputs at every kind of offset inside larger buffers, widths
    that shift every row: results right, and nothing beside the outputs is
    written."""
    rng = np.random.default_rng(H)
    T, k, E = 9, 3, 6
    r = make_route(milo, rng, T, k, E, "some")
    inv = r["inv_perm"].cpu().numpy().reshape(T, k).astype(int)
    w = n64(r["w"])

    def inside(rows, d, off):
        buf = rand(rng, (rows * H + off + 16,), d)
        return buf, buf[off:off + rows * H].view(rows, H)

    _, x = inside(T, dt, so)
    _, rows = inside(T * k, dt, so)
    for name in ("dispatch", "combine", "dispatch_backward", "combine_backward"):
        expert = name in ("dispatch", "combine_backward")
        n = T * k if expert else T
        buf, o = inside(n, out, oo)
        before, was = buf.clone(), n64(o)
        _, res = inside(T, out, so)
        if name == "dispatch":
            milo.milo_dispatch(x, r, r["w"], xs=o)
            want = R.dispatch(n64(x), inv, w, out, was)
        elif name == "combine":
            milo.milo_combine(rows, r, r["w"], res, y=o)
            want = R.combine(n64(rows), inv, w, n64(res), out)
        elif name == "dispatch_backward":
            _, dw = milo.milo_dispatch_backward(rows, r, x, r["w"], dx=o)
            want = R.combine(n64(rows), inv, w, None, out)
            check(dw, *R.slot_dots(n64(x), n64(rows), inv), name)
        else:
            _, dw = milo.milo_combine_backward(x, r, rows, r["w"], dys=o)
            want = R.dispatch(n64(x), inv, w, out, was)
            check(dw, *R.slot_dots(n64(x), n64(rows), inv), name)
        check(o, *want, name)
        assert torch.equal(buf[:oo], before[:oo]) and torch.equal(buf[oo + n * H:], before[oo + n * H:]), name


def test_no_tokens(milo):
    r = {"ids": torch.empty((0, 2), dtype=torch.int32, device="cuda"), "w": torch.empty((0, 2), device="cuda"),
         "inv_perm": torch.empty(0, dtype=torch.int32, device="cuda")}
    x = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    assert milo.milo_dispatch(x, r).shape == (0, 24) and milo.milo_combine(x, r, r["w"], x).shape == (0, 24)
    for grads in (milo.milo_dispatch_backward(x, r, x, r["w"]), milo.milo_combine_backward(x, r, x, r["w"])):
        assert grads[0].shape == (0, 24) and grads[1].shape == (0, 2)
    assert milo.milo_route_backward(r, r["w"], True, 8).shape == (0, 8)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [131, 2051])
def test_residual_in_place_at_odd_widths(milo, dt, H):
    """Rows whose 16-byte pieces are shared with their neighbours', read and
    written by different warps."""
    rng = np.random.default_rng(H)
    T, k = 900, 3
    r = make_route(milo, rng, T, k, 8, "none")
    inv = r["inv_perm"].cpu().numpy().reshape(T, k).astype(int)
    rows, y = rand(rng, (T * k, H), dt), rand(rng, (T, H), dt)
    want = R.combine(n64(rows), inv, n64(r["w"]), n64(y), dt)
    milo.milo_combine(rows, r, r["w"], y, y=y)
    check(y, *want, "in place")


@pytest.mark.parametrize("H", [64, 67])
def test_weights_of_dropped_slots_do_not_matter(milo, H):
    rng = np.random.default_rng(15)
    T, k = 40, 4
    r = make_route(milo, rng, T, k, 8, "some")
    inv = r["inv_perm"].cpu().numpy().reshape(T, k).astype(int)
    w = n64(r["w"])
    bad = r["w"].clone()
    bad[torch.from_numpy(inv < 0).cuda()] = float("nan")
    x, rows = rand(rng, (T, H), "bf16"), rand(rng, (T * k, H), "bf16")
    zero = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
    z64 = np.zeros((T * k, H))
    check(milo.milo_dispatch(x, r, bad, xs=zero.clone()), *R.dispatch(n64(x), inv, w, "bf16", z64), "dispatch")
    check(milo.milo_combine(rows, r, bad), *R.combine(n64(rows), inv, w, None, "bf16"), "combine")
    dx, dw = milo.milo_dispatch_backward(rows, r, x, bad)
    check(dx, *R.combine(n64(rows), inv, w, None, "bf16"), "dx")
    check(dw, *R.slot_dots(n64(x), n64(rows), inv), "dw")
    dys, dw = milo.milo_combine_backward(x, r, rows, bad, dys=zero.clone())
    check(dys, *R.dispatch(n64(x), inv, w, "bf16", z64), "dys")
    check(dw, *R.slot_dots(n64(x), n64(rows), inv), "dw")


def test_bad_rows_are_flagged_and_skipped(milo):
    rng = np.random.default_rng(8)
    T, k, H = 4, 2, 32
    r = make_route(milo, rng, T, k, 4, "none")
    inv = r["inv_perm"].clone()
    inv[3], inv[5] = T * k, -7
    r = dict(r, inv_perm=inv)
    good = np.where((n := inv.cpu().numpy().reshape(T, k).astype(int)) >= T * k, -1, n)
    good = np.where(good < 0, -1, good)
    x, rows, kept = rand(rng, (T, H), "bf16"), rand(rng, (T * k, H), "bf16"), rand(rng, (T * k, H), "bf16")
    w = n64(r["w"])
    for name in ("dispatch", "combine", "dispatch_backward", "combine_backward"):
        st = milo.new_status()
        if name == "dispatch":
            check(milo.milo_dispatch(x, r, r["w"], xs=kept.clone(), dev_status=st),
                  *R.dispatch(n64(x), good, w, "bf16", n64(kept)), name)
        elif name == "combine":
            check(milo.milo_combine(rows, r, r["w"], dev_status=st), *R.combine(n64(rows), good, w, None, "bf16"), name)
        elif name == "dispatch_backward":
            dx, dw = milo.milo_dispatch_backward(rows, r, x, r["w"], dev_status=st)
            check(dw, *R.slot_dots(n64(x), n64(rows), good), name)
        else:
            dys, dw = milo.milo_combine_backward(x, r, rows, r["w"], dys=kept.clone(), dev_status=st)
            check(dys, *R.dispatch(n64(x), good, w, "bf16", n64(kept)), name)
            check(dw, *R.slot_dots(n64(x), n64(rows), good), name)
        assert int(st.item()) == milo.MILO_DEV_BOUNDS, name


def test_fp16_overflow_is_flagged(milo):
    rng = np.random.default_rng(9)
    r = make_route(milo, rng, 4, 2, 4, "none")
    rows = torch.full((8, 16), 60000.0, device="cuda")
    st = milo.new_status()
    y = milo.milo_combine(rows, r, None, out_dtype=torch.float16, dev_status=st)
    assert torch.isinf(y).all() and int(st.item()) == milo.MILO_DEV_FP16_RANGE
    st = milo.new_status()
    x = torch.full((4, 16), float("inf"), device="cuda")        # an infinity is not an overflow
    assert torch.isinf(milo.milo_dispatch(x, r, out_dtype=torch.float16, dev_status=st)).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 64, 6), (300, 33, 16), (65, 256, 16), (1000, 256, 1)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("out", ["f16", "f32", "bf16"])
def test_route_backward(milo, T, E, k, renorm, out):
    rng = np.random.default_rng(T + E + k)
    logits = rand(rng, (T, E), "f16")
    st = milo.new_status()
    r = milo.milo_route(logits, k, renorm, dev_status=st)
    dw = rand(rng, (T, k), "f32")
    dl = milo.milo_route_backward(r, dw, renorm, E, None if renorm else logits, out_dtype=DT[out], dev_status=st)
    want, bound = R.route_backward(n64(logits), n64(r["ids"]).astype(int), n64(r["w"]), n64(dw), E, renorm, out)
    check(dl, want, bound, "dlogits")
    assert int(st.item()) == 0


def test_route_backward_extremes(milo):
    """Masked logits (the type's lowest value), equal logits, one expert far
    ahead; ids outside the experts."""
    rng = np.random.default_rng(11)
    T, E, k = 6, 40, 3
    logits = rand(rng, (T, E), "f16")
    logits[0, 5:] = -65504.0
    logits[1] = 0.5
    logits[2, 7] = 60.0
    logits[3, :] = -65504.0
    logits[3, :k] = 1.0
    st = milo.new_status()
    for renorm in (True, False):
        r = milo.milo_route(logits, k, renorm, dev_status=st)
        dw = rand(rng, (T, k), "f32")
        dl = milo.milo_route_backward(r, dw, renorm, E, logits, out_dtype=torch.float32, dev_status=st)
        want, bound = R.route_backward(n64(logits), n64(r["ids"]).astype(int), n64(r["w"]), n64(dw), E, renorm, "f32")
        check(dl, want, bound, "dlogits")
    assert int(st.item()) == 0
    ids = r["ids"].clone()
    ids[4, 1] = E
    got = milo.milo_route_backward(dict(r, ids=ids), dw, True, E, out_dtype=torch.float32, dev_status=st)
    assert int(st.item()) == milo.MILO_DEV_BAD_EXPERT_ID
    w2 = n64(r["w"])
    w2[4, 1] = 0.0
    i2 = n64(r["ids"]).astype(int)
    want, bound = R.route_backward(n64(logits), i2, w2, n64(dw), E, True, "f32")
    check(got, want, bound, "bad id")
    st = milo.new_status()
    bad = logits.clone()
    bad[2, 3] = float("nan")
    milo.milo_route_backward(r, dw, False, E, bad, dev_status=st)
    assert int(st.item()) & milo.MILO_DEV_NONFINITE


def test_route_backward_of_repeated_picks(milo):
    """Ids a caller made up: a token's two or three picks of one expert add up,
    in the same bits every time."""
    rng = np.random.default_rng(14)
    T, E, k = 70, 12, 5
    ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).cuda()
    ids[3] = 7
    r = {"ids": ids, "w": rand(rng, (T, k), "f32")}
    dw = rand(rng, (T, k), "f32")
    logits = rand(rng, (T, E), "f16")
    dl = milo.milo_route_backward(r, dw, False, E, logits, out_dtype=torch.float32)
    lg, w = n64(logits), n64(r["w"])
    p = np.exp(lg - lg.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    want = -p * (w * n64(dw)).sum(1, keepdims=True)
    np.add.at(want, (np.arange(T)[:, None], ids.cpu().numpy()), w * n64(dw))
    # as R.route_backward: (k + 4) 2^-24 of the terms and 2^-18 + E 2^-24 of p |s|, all at most mag
    mag = np.abs(w * n64(dw)).sum(1, keepdims=True) + 0 * want
    check(dl, want, 2.0 ** -17 * mag, "repeated")
    for _ in range(3):
        assert torch.equal(milo.milo_route_backward(r, dw, False, E, logits, out_dtype=torch.float32), dl)


def test_chain_around_the_grouped_linear(milo):
    """route -> dispatch -> grouped int3 product over the grouped rows ->
    combine: the slots' rows are bit for bit those of the ungrouped call, and
    the combine is within its bound of them."""
    import workloads as wl
    from parity_util import f16_dev
    rng = np.random.default_rng(12)
    T, k, E = 21, 2, 4
    P = [wl.make_projection("t_chain", "w", e, 256, 384, rk) for e, rk in enumerate((16, 0, 8, 32))]
    lin = milo.GroupedLinear([milo.QWeight.quantize(f16_dev(p.W), f16_dev(p.U) if p.rank else None,
                                                    f16_dev(p.V) if p.rank else None) for p in P])
    x, logits = rand(rng, (T, 384), "bf16"), rand(rng, (T, E), "f16")
    st = milo.new_status()
    r = milo.milo_route(logits, k, True, dev_status=st)
    xs = milo.milo_dispatch(x, r, dev_status=st)
    ys = lin(xs, r["offsets"], None, dev_status=st)
    slots = lin(x, r["offsets"], r["perm"], k=k, dev_status=st)
    inv = r["inv_perm"].long()
    assert torch.equal(ys[inv], slots)
    res = rand(rng, (T, 256), "f32")
    y = milo.milo_combine(ys, r, r["w"], res, dev_status=st)
    check(y, *R.combine(n64(ys), inv.cpu().numpy().reshape(T, k), n64(r["w"]), n64(res), "f32"), "combine")
    # backwards: the output's gradient to the expert rows, the weights and the logits
    dy = rand(rng, (T, 256), "f32")
    dys, dw = milo.milo_combine_backward(dy, r, ys, r["w"], dev_status=st)
    i2 = inv.cpu().numpy().reshape(T, k)
    check(dys, *R.dispatch(n64(dy), i2, n64(r["w"]), "f32", np.zeros((T * k, 256))), "dys")
    check(dw, *R.slot_dots(n64(dy), n64(ys), i2), "dw")
    dl = milo.milo_route_backward(r, dw, True, E, out_dtype=torch.float32, dev_status=st)
    check(dl, *R.route_backward(n64(logits), n64(r["ids"]).astype(int), n64(r["w"]), n64(dw), E, True, "f32"), "dl")
    assert int(st.item()) == 0


def test_captured_replayed_and_on_a_side_stream(milo):
    rng = np.random.default_rng(13)
    T, k, H = 33, 4, 520
    r = make_route(milo, rng, T, k, 8, "none")
    x, rows = rand(rng, (T, H), "bf16"), rand(rng, (T * k, H), "bf16")

    def run():
        xs = milo.milo_dispatch(x, r)
        y = milo.milo_combine(rows, r, r["w"], x)
        dx, dw = milo.milo_dispatch_backward(rows, r, x, r["w"])
        dys, dw2 = milo.milo_combine_backward(x, r, rows, r["w"])
        dl = milo.milo_route_backward(r, dw2, True, 8)
        return xs, y, dx, dw, dys, dw2, dl

    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    x.copy_(rand(rng, (T, H), "bf16"))
    rows.copy_(rand(rng, (T * k, H), "bf16"))
    want = [t.clone() for t in run()]
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_offsets_past_32_bits(milo):
    """T*k*H above 2^31 elements: the last expert rows are where they belong."""
    T, k, H = 70000, 8, 4096
    inv = (torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k).flip(0)).reshape(-1).contiguous()
    r = {"ids": torch.zeros((T, k), dtype=torch.int32, device="cuda"), "inv_perm": inv}
    x = torch.randn((T, H), device="cuda", dtype=torch.bfloat16)
    xs = milo.milo_dispatch(x, r)
    for t in (0, 1, T // 2, T - 2, T - 1):
        for j in (0, k - 1):
            assert torch.equal(xs[(T - 1 - t) * k + j], x[t])
    y = milo.milo_combine(xs, r)
    w = torch.ones((T, k), device="cuda")
    dx, dw = milo.milo_dispatch_backward(xs, r, x, w)
    assert torch.equal(dx, y)
    for t in (0, T - 1):
        assert torch.equal(y[t], (x[t].float() * k).bfloat16())
    d = (x[0].double() ** 2).sum()
    assert abs(float(dw[0, k - 1]) - float(d)) <= H * 2.0 ** -24 * float(d)
