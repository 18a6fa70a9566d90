"""The timed calls of the 16-bit operators around the int3 MoE layer: the dense
product with its epilogue (milo_dense_linear and its gradients), the move of
token rows into expert order and back (milo_dispatch, milo_combine and their
gradients) and the router's gradient (milo_route_backward).

With `own` false every operator is computed in its plain form, elementary torch
operations in 32 bits rounded once at the end; with `own` true the same inputs
go through the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token through a square 16-bit projection with its residual (an
        # attention output projection beside a Mixtral-shaped layer): latency
        # and the weight's bytes
        dict(name="linear_token", op="linear", M=1, N=4096, K=4096, dtype="bf16", out="bf16", bias=False,
             act="none", residual=True, z=False),
        # a decode batch through the two DeepSeekMoE-shaped shared experts'
        # up-projection, fp16
        dict(name="linear_decode", op="linear", M=64, N=2816, K=2048, dtype="f16", out="f16", bias=False,
             act="silu", residual=False, z=False),
        # router logits of a ragged batch: few outputs, fp16 as milo_route takes them
        dict(name="linear_router", op="linear", M=4999, N=64, K=2048, dtype="bf16", out="f16", bias=True,
             act="none", residual=False, z=False),
        # the up-projection of a Mixtral-shaped expert kept in 16 bits, prefill
        dict(name="linear_prefill", op="linear", M=8192, N=14336, K=4096, dtype="bf16", out="bf16", bias=True,
             act="gelu_tanh", residual=False, z=False),
        # gradients of a square projection with an activation, a training batch
        dict(name="linear_grad", op="linear_backward", M=8192, N=4096, K=4096, dtype="bf16", bias=True, act="silu"),
        # gradients at sizes that fill no tile evenly, fp16
        dict(name="linear_grad_ragged", op="linear_backward", M=1531, N=1411, K=2056, dtype="f16", bias=True,
             act="relu"),
        # a Mixtral-shaped decode batch into expert order: launch latency
        dict(name="dispatch_decode", op="dispatch", T=16, H=4096, E=8, k=2, dtype="bf16", out="bf16", weights=False,
             drop=0.0),
        # prefill of a DeepSeekMoE-shaped layer: back to token order, router
        # weights applied, the residual stream added
        dict(name="combine_prefill", op="combine", T=8192, H=2048, E=64, k=6, dtype="bf16", out="bf16",
             weights=True, drop=0.0, residual=True),
        # training, Mixtral-shaped: the experts' input gradients back to token order
        dict(name="dispatch_grad", op="dispatch_backward", T=8192, H=4096, E=8, k=2, dtype="bf16", out="bf16",
             weights=False, drop=0.0),
        # training with a ragged batch, an odd width and slots dropped at the
        # experts' capacity: gradients of the expert rows and of the router weights
        dict(name="combine_grad_ragged", op="combine_backward", T=5003, H=2051, E=64, k=6, dtype="f16", out="f16",
             weights=True, drop=0.05),
        # the router's gradient of a small renormalised batch
        dict(name="route_grad_small", op="route_backward", T=256, E=8, k=2, renorm=True, out="f16"),
        # the same over many tokens, full softmax
        dict(name="route_grad", op="route_backward", T=65536, E=64, k=6, renorm=False, out="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MAX_MACS = 8192 * 14336 * 4096        # the largest listed product
MAX_ROW_ELEMS = 8192 * 6 * 2048       # the largest listed move


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "linear_backward", "linear_backward", "dispatch", "combine",
                     "dispatch_backward", "combine_backward", "route_backward"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("linear", "linear_backward"):
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
        macs = MAX_MACS // (2 if op == "linear_backward" else 1)
        while True:
            M, N = _log(rng, 1, 8192), _log(rng, 1, 14336)
            K = 8 * _log(rng, 8, 1792)
            if rng.random() < 0.5:
                N = max(8, N // 8 * 8)
            if M * N * K <= macs:
                break
        c = dict(op=op, M=M, N=N, K=K, dtype=dtype, bias=rng.random() < 0.5, act=act)
        if op == "linear":
            c.update(out=rng.choice([dtype, dtype, dtype, "f32", "f16"]), residual=rng.random() < 0.5,
                     z=act != "none" and rng.random() < 0.3)
        return c
    k = rng.randint(1, 8)
    E = max(k, _log(rng, 2, 256))
    if op == "route_backward":
        T = min(_log(rng, 1, 65536), 65536 * 64 // E)
        return dict(op=op, T=T, E=E, k=k, renorm=rng.random() < 0.5, out=rng.choice(["f16", "f32"]))
    while True:
        T, H = _log(rng, 1, 16384), _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = H // 8 * 8
        if T * k * H <= MAX_ROW_ELEMS:
            break
    c = dict(op=op, T=T, H=H, E=E, k=k, dtype=dtype, out=rng.choice([dtype, dtype, "f32"]),
             weights=op in ("combine", "combine_backward") or rng.random() < 0.3,
             drop=rng.choice([0.0, 0.0, 0.1]))
    if op == "combine":
        c["residual"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _route(gen, case):
    """Routing of T tokens over E experts, k picks each: logits with a fixed
    skew per expert, ids by descending logit, weights by softmax, and the
    grouping (expert offsets, slots in expert order, its inverse).  A share
    `drop` of the slots has no expert (id -1)."""
    T, E, k = case["T"], case["E"], case["k"]
    bias = torch.randn(E, generator=gen, device="cuda") * 0.5
    logits = (torch.randn((T, E), generator=gen, device="cuda") + bias).half()
    lf = logits.float()
    ids = torch.sort(lf, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.exp(lf - lf.max(dim=1, keepdim=True).values)
    pk = torch.gather(p, 1, ids)
    w = pk / (pk.sum(1, keepdim=True) if case.get("renorm", True) else p.sum(1, keepdim=True))
    if case.get("drop", 0.0) > 0.0:
        gone = torch.rand((T, k), generator=gen, device="cuda") < case["drop"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    flat = ids.reshape(-1)
    order = torch.sort(torch.where(flat < 0, torch.full_like(flat, E), flat), stable=True).indices
    n = int((flat >= 0).sum())
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat[flat >= 0], minlength=E), 0).int()
    inv = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    inv[order[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    return logits, dict(ids=ids.int().contiguous(), w=w.contiguous(), offsets=offsets, perm=order.int(),
                        inv_perm=inv)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("linear", "linear_backward"):
        M, N, K, dt = case["M"], case["N"], case["K"], DTYPES[case["dtype"]]
        s["x"] = _normal(gen, (M, K), 1.0, dt)
        s["W"] = _normal(gen, (N, K), 0.02, dt)
        s["bias"] = _normal(gen, (N,), 0.1, dt) if case["bias"] else None
        if op == "linear":
            s["residual"] = _normal(gen, (M, N), 1.0, DTYPES[case["out"]]) if case["residual"] else None
        else:
            s["dy"] = _normal(gen, (M, N), 1.0, dt)
            # the pre-activations that the forward call kept
            s["z"] = _normal(gen, (M, N), 0.02 * math.sqrt(K), dt) if case["act"] != "none" else None
        return s
    if op == "route_backward":
        s["logits"], s["route"] = _route(gen, case)
        s["dw"] = torch.randn((case["T"], case["k"]), generator=gen, device="cuda")
        return s
    T, H, k, dt, out = case["T"], case["H"], case["k"], DTYPES[case["dtype"]], DTYPES[case["out"]]
    _, s["route"] = _route(gen, case)
    s["w"] = s["route"]["w"] if case["weights"] else None
    # rows behind the last expert's stay as the caller's buffer has them
    s["rows_out"] = (torch.zeros((T * k, H), dtype=out, device="cuda")
                     if op in ("dispatch", "combine_backward") and case["drop"] > 0.0 else None)
    if op == "dispatch":
        s["x"] = _normal(gen, (T, H), 1.0, dt)
    elif op == "combine":
        s["ys"] = _normal(gen, (T * k, H), 1.0, dt)
        s["residual"] = _normal(gen, (T, H), 1.0, out) if case["residual"] else None
    elif op == "dispatch_backward":
        s["dxs"] = _normal(gen, (T * k, H), 1.0, dt)
        s["x"] = _normal(gen, (T, H), 1.0, dt) if case["weights"] else None
    else:
        s["dy"] = _normal(gen, (T, H), 1.0, dt)
        s["ys"] = _normal(gen, (T * k, H), 1.0, dt)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _dact(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        z = s["x"].float() @ s["W"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(case["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        y = y.to(DTYPES[case["out"]])
        return (y, z.to(s["x"].dtype)) if case["z"] else y
    if op == "linear_backward":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _dact(case["act"], s["z"].float())
        dt = s["x"].dtype
        out = [(dz @ s["W"].float()).to(dt), (dz.t() @ s["x"].float()).to(dt)]
        return out + [dz.sum(0).to(dt)] if case["bias"] else out
    r = s["route"]
    T, k = r["ids"].shape
    if op == "route_backward":
        g = r["w"] * s["dw"]
        total = g.sum(1, keepdim=True)
        ids = r["ids"].long()
        if case["renorm"]:
            dl = torch.zeros((T, case["E"]), device=g.device).scatter_(1, ids, g - r["w"] * total)
        else:
            lf = s["logits"].float()
            p = torch.exp(lf - lf.max(1, keepdim=True).values)
            p = p / p.sum(1, keepdim=True)
            dl = (-p * total).scatter_add_(1, ids, g)
        return dl.to(DTYPES[case["out"]])
    out = DTYPES[case["out"]]
    slots = r["perm"].long()
    inv = r["inv_perm"].long()
    w = None if s["w"] is None else s["w"].reshape(-1)
    if op in ("combine", "dispatch_backward"):
        src = s["ys"] if op == "combine" else s["dxs"]
        rows = src.float()[inv.clamp(min=0)]
        if case["drop"] > 0.0:
            rows = rows * (inv >= 0)[:, None]
        weighted = rows if w is None else rows * w[:, None]
        y = weighted.view(T, k, -1).sum(1)
        if op == "combine":
            if s["residual"] is not None:
                y = y + s["residual"].float()
            return y.to(out)
        if w is None:
            return y.to(out)
        return y.to(out), (rows.view(T, k, -1) * s["x"].float()[:, None, :]).sum(2)
    src = s["x"] if op == "dispatch" else s["dy"]
    rows = src.float()[torch.div(slots, k, rounding_mode="floor")]
    dw = None
    if op == "combine_backward":
        dw = torch.zeros(T * k, device=rows.device)
        dw[slots] = (rows * s["ys"].float()).sum(1)
        dw = torch.where(inv >= 0, dw, torch.zeros_like(dw)).view(T, k)
    if w is not None:
        rows = rows * w[slots, None]
    rows = rows.to(out)
    if s["rows_out"] is not None:
        # the dropped slots stand last: their rows keep what the buffer held
        live = torch.arange(T * k, device=rows.device) < r["offsets"][-1]
        rows = torch.where(live[:, None], rows, s["rows_out"])
    return rows if dw is None else (rows, dw)


def _calls(s):
    import int3_gemm_rank_b200 as milo
    case = s["case"]
    op = case["op"]
    if op == "linear":
        z = torch.empty((case["M"], case["N"]), dtype=s["x"].dtype, device=s["x"].device) if case["z"] else None
        y = milo.milo_dense_linear(s["x"], s["W"], s["bias"], case["act"], s["residual"],
                                   out_dtype=DTYPES[case["out"]], z=z)
        return (y, z) if case["z"] else y
    if op == "linear_backward":
        need = ("dx", "dW", "db") if case["bias"] else ("dx", "dW")
        g = milo.milo_dense_linear_backward(s["dy"], s["x"], s["W"], case["act"], s["z"], need=need)
        return [g[name] for name in need]
    if op == "route_backward":
        return milo.milo_route_backward(s["route"], s["dw"], case["renorm"], case["E"], s["logits"],
                                        out_dtype=DTYPES[case["out"]])
    out = DTYPES[case["out"]]
    if op == "dispatch":
        return milo.milo_dispatch(s["x"], s["route"], s["w"], out_dtype=out, xs=s["rows_out"])
    if op == "combine":
        return milo.milo_combine(s["ys"], s["route"], s["w"], s["residual"], out_dtype=out)
    if op == "dispatch_backward":
        dx, dw = milo.milo_dispatch_backward(s["dxs"], s["route"], s["x"], s["w"], out_dtype=out)
        return dx if dw is None else (dx, dw)
    return milo.milo_combine_backward(s["dy"], s["route"], s["ys"], s["w"], out_dtype=out, dys=s["rows_out"])


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = lambda t: t.double()
    if op in ("linear", "linear_backward"):
        act = case["act"]
        if op == "linear":
            z = torch.matmul(d(s["x"]), d(s["W"]).T)
            if case["bias"]:
                z += d(s["bias"])
        else:
            z = d(s["z"]) if act != "none" else None
        c = 0.7978845608028653559          # sqrt(2 / pi)
        if op == "linear":
            if act == "relu":
                y = z.clamp(min=0)
            elif act == "silu":
                y = z * torch.sigmoid(z)
            elif act == "gelu":
                y = z * torch.erfc(-z / 1.4142135623730950488) / 2
            elif act == "gelu_tanh":
                y = z * torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
            else:
                y = z
            if case["residual"]:
                y = y + d(s["residual"])
            return (y, z) if case["z"] else y
        if act == "relu":
            slope = torch.gt(z, 0).double()
        elif act == "silu":
            slope = torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
        elif act == "gelu":
            slope = torch.erfc(-z / 1.4142135623730950488) / 2 + z * c / 2 * torch.exp(-z * z / 2)
        elif act == "gelu_tanh":
            u = 2 * c * (z + 0.044715 * z ** 3)
            slope = torch.sigmoid(u) + z * torch.sigmoid(u) * torch.sigmoid(-u) * 2 * c * (1 + 0.134145 * z ** 2)
        dz = d(s["dy"]) if act == "none" else d(s["dy"]) * slope
        grads = [torch.matmul(dz, d(s["W"])), torch.matmul(dz.T, d(s["x"]))]
        if case["bias"]:
            grads.append(torch.sum(dz, dim=0))
        return grads
    r = s["route"]
    if op == "route_backward":
        # the Jacobian of the softmax: dl_e = sum_j dw_j w_j ([e = e_j] - q_e), q the
        # softmax over the picked experts (renormalised) or over all
        w, dw, ids = d(r["w"]), d(s["dw"]), r["ids"].long()
        hot = torch.zeros((case["T"], case["E"]), dtype=torch.float64, device=w.device)
        if case["renorm"]:
            q = hot.scatter(1, ids, w)
        else:
            q = torch.softmax(d(s["logits"]), dim=1)
        g = dw * w
        return hot.scatter(1, ids, g) - q * g.sum(dim=1, keepdim=True)
    T, k, H = case["T"], case["k"], case["H"]
    inv = r["inv_perm"].view(T, k).long()
    w = d(s["w"]) if case["weights"] else torch.ones((T, k), dtype=torch.float64, device=inv.device)
    if op in ("dispatch", "combine_backward"):
        src = d(s["x"] if op == "dispatch" else s["dy"])
        rows = torch.zeros((T * k, H), dtype=torch.float64, device=inv.device)
        dw = torch.zeros((T, k), dtype=torch.float64, device=inv.device)
        for j in range(k):
            live = inv[:, j] >= 0
            rows[inv[live, j]] = src[live] * w[live, j].unsqueeze(1)
            if op == "combine_backward":
                dw[live, j] = torch.einsum("th,th->t", src[live], d(s["ys"][inv[live, j]]))
        return rows if op == "dispatch" else (rows, dw)
    src = s["ys"] if op == "combine" else s["dxs"]
    y = torch.zeros((T, H), dtype=torch.float64, device=inv.device)
    dw = torch.zeros((T, k), dtype=torch.float64, device=inv.device)
    for j in range(k):
        live = inv[:, j] >= 0
        part = d(src[inv[live, j]])
        y[live] += part * w[live, j].unsqueeze(1)
        if op == "dispatch_backward" and case["weights"]:
            dw[live, j] = torch.einsum("th,th->t", part, d(s["x"][live]))
    if op == "combine":
        return y + d(s["residual"]) if case["residual"] else y
    return (y, dw) if case["weights"] else y


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("linear", "linear_backward"):
        M, N, K, s = case["M"], case["N"], case["K"], BYTES[case["dtype"]]
        if op == "linear":
            o = BYTES[case["out"]]
            b = (M * K + N * K) * s + M * N * o * (2 if case["residual"] else 1)
            b += N * s * case["bias"] + M * N * s * case["z"]
            return {"bytes": b, "flops": 2 * M * N * K}
        b = (M * K + N * K) * s * 2 + M * N * s * (2 if case["act"] != "none" else 1) + N * s * case["bias"]
        return {"bytes": b, "flops": 4 * M * N * K}
    T, k = case["T"], case["k"]
    if op == "route_backward":
        E = case["E"]
        b = T * E * BYTES[case["out"]] + T * k * 12 + (0 if case["renorm"] else T * E * 2)
        return {"bytes": b, "flops": T * k * 4 + (0 if case["renorm"] else T * E * 4)}
    H, s, o = case["H"], BYTES[case["dtype"]], BYTES[case["out"]]
    rows = int(T * k * (1.0 - case["drop"]))
    idx = T * k * (8 if case["weights"] else 4)
    if op == "dispatch":
        return {"bytes": T * H * s + rows * H * o + idx, "flops": rows * H * case["weights"]}
    if op == "combine":
        return {"bytes": rows * H * s + T * H * o * (2 if case["residual"] else 1) + idx, "flops": 2 * rows * H}
    if op == "dispatch_backward":
        b = rows * H * s + T * H * o + idx + ((T * H * s + T * k * 4) if case["weights"] else 0)
        return {"bytes": b, "flops": rows * H * (4 if case["weights"] else 1)}
    return {"bytes": T * H * s + rows * H * (s + o) + idx + T * k * 4, "flops": 3 * rows * H}
