"""Timed cases of the training operators that surround the optimizer step:
layer norm (forward, backward with the weight gradients), the orthogonalised
update (Newton-Schulz products) and the Muon step built on it.

Every case runs in two forms on the same inputs: `own = False` is the plain
one, elementary torch operations in 32 bits; `own = True` calls the library.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# the quintic Newton-Schulz iteration x <- a x + b x^3 + c x^5 on singular values
NS_STEPS = 5
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
NS_EPS = 1e-7


# --------------------------------------------------------------------- cases
def listed():
    ln_f = lambda name, rows, cols, dt, w, pad=0: dict(name=name, op="ln_forward", rows=rows, cols=cols, dtype=dt, w_dtype=w, pad=pad)  # noqa: E731
    ln_b = lambda name, rows, cols, dt, w, pad=0: dict(name=name, op="ln_backward", rows=rows, cols=cols, dtype=dt, w_dtype=w, pad=pad)  # noqa: E731
    orth = lambda name, rows, cols, batch, dt: dict(name=name, op="orthogonalize", rows=rows, cols=cols, batch=batch, dtype=dt)  # noqa: E731
    muon = lambda name, rows, cols, batch, n_d, dt: dict(name=name, op="muon_step", rows=rows, cols=cols, batch=batch, n_d=n_d, dtype=dt)  # noqa: E731
    return [
        # a handful of tokens through one norm of a GPT-2-small-sized layer: latency
        ln_f("ln_forward 8x768 bf16", 8, 768, "bf16", "fp32"),
        # one micro-batch of 8192 tokens of a 4096-wide layer
        ln_f("ln_forward 8192x4096 bf16", 8192, 4096, "bf16", "bf16"),
        # fp32 activations of an odd width cut from a wider buffer
        ln_f("ln_forward 2999x1601 fp32", 2999, 1601, "fp32", "fp32", pad=5),
        # a short sequence: few rows for the weight gradients to be split over
        ln_b("ln_backward 256x768 bf16", 256, 768, "bf16", "bf16"),
        # a micro-batch of 16384 tokens, gradients left in the ranks' type
        ln_b("ln_backward 16384x4096 bf16", 16384, 4096, "bf16", "bf16"),
        # an odd width in fp16 with fp32 weight gradients
        ln_b("ln_backward 5003x1601 fp16", 5003, 1601, "fp16", "fp32"),
        # one small projection: launches and latency
        orth("orthogonalize 96x160 bf16", 96, 160, 1, "bf16"),
        # the twelve 768-wide square projections of GPT-2 small, one call
        orth("orthogonalize 12x768x768 bf16", 768, 768, 12, "bf16"),
        # a feed-forward matrix of the 8-billion-parameter layer configuration
        orth("orthogonalize 4096x14336 bf16", 4096, 14336, 1, "bf16"),
        # an odd, tall matrix
        orth("orthogonalize 1601x333 fp16", 1601, 333, 1, "fp16"),
        # the fused attention projection of GPT-2 small over 8 ranks
        muon("muon_step 768x2304 nd8", 768, 2304, 1, 8, "bf16"),
        # two square projections of the 8-billion-parameter layer over 4 ranks
        muon("muon_step 2x4096x4096 nd4", 4096, 4096, 2, 4, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _ns_flops(rows, cols, batch):
    m, n = min(rows, cols), max(rows, cols)
    # per step: X X^T and A A are symmetric (half their entries), then B X
    return batch * NS_STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)


def draw(rng):
    op = rng.choice(["ln_forward", "ln_backward", "orthogonalize", "muon_step"])
    if op.startswith("ln"):
        cols = rng.choice([_log_int(rng, 33, 8192), 8 * _log_int(rng, 8, 1024)])
        rows = _log_int(rng, 1, min(16384, 16384 * 4096 // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), w_dtype=rng.choice(["fp32", "bf16"]),
                    pad=rng.choice([0, 0, 3, 8]))
    while True:
        rows, cols = ((8 * _log_int(rng, 3, 640), 8 * _log_int(rng, 3, 640)) if rng.random() < 0.6 else (_log_int(rng, 17, 4096), _log_int(rng, 17, 4096)))
        batch = _log_int(rng, 1, 24)
        if _ns_flops(rows, cols, batch) <= (_ns_flops(4096, 14336, 1) if op == "orthogonalize" else _ns_flops(4096, 4096, 2)) and batch * rows * cols <= 4096 * 14336:
            break
    if op == "orthogonalize":
        return dict(op=op, rows=rows, cols=cols, batch=batch, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    return dict(op=op, rows=rows, cols=cols, batch=batch, n_d=rng.choice([1, 2, 3, 4, 8, 16]), dtype=rng.choice(["bf16", "bf16", "fp16"]))


def work(case):
    r, c = case["rows"], case["cols"]
    b = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if case["op"].startswith("ln"):
        w = {"bf16": 2, "fp32": 4}[case["w_dtype"]]
        if case["op"] == "ln_forward":   # x in, y out; gain, bias; mean, 1/std
            return {"bytes": 2 * r * c * b + 2 * c * w + 8 * r, "flops": 8 * r * c}
        # dy, x in, dx out; gain; both weight gradients; mean, 1/std
        return {"bytes": 3 * r * c * b + 3 * c * w + 8 * r, "flops": 14 * r * c}
    n = case["batch"] * r * c
    if case["op"] == "orthogonalize":
        return {"bytes": 2 * n * b, "flops": _ns_flops(r, c, case["batch"])}
    # rank gradients; momentum and master in and out; 16-bit weights out
    return {"bytes": n * (case["n_d"] * b + 8 + 8 + 2), "flops": _ns_flops(r, c, case["batch"])}


# -------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _gradients(g, batch, rows, cols):
    """Gradients of linear layers: a few strong directions over a broad floor."""
    k = max(1, min(rows, cols) // 16)
    low = torch.matmul(_randn(g, batch, rows, k), _randn(g, batch, k, cols)) / math.sqrt(k)
    return 1e-3 * (low + _randn(g, batch, rows, cols))


def prepare(case, seed):
    g, dt = _gen(seed), DT[case["dtype"]]
    r, c = case["rows"], case["cols"]
    s = {"case": case}
    if case["op"].startswith("ln"):
        wdt = DT[case["w_dtype"]]
        wide = torch.zeros(r, c + case["pad"], device="cuda", dtype=dt)
        # activations with per-channel offsets and a few strong channels
        chan = _randn(g, c) * 0.5
        amp = torch.exp(0.3 * _randn(g, c))
        wide[:, :c] = (_randn(g, r, c) * amp + chan).to(dt)
        s["x"] = wide[:, :c]
        s["gain"] = (1.0 + 0.1 * _randn(g, c)).to(wdt)
        if case["op"] == "ln_forward":
            s["bias"] = (0.1 * _randn(g, c)).to(wdt)
            s["out"] = (torch.empty(r, c, device="cuda", dtype=dt), torch.empty(r, device="cuda"), torch.empty(r, device="cuda"))
        else:
            s["dy"] = (_randn(g, r, c) * 1e-2).to(dt)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + 1e-5)
            s["out"] = (torch.empty(r, c, device="cuda", dtype=dt), torch.empty(c, device="cuda", dtype=wdt), torch.empty(c, device="cuda", dtype=wdt))
    elif case["op"] == "orthogonalize":
        s["g"] = _gradients(g, case["batch"], r, c).to(dt)
        s["out"] = torch.empty_like(s["g"])
    else:
        base = _gradients(g, case["batch"], r, c)
        step = (r * c + 7) // 8 * 8   # each matrix starts on a multiple of 8 elements
        flat = lambda dtype: torch.zeros(case["batch"] * step, device="cuda", dtype=dtype)  # noqa: E731
        view = lambda t: t.view(case["batch"], step)[:, : r * c].view(case["batch"], r, c)  # noqa: E731
        s["view"], s["grads"] = view, []
        for _ in range(case["n_d"]):
            t = flat(dt)
            view(t).copy_((base + 1e-3 * _randn(g, case["batch"], r, c)).to(dt))
            s["grads"].append(t)
        s["momentum"], s["master"], s["weights"] = flat(torch.float32), flat(torch.float32), flat(dt)
        view(s["momentum"]).copy_(4.0 * _gradients(g, case["batch"], r, c))
        view(s["master"]).copy_(0.02 * _randn(g, case["batch"], r, c))
    if own:
        _plan(case, s)
    return s


def _plan(case, s):
    """What a program keeps beside its tensors: the descriptors and a workspace."""
    import zero_optimizer_step_02_gb300 as z

    zt = {"bf16": z.ZERO_BF16, "fp16": z.ZERO_FP16, "fp32": z.ZERO_FP32}
    r, c = case["rows"], case["cols"]
    s["z"] = z
    if case["op"].startswith("ln"):
        s["desc"] = z.layernorm(r, c, dtype=zt[case["dtype"]], w_dtype=zt[case["w_dtype"]], x_stride=c + case["pad"])
        size = z.zero_layernorm_workspace_bytes(s["desc"])
    elif case["op"] == "orthogonalize":
        s["desc"] = z.matrices(r, c, batch=case["batch"], dtype=zt[case["dtype"]])
        size = z.zero_orthogonalize_workspace_bytes(s["desc"])
    else:
        s["desc"] = z.matrices(r, c, batch=case["batch"], dtype=zt[case["dtype"]], stride=(r * c + 7) // 8 * 8)
        s["hp"] = z.muon_hparams(lr=MUON["lr"], momentum=MUON["momentum"], weight_decay=MUON["wd"], rms_scale=MUON["rms"])
        s["ranks"] = z.rank_ptrs(s["grads"])
        size = z.zero_muon_workspace_bytes(s["desc"])
    s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")


MUON = {"lr": 1e-3, "momentum": 0.95, "wd": 0.1, "rms": 0.2}


# ----------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    z, op = s["z"], s["case"]["op"]
    if op == "ln_forward":
        y, mean, rstd = s["out"]
        z.zero_layernorm_forward(s["desc"], s["x"], s["gain"], s["bias"], y, mean, rstd)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_backward":
        dx, dgain, dbias = s["out"]
        z.zero_layernorm_backward(s["desc"], s["dy"], s["x"], s["gain"], s["mean"], s["rstd"], dx, dgain, dbias, s["ws"])
        return {"dx": dx, "dgain": dgain, "dbias": dbias}
    if op == "orthogonalize":
        z.zero_orthogonalize(s["desc"], s["g"], s["out"], s["ws"])
        return {"o": s["out"]}
    z.zero_muon_step(s["desc"], s["hp"], s["ranks"], s["momentum"], s["master"], s["weights"], s["ws"])
    return _muon_out(s)


def _muon_out(s):
    return {k: s["view"](s[k]) for k in ("momentum", "master", "weights")}


def _plain_ns(x):
    """Newton-Schulz in 32 bits on [batch, rows, cols]; the short side first."""
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (torch.sqrt(torch.sum(x * x, (1, 2), keepdim=True)) + NS_EPS)
    for _ in range(NS_STEPS):
        a = torch.matmul(x, x.transpose(1, 2))
        b = NS_B * a + NS_C * torch.matmul(a, a)
        x = NS_A * x + torch.matmul(b, x)
    return x.transpose(1, 2) if tall else x


def _run_plain(s):
    op = s["case"]["op"]
    if op == "ln_forward":
        x = s["x"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).mean(1) + 1e-5)
        y = d * rstd[:, None] * s["gain"].float() + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "ln_backward":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["gain"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        wdt = s["gain"].dtype
        return {"dx": dx.to(s["x"].dtype), "dgain": (dy * xhat).sum(0).to(wdt), "dbias": dy.sum(0).to(wdt)}
    if op == "orthogonalize":
        return {"o": _plain_ns(s["g"].float()).to(s["g"].dtype).contiguous()}
    view, n_d = s["view"], s["case"]["n_d"]
    g = view(s["grads"][0]).float()
    for t in s["grads"][1:]:
        g = g + view(t).float()
    g = g / n_d
    buf = MUON["momentum"] * view(s["momentum"]) + g
    o = _plain_ns(g + MUON["momentum"] * buf)
    scale = MUON["lr"] * MUON["rms"] * math.sqrt(max(o.shape[1], o.shape[2]))
    w = view(s["master"]) * (1.0 - MUON["lr"] * MUON["wd"]) - scale * o
    view(s["momentum"]).copy_(buf)
    view(s["master"]).copy_(w)
    view(s["weights"]).copy_(w.to(s["weights"].dtype))
    return _muon_out(s)


# ------------------------------------------------------------ 64-bit results
def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] == "ln_forward":
        x = f64(s["x"])
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = (var + 1e-5) ** -0.5
        return {"y": torch.addcmul(f64(s["bias"]), (x - mean[:, None]) * rstd[:, None], f64(s["gain"])), "mean": mean, "rstd": rstd}
    if case["op"] == "ln_backward":
        # dx is the product of dy * gain with the Jacobian rstd (I - 1/c - xhat xhat^T / c)
        c = case["cols"]
        xhat = (f64(s["x"]) - f64(s["mean"])[:, None]) * f64(s["rstd"])[:, None]
        dy = f64(s["dy"])
        v = dy * f64(s["gain"])
        along = torch.einsum("rc,rc->r", v, xhat)[:, None] * xhat
        dx = (v - (v.sum(1, keepdim=True) + along) / c) * f64(s["rstd"])[:, None]
        return {"dx": dx, "dgain": torch.einsum("rc,rc->c", dy, xhat), "dbias": torch.einsum("rc->c", dy)}
    if case["op"] == "orthogonalize":
        return {"o": _exact_ns(f64(s["g"]))}
    mu, mats = MUON["momentum"], lambda k: f64(s["view"](s[k]))
    g = torch.zeros_like(mats("master"))
    for t in s["grads"]:
        g += f64(s["view"](t))
    g /= case["n_d"]
    buf = mu * mats("momentum") + g
    o = _exact_ns(g + mu * buf)
    w = mats("master") - MUON["lr"] * (MUON["wd"] * mats("master") + MUON["rms"] * max(case["rows"], case["cols"]) ** 0.5 * o)
    return {"momentum": buf, "master": w, "weights": w}


def _exact_ns(g):
    """One matrix at a time; q(S) = a + b S + c S^2 of the Gram matrix S on the
    short side, x <- q(S) x (or x q(S))."""
    out = torch.empty_like(g)
    for i in range(g.shape[0]):
        x = g[i] / (torch.linalg.norm(g[i]) + NS_EPS)
        eye = torch.eye(min(x.shape), dtype=x.dtype, device=x.device)
        for _ in range(NS_STEPS):
            if x.shape[0] <= x.shape[1]:
                gram = x @ x.mT
                x = (NS_A * eye + (NS_B * eye + NS_C * gram) @ gram) @ x
            else:
                gram = x.mT @ x
                x = x @ (NS_A * eye + gram @ (NS_B * eye + NS_C * gram))
        out[i] = x
    return out
