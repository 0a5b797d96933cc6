"""What is measured of the operators at the two ends of a Linear's training step, each in its plain form and through
the framework.

  norm      layer or RMS norm whose output is the next Linear's FP8 operand, in one tiling (inference) or both (training),
            with the statistics that its backward pass needs
  grad      the norm's backward pass: the input's gradient, with the residual's added, and the weight's and bias's
  update    the orthogonalised update of a weight from its gradient or momentum, by Newton-Schulz products

FP8 is OCP E4M3 in 1x128 tiles, scale = max-abs / 448, or the next power of two. Codes come back as float8 tensors,
next to their float32 scales.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = {"layer": 1e-5, "rms": 1e-6}
STEPS, COEFFICIENTS = 5, (3.4445, -4.7750, 2.0315)


# ---- cases -------------------------------------------------------------------------------------------

def listed():
    return [
        # one token on its way into a small projection: the latency of one call
        dict(name="norm_1_token", op="norm", rows=1, cols=1024, kind="rms", x="bf16", weight="bf16", beta=False,
             pow2=False, tokens=False, y=False),
        # a short prompt: rows that fill no tile, an fp32 residual stream, power-of-2 scales, the output in bf16 as well
        dict(name="norm_ragged_prompt", op="norm", rows=300, cols=2048, kind="layer", x="f32", weight="f32", beta=True,
             pow2=True, tokens=False, y=True),
        # the dense MLP's input in training: both tilings
        dict(name="norm_train", op="norm", rows=4096, cols=7168, kind="rms", x="bf16", weight="f32", beta=False,
             pow2=False, tokens=True, y=False),
        # a wide layer with an fp32 residual stream
        dict(name="norm_train_wide", op="norm", rows=4096, cols=18432, kind="layer", x="f32", weight="f32", beta=True,
             pow2=False, tokens=True, y=False),
        # one micro-batch of a small model
        dict(name="grad_small", op="grad", rows=256, cols=1024, kind="layer", x="bf16", weight="bf16", beta=True,
             dy="bf16", residual="bf16", dx="bf16"),
        # the dense MLP's input in training: FP32 gradients from Dgrad, the residual's in bf16
        dict(name="grad_train", op="grad", rows=4096, cols=7168, kind="rms", x="bf16", weight="f32", beta=False,
             dy="f32", residual="bf16", dx="bf16"),
        # many tokens of a small model, everything in fp32
        dict(name="grad_train_fp32", op="grad", rows=16384, cols=2048, kind="layer", x="f32", weight="f32", beta=True,
             dy="f32", residual="f32", dx="f32"),
        # a small model's weight: the latency of the products that follow each other
        dict(name="update_small", op="update", batch=1, n=256, k=1024, g="f32"),
        # sizes that fill no tile, more rows than columns
        dict(name="update_ragged", op="update", batch=1, n=2001, k=1000, g="bf16"),
        # the routed experts of one GPU
        dict(name="update_experts", op="update", batch=8, n=2048, k=7168, g="f32"),
        # the dense MLP's weight
        dict(name="update_dense", op="update", batch=1, n=18432, k=7168, g="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "grad", "grad", "update"])
    while True:
        if op == "update":
            c = dict(op=op, batch=rng.choice([1, 1, 1, 2, 8]), n=_log(rng, 64, 18432), k=_log(rng, 64, 18432),
                     g=rng.choice(["f32", "bf16"]))
            if c["batch"] * c["n"] * c["k"] * min(c["n"], c["k"]) > 18432 * 7168 * 7168:
                continue
            return c
        kind = rng.choice(["layer", "rms"])
        c = dict(op=op, rows=_log(rng, 1, 16384), cols=128 * _log(rng, 1, 144), kind=kind, x=rng.choice(["f32", "bf16"]),
                 weight=rng.choice(["f32", "bf16"]), beta=kind == "layer" and rng.random() < 0.75)
        if op == "norm":
            tokens = rng.random() < 0.5
            if tokens:
                c["rows"] = 128 * -(-c["rows"] // 128)
            # fp32 sums in any order leave one max-abs in some millions on either side of a power of two, which is a
            # factor of two in its scale: power-of-2 scales are drawn where there are few tiles
            c |= dict(pow2=rng.random() < 0.5 and c["rows"] * c["cols"] <= 1 << 22, tokens=tokens, y=rng.random() < 0.25)
        else:
            residual = rng.choice(["", "f32", "bf16"])
            c |= dict(dy=rng.choice(["f32", "bf16"]), residual=residual, dx=residual or rng.choice(["f32", "bf16"]))
        if c["rows"] * c["cols"] > 4096 * 18432:
            continue
        return c


SIZE = {"": 0, "f32": 4, "bf16": 2}


def work(case):
    c = case
    if c["op"] == "update":
        m, n = sorted((c["n"], c["k"]))
        # X X^T and A A are symmetric: half of each is enough
        flops = STEPS * (m * m * n + m ** 3 + 2 * m * m * n)
        return dict(bytes=c["batch"] * m * n * (SIZE[c["g"]] + 2), flops=c["batch"] * flops)
    e, stats = c["rows"] * c["cols"], c["rows"] * (8 if c["kind"] == "layer" else 4)
    if c["op"] == "norm":
        b = e * (SIZE[c["x"]] + (1 + 4 / 128) * (2 if c["tokens"] else 1) + (2 if c["y"] else 0))
        return dict(bytes=b + stats + c["cols"] * SIZE[c["weight"]] * (2 if c["beta"] else 1), flops=e * 12)
    b = e * (SIZE[c["x"]] + SIZE[c["dy"]] + SIZE[c["residual"]] + SIZE[c["dx"]])
    return dict(bytes=b + stats + c["cols"] * (SIZE[c["weight"]] + 4 * (2 if c["beta"] else 1)), flops=e * 16)


# ---- inputs ------------------------------------------------------------------------------------------

def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    s = dict(case=c)
    if c["op"] == "update":
        # the gradient of a Linear over more tokens than its smaller side, with outlier channels, as momentum is
        b, n, k = c["batch"], c["n"], c["k"]
        t = 2 * min(n, k) + 64
        grads = torch.empty(b, n, k, device="cuda")
        for i in range(b):
            x = normal(t, k)
            x[:, torch.randperm(k, generator=g, device="cuda")[:max(1, k // 100)]] *= 5
            torch.matmul((normal(t, n, std=1e-3)).t(), x, out=grads[i])
        s["g"] = (grads if b > 1 else grads[0]).to(TYPES[c["g"]])
        return s
    r, w = c["rows"], c["cols"]
    x = normal(r, w) * torch.exp(normal(r, 1, std=0.5)) + 0.2               # tokens of different sizes, off centre
    x[:, torch.randperm(w, generator=g, device="cuda")[:max(1, w // 100)]] *= 20
    s["x"] = x.to(TYPES[c["x"]])
    s["gamma"] = (1 + normal(w, std=0.2)).to(TYPES[c["weight"]])
    s["beta"] = normal(w, std=0.1).to(TYPES[c["weight"]]) if c["beta"] else None
    if c["op"] == "grad":
        v = s["x"].double()
        mean = v.mean(1) if c["kind"] == "layer" else torch.zeros_like(v[:, 0])
        s["rstd"] = ((v - mean[:, None]).square().mean(1) + EPS[c["kind"]]).rsqrt().float()
        s["mean"] = mean.float() if c["kind"] == "layer" else None
        s["dy"] = normal(r, w, std=1e-3).to(TYPES[c["dy"]])
        s["residual"] = normal(r, w, std=1e-3).to(TYPES[c["residual"]]) if c["residual"] else None
    return s


# ---- one pass ----------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import fp8_fine_grained_amax_amd as fg

    c = s["case"]
    if c["op"] == "update":
        return dict(out=fg.fg_orthogonalize(s["g"], steps=STEPS, coefficients=COEFFICIENTS,
                                            scale=max(1.0, c["n"] / c["k"]) ** 0.5))
    kind = fg.FG_NORM_LAYER if c["kind"] == "layer" else fg.FG_NORM_RMS
    if c["op"] == "norm":
        r = fg.fg_norm_quantize(s["x"], s["gamma"], s["beta"], kind=kind, eps=EPS[c["kind"]], pow2=c["pow2"],
                                token_tiles=c["tokens"], with_y=c["y"])
        out = dict(q=r.q_cols.view(F8), s=r.s_cols, rstd=r.rstd)
        if c["kind"] == "layer":
            out["mean"] = r.mean
        if c["tokens"]:
            out |= dict(q_t=r.q_rows.view(F8), s_t=r.s_rows)
        return out | dict(y=r.y) if c["y"] else out
    r = fg.fg_norm_bwd(s["x"], s["mean"], s["rstd"], s["gamma"], s["dy"], residual_grad=s["residual"], kind=kind,
                       out_dtype=TYPES[c["dx"]], bias_grad=c["beta"])
    out = dict(dx=r.dx, dgamma=r.dgamma)
    return out | dict(dbeta=r.dbeta) if c["beta"] else out


def _scale(amax, pow2):
    # divided by a tensor: by a number, torch multiplies with its reciprocal, and the scale is often one bit off
    s = (amax / torch.full_like(amax, 448)).clamp(min=torch.finfo(torch.float32).tiny)
    if pow2:
        m, e = torch.frexp(s)
        s = torch.where(m == 0.5, s, torch.ldexp(torch.ones_like(s), e))
    return torch.where(amax == 0, torch.ones_like(s), s)


def _tiles(v, pow2):
    """1x128 tiles along the last axis: float8 codes like v, scales [last / 128, rows]."""
    t = v.unflatten(-1, (-1, 128))
    s = _scale(t.abs().amax(-1), pow2)
    return (t / s[..., None]).to(F8).flatten(-2), s.t().contiguous()


def _plain(s):
    c = s["case"]
    if c["op"] == "update":
        a, b, cc = COEFFICIENTS
        x = s["g"].float()
        tall = c["n"] > c["k"]
        if tall:
            x = x.mT
        x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + 1e-7)
        for _ in range(STEPS):
            p = torch.matmul(x, x.mT)
            x = a * x + torch.matmul(b * p + cc * torch.matmul(p, p), x)
        return dict(out=(max(1.0, c["n"] / c["k"]) ** 0.5 * (x.mT if tall else x)).to(torch.bfloat16).contiguous())
    x, gamma = s["x"].float(), s["gamma"].float()
    layer = c["kind"] == "layer"
    if c["op"] == "norm":
        mean = x.mean(1) if layer else None
        d = x - mean[:, None] if layer else x
        rstd = 1 / torch.sqrt(d.square().mean(1) + EPS[c["kind"]])
        y = d * rstd[:, None] * gamma
        if c["beta"]:
            y = y + s["beta"].float()
        q, sc = _tiles(y, c["pow2"])
        out = dict(q=q, s=sc, rstd=rstd)
        if layer:
            out["mean"] = mean
        if c["tokens"]:
            out["q_t"], out["s_t"] = _tiles(y.t().contiguous(), c["pow2"])
        return out | dict(y=y.to(torch.bfloat16)) if c["y"] else out
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None] if layer else x) * rstd
    g = dy * gamma
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if layer:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    out = dict(dx=dx.to(TYPES[c["dx"]]), dgamma=(dy * xh).sum(0))
    return out | dict(dbeta=dy.sum(0)) if c["beta"] else out


# ---- the definition in 64 bits -----------------------------------------------------------------------

def _grid(v):
    """float64 -> the nearest E4M3 value (ties to even, saturated at 448), as float64."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_tiles(v, pow2):
    r, n = v.shape
    t = v.reshape(r, n // 128, 128)
    amax = t.abs().max(2).values
    # the scale and the quotient by it are held in 32 bits by definition: products of bf16 values often lie on a border
    # between two codes exactly
    s = (amax / 448).to(torch.float32).to(torch.float64).clamp(min=2.0 ** -126)
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    s = torch.where(amax == 0, torch.ones_like(s), s)
    return _grid((t / s[:, :, None]).to(torch.float32).to(torch.float64)).reshape(r, n), s.t()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "update":
        g = s["g"].double().reshape(c["batch"], c["n"], c["k"])
        out = []
        for m in g:
            wide = m if c["n"] <= c["k"] else m.t().contiguous()
            x = wide / (torch.linalg.matrix_norm(wide) + 1e-7)
            for _ in range(STEPS):
                p = x @ x.t()
                p = COEFFICIENTS[1] * p + COEFFICIENTS[2] * (p @ p)
                p.diagonal().add_(COEFFICIENTS[0])
                x = p @ x
            out.append((x if c["n"] <= c["k"] else x.t()) * math.sqrt(max(1.0, c["n"] / c["k"])))
        return dict(out=torch.stack(out) if c["batch"] > 1 else out[0].contiguous())
    x, gamma = s["x"].double(), s["gamma"].double()
    if c["op"] == "norm":
        var, mean = torch.var_mean(x, 1, correction=0)
        if c["kind"] == "rms":
            var, mean = var + mean.square(), torch.zeros_like(mean)
        rstd = (var + EPS[c["kind"]]) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * gamma
        if c["beta"]:
            y += s["beta"].double()
        out = dict(rstd=rstd)
        out["q"], out["s"] = _exact_tiles(y, c["pow2"])
        if c["kind"] == "layer":
            out["mean"] = mean
        if c["tokens"]:
            out["q_t"], out["s_t"] = _exact_tiles(y.t(), c["pow2"])
        return out | dict(y=y) if c["y"] else out
    dy, rstd = s["dy"].double(), s["rstd"].double()
    xh = x * rstd[:, None] if s["mean"] is None else torch.addcmul(-(s["mean"].double() * rstd)[:, None], x, rstd[:, None])
    # the Jacobian of the norm's row, applied: rstd (I - [1 1^T] / n - xh xh^T / n) diag(gamma)
    t = dy * gamma
    dot = (t * xh).sum(1) / c["cols"]
    dx = torch.addcmul(t, xh, dot[:, None], value=-1)
    if c["kind"] == "layer":
        dx -= (t.sum(1) / c["cols"])[:, None]
    dx *= rstd[:, None]
    if c["residual"]:
        dx += s["residual"].double()
    out = dict(dx=dx, dgamma=(dy * xh).sum(0))
    return out | dict(dbeta=dy.sum(0)) if c["beta"] else out
