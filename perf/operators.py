"""What is measured of the FP8 feed-forward operators, each in its plain form and through the framework.

  linear   a Linear's product from FP8 codes with bias, activation and residual in its epilogue
  forward  an activation function that leaves its input as an FP8 checkpoint and its output as FP8 tiles
  backward the same function's gradient from the FP8 checkpoint, quantized in both tilings for the Dgrad and
           Wgrad that follow, with the recomputed output and the bias gradient
  experts  a whole mixture-of-experts feed-forward for a few tokens

FP8 is OCP E4M3 in 1x128 tiles (activations) and 128x128 blocks (weights), scale = max-abs / 448, or the next
power of two. Codes come back as float8 tensors, next to their float32 scales.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases -------------------------------------------------------------------------------------------

def listed():
    return [
        # one token through a small projection: the latency of one call
        dict(name="linear_1_token_small", op="linear", rows=1, out=1024, inner=1024, bias="bf16", act="silu",
             residual="", pow2=False),
        # a decoding batch through the dense MLP's down-projection: the weight is read once, and the residual
        # stream is added
        dict(name="linear_16_tokens_down", op="linear", rows=16, out=7168, inner=18432, bias="", act="none",
             residual="bf16", pow2=False),
        # a short prompt, sizes that fill no tile
        dict(name="linear_ragged_prompt", op="linear", rows=300, out=2001, inner=2048, bias="f32", act="relu",
             residual="f32", pow2=False),
        # the dense MLP's training step
        dict(name="linear_train", op="linear", rows=4096, out=18432, inner=7168, bias="f32", act="gelu",
             residual="", pow2=True),
        # the activation of a handful of tokens
        dict(name="forward_7_tokens", op="forward", rows=7, width=2048, gated=True, act="silu"),
        # the gated activation of the dense MLP in training
        dict(name="forward_train_gated", op="forward", rows=4096, width=18432, gated=True, act="silu"),
        # one micro-batch of a small model
        dict(name="backward_small", op="backward", rows=256, width=1024, gated=False, act="gelu", grad="bf16",
             bias=True, tokens=True),
        # the dense MLP's backward step: FP32 gradients from Dgrad
        dict(name="backward_train_gated", op="backward", rows=4096, width=18432, gated=True, act="silu", grad="f32",
             bias=False, tokens=True),
        # an MLP with biases in training: bf16 gradients, the bias gradient in the same pass
        dict(name="backward_train_bias", op="backward", rows=8192, width=7168, gated=False, act="gelu", grad="bf16",
             bias=True, tokens=True),
        # one token through a small mixture: the latency of one call
        dict(name="experts_1_token_small", op="experts", rows=1, experts=8, total=8, top=2, hidden=1024, inner=512,
             act="silu", pow2=False),
        # one token through eight large experts: every weight of theirs is read once
        dict(name="experts_1_token_large", op="experts", rows=1, experts=8, total=8, top=8, hidden=7168, inner=2048,
             act="silu", pow2=False),
        # a decoding batch on one GPU's share of an expert-parallel layer: most choices live on other GPUs
        dict(name="experts_64_tokens_share", op="experts", rows=64, experts=16, total=64, top=8, hidden=7168,
             inner=2048, act="silu", pow2=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "forward", "backward", "experts"])
    act = rng.choice(["relu", "gelu", "silu"])
    while True:
        if op == "linear":
            c = dict(op=op, rows=_log(rng, 1, 4096), out=_log(rng, 64, 18432), inner=128 * _log(rng, 1, 144),
                     bias=rng.choice(["", "f32", "bf16"]), act=rng.choice(["none", act]),
                     residual=rng.choice(["", "f32", "bf16"]), pow2=rng.random() < 0.5)
            if c["rows"] * c["out"] * c["inner"] > 4096 * 18432 * 7168:
                continue
        elif op == "forward":
            c = dict(op=op, rows=_log(rng, 1, 8192), width=128 * _log(rng, 1, 144), gated=rng.random() < 0.5, act=act)
            if c["rows"] * c["width"] > 4096 * 18432:
                continue
        elif op == "backward":
            tokens = rng.random() < 0.75
            c = dict(op=op, rows=128 * _log(rng, 1, 64) if tokens else _log(rng, 1, 8192), width=128 * _log(rng, 1, 144),
                     gated=rng.random() < 0.5, act=act, grad=rng.choice(["f32", "bf16"]), bias=rng.random() < 0.5,
                     tokens=tokens)
            if c["rows"] * c["width"] > 4096 * 18432:
                continue
        else:
            experts = _log(rng, 1, 64)
            total = experts * rng.choice([1, 1, 2, 4])
            c = dict(op=op, rows=_log(rng, 1, 64), experts=experts, total=total, top=rng.randint(1, min(8, total)),
                     hidden=128 * _log(rng, 2, 56), inner=128 * _log(rng, 1, 16), act=act, pow2=rng.random() < 0.5)
            if c["experts"] * c["hidden"] * c["inner"] > 16 * 7168 * 2048:
                continue
        return c


def work(case):
    c = case
    if c["op"] == "linear":
        m, n, k = c["rows"], c["out"], c["inner"]
        size = {"": 0, "f32": 4, "bf16": 2}
        b = m * k + n * k + 4 * (m * k // 128 + -(-n // 128) * (k // 128)) + 2 * m * n
        return dict(bytes=b + size[c["bias"]] * n + size[c["residual"]] * m * n, flops=2 * m * n * k)
    if c["op"] == "forward":
        e, w = c["rows"] * c["width"], 2 if c["gated"] else 1
        return dict(bytes=e * (2 * w + w + 1) + e // 128 * 4 * (w + 1), flops=e * 16)
    if c["op"] == "backward":
        e, w = c["rows"] * c["width"], 2 if c["gated"] else 1
        b = e * (w + (4 if c["grad"] == "f32" else 2) + w) + e // 128 * 4 * 2 * w
        if c["tokens"]:
            b += (e + e // 128 * 4) * (w + 1)
        if c["bias"]:
            b += 4 * w * c["width"]
        return dict(bytes=b, flops=e * 32)
    # the expected number of local experts that some token chose, and of local choices
    t, e, p = c["rows"], c["experts"], c["top"] / c["total"]
    used = e * (1 - (1 - p) ** t)
    b = used * 3 * c["hidden"] * c["inner"] * (1 + 4 / 16384) + t * c["hidden"] * 4 + t * c["top"] * 8
    return dict(bytes=b, flops=t * e * p * 6 * c["hidden"] * c["inner"])


# ---- inputs ------------------------------------------------------------------------------------------

def _scale(amax, pow2):
    # divided by a tensor: by a number, torch multiplies with its reciprocal, and the scale is often one bit off
    s = (amax / torch.full_like(amax, 448)).clamp(min=torch.finfo(torch.float32).tiny)
    if pow2:
        m, e = torch.frexp(s)
        s = torch.where(m == 0.5, s, torch.ldexp(torch.ones_like(s), e))
    return torch.where(amax == 0, torch.ones_like(s), s)


def _tiles(v, pow2=False):
    """1x128 tiles along the last axis: float8 codes like v, scales [..., last / 128]."""
    t = v.unflatten(-1, (-1, 128))
    s = _scale(t.abs().amax(-1), pow2)
    return (t / s[..., None]).to(F8).flatten(-2), s


def _blocks(w, pow2=False):
    """128x128 blocks of the last two axes: float8 codes like w, scales [..., ceil(n / 128), k / 128]."""
    n, k = w.shape[-2:]
    v = torch.nn.functional.pad(w, (0, 0, 0, -n % 128)).unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    s = _scale(v.abs().amax((-3, -1)), pow2)
    q = (v / s[..., :, None, :, None]).to(F8)
    return q.flatten(-2).flatten(-3, -2)[..., :n, :].contiguous(), s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=c)
    if c["op"] == "linear":
        m, n, k = c["rows"], c["out"], c["inner"]
        x = normal(m, k)
        x[:, torch.randperm(k, generator=g, device="cuda")[:max(1, k // 100)]] *= 20   # outlier channels
        q, sx = _tiles(x.float(), c["pow2"])
        s["xq"], s["sx"] = q.view(torch.uint8), sx.t().contiguous()
        q, s["sw"] = _blocks(normal(n, k, std=0.5 * k ** -0.5).float(), c["pow2"])
        s["wq"] = q.view(torch.uint8)
        s["bias"] = normal(n, std=0.1, dtype=TYPES[c["bias"]]) if c["bias"] else None
        s["residual"] = normal(m, n, dtype=TYPES[c["residual"]]) if c["residual"] else None
    elif c["op"] == "forward":
        s["z"] = normal(c["rows"], c["width"] * (2 if c["gated"] else 1), std=2.0)
    elif c["op"] == "backward":
        q, sz = _tiles(normal(c["rows"], c["width"] * (2 if c["gated"] else 1), std=2.0).float())
        s["zq"], s["sz"] = q.view(torch.uint8), sz.t().contiguous()
        s["da"] = normal(c["rows"], c["width"], std=1e-3, dtype=TYPES[c["grad"]])
    else:
        t, e, h, i = c["rows"], c["experts"], c["hidden"], c["inner"]
        s["x"] = normal(t, h)
        q, s["s1"] = _blocks(normal(e, 2 * i, h, std=h ** -0.5).float())
        s["w1"] = q.view(torch.uint8)
        q, s["s2"] = _blocks(normal(e, h, i, std=i ** -0.5).float())
        s["w2"] = q.view(torch.uint8)
        score, ids = torch.randn(t, c["total"], generator=g, device="cuda").topk(c["top"], dim=1)
        s["weights"] = score.softmax(1)
        s["ids"] = torch.where(ids < e, ids, -1).to(torch.int32)        # -1: the expert lives on another GPU
    return s


# ---- one pass ----------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import fp8_fine_grained_amax_amd as fg

    c = s["case"]
    act = {"none": fg.FG_ACT_NONE, "relu": fg.FG_ACT_RELU, "gelu": fg.FG_ACT_GELU_TANH, "silu": fg.FG_ACT_SILU}[c["act"]]
    if c["op"] == "linear":
        return dict(y=fg.fg_fp8_gemm_fprop_epilogue(s["xq"], s["sx"], s["wq"], s["sw"], bias=s["bias"], act=act,
                                                    residual=s["residual"], pow2=c["pow2"]))
    if c["op"] == "forward":
        zq, sz, aq, sa = fg.fg_act_checkpoint_fwd(s["z"], act, gated=c["gated"])
        return dict(zq=zq.view(F8), sz=sz, aq=aq.view(F8), sa=sa)
    if c["op"] == "backward":
        r = fg.fg_act_checkpoint_bwd(s["zq"], s["sz"], s["da"], act, gated=c["gated"], token_tiles=c["tokens"],
                                     recompute=c["tokens"], bias_grad=c["bias"])
        out = dict(dzq=r.dzq_cols.view(F8), sdz=r.sdz_cols)
        if c["tokens"]:
            out |= dict(dzq_t=r.dzq_rows.view(F8), sdz_t=r.sdz_rows, aq_t=r.aq_rows.view(F8), sa_t=r.sa_rows)
        return out | dict(db=r.dbias) if c["bias"] else out
    return dict(y=fg.fg_moe_few_tokens(s["x"], s["ids"], s["weights"], s["w1"], s["s1"], s["w2"], s["s2"], act=act,
                                       pow2=c["pow2"]))


def _act(z, kind):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * torch.sigmoid(1.5957691216057308 * (z + 0.044715 * z * z * z))   # 2 sqrt(2 / pi)
    return z


def _slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    k = torch.sigmoid(z if kind == "silu" else 1.5957691216057308 * (z + 0.044715 * z * z * z))
    return k + z * k * (1 - k) * (1 if kind == "silu" else 1.5957691216057308 * (1 + 0.134145 * z * z))


def _decode(q, s):
    """codes [..., cols] in 1x128 tiles with scales [..., cols / 128] -> float32."""
    return (q.view(F8).float().unflatten(-1, (-1, 128)) * s[..., None]).flatten(-2)


def _decode_blocks(q, s):
    rows = s.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    return _decode(q, rows)


def _tiles_t(v):
    """1x128 tiles along the rows of v: transposed codes [cols, rows], scales [rows / 128, cols]."""
    q, s = _tiles(v.t().contiguous())
    return q, s.t().contiguous()


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        z = _decode(s["xq"], s["sx"].t()) @ _decode_blocks(s["wq"], s["sw"]).t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return dict(y=y.to(torch.bfloat16))
    if c["op"] == "forward":
        z = s["z"].float()
        zq, sz = _tiles(z)
        w = c["width"]
        aq, sa = _tiles(_act(z[:, :w], c["act"]) * z[:, w:] if c["gated"] else _act(z, c["act"]))
        return dict(zq=zq, sz=sz.t().contiguous(), aq=aq, sa=sa.t().contiguous())
    if c["op"] == "backward":
        z, da, w = _decode(s["zq"], s["sz"].t()), s["da"].float(), c["width"]
        if c["gated"]:
            gate, up = z[:, :w], z[:, w:]
            a = _act(gate, c["act"])
            dz, a = torch.cat([da * up * _slope(gate, c["act"]), da * a], 1), a * up
        else:
            dz, a = da * _slope(z, c["act"]), _act(z, c["act"])
        q, sc = _tiles(dz)
        out = dict(dzq=q, sdz=sc.t().contiguous())
        if c["tokens"]:
            out["dzq_t"], out["sdz_t"] = _tiles_t(dz)
            out["aq_t"], out["sa_t"] = _tiles_t(a)
        if c["bias"]:
            out["db"] = dz.sum(0)
        return out
    t, e, h, i = c["rows"], c["experts"], c["hidden"], c["inner"]
    x = _decode(*_tiles(s["x"].float(), c["pow2"]))
    here = s["ids"] >= 0
    pick = s["ids"].clamp(min=0).long()
    if t * c["top"] <= e:                    # only the chosen experts' weights
        pick = pick.flatten()
        x = x.repeat_interleave(c["top"], 0)[:, :, None]
        gu = torch.bmm(_decode_blocks(s["w1"][pick], s["s1"][pick]), x)[:, :, 0]
        a = _decode(*_tiles(_act(gu[:, :i], c["act"]) * gu[:, i:], c["pow2"]))
        y = torch.bmm(_decode_blocks(s["w2"][pick], s["s2"][pick]), a[:, :, None]).view(t, c["top"], h)
        y = torch.where(here[:, :, None], s["weights"][:, :, None] * y, 0).sum(1)
    else:                                    # every expert for every token, weighted
        gu = (x @ _decode_blocks(s["w1"], s["s1"]).view(e * 2 * i, h).t()).view(t, e, 2 * i)
        a = _decode(*_tiles(_act(gu[..., :i], c["act"]) * gu[..., i:], c["pow2"]))
        share = torch.zeros(t, e, device=x.device).scatter_add_(1, pick, torch.where(here, s["weights"], 0))
        y = (share[:, :, None] * a).view(t, e * i) @ _decode_blocks(s["w2"], s["s2"]).transpose(1, 2).reshape(e * i, h)
    return dict(y=y.to(torch.bfloat16))


# ---- the definition in 64 bits -----------------------------------------------------------------------

def _grid(v):
    """float64 -> the nearest E4M3 value (ties to even, saturated at 448), as float64."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_tiles(v, pow2=False):
    r, n = v.shape
    t = v.reshape(r, n // 128, 128)
    s = t.abs().max(2).values / 448
    # the scale and the quotient by it are held in 32 bits by definition: bf16 values often lie on a border
    # between two codes exactly
    s = s.to(torch.float32).to(torch.float64).clamp(min=2.0 ** -126)
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    s = torch.where(t.abs().max(2).values == 0, torch.ones_like(s), s)
    return _grid((t / s[:, :, None]).to(torch.float32).to(torch.float64)).reshape(r, n), s


def _exact_act(z, kind):
    """(value, derivative)"""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return torch.relu(z), torch.heaviside(z, torch.zeros_like(z))
    if kind == "silu":
        k = 1 / (1 + torch.exp(-z))
        return z * k, k * (1 + z * (1 - k))
    a = math.sqrt(2 / math.pi)
    th = torch.tanh(a * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + th), 0.5 * (1 + th) + 0.5 * z * (1 - th ** 2) * a * (1 + 3 * 0.044715 * z ** 2)


def _wide(q, s):
    """codes [r, c] and per-tile scales [r, c / 128] -> float64 values"""
    return q.view(F8).double() * s.double().repeat_interleave(128, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        y = _wide(s["xq"], s["sx"].t()) @ _wide(s["wq"], s["sw"].repeat_interleave(128, 0)[:c["out"]]).t()
        if c["bias"]:
            y += s["bias"].double()
        y = _exact_act(y, c["act"])[0]
        return dict(y=y + s["residual"].double() if c["residual"] else y)
    if c["op"] == "forward":
        z = s["z"].double()
        out = {}
        out["zq"], sz = _exact_tiles(z)
        if c["gated"]:
            gate, up = z.chunk(2, 1)
            a = _exact_act(gate, c["act"])[0] * up
        else:
            a = _exact_act(z, c["act"])[0]
        out["aq"], sa = _exact_tiles(a)
        return out | dict(sz=sz.t(), sa=sa.t())
    if c["op"] == "backward":
        z, da = _wide(s["zq"], s["sz"].t()), s["da"].double()
        if c["gated"]:
            gate, up = z.chunk(2, 1)
            a, slope = _exact_act(gate, c["act"])
            dz, a = torch.hstack([da * up * slope, da * a]), a * up
        else:
            a, slope = _exact_act(z, c["act"])
            dz = da * slope
        out = {}
        out["dzq"], sdz = _exact_tiles(dz)
        out["sdz"] = sdz.t()
        if c["tokens"]:
            out["dzq_t"], sdz = _exact_tiles(dz.t())
            out["aq_t"], sa = _exact_tiles(a.t())
            out |= dict(sdz_t=sdz.t(), sa_t=sa.t())
        if c["bias"]:
            out["db"] = dz.sum(0)
        return out
    i = c["inner"]
    q, sx = _exact_tiles(s["x"].double(), c["pow2"])
    x = q * sx.repeat_interleave(128, 1)
    y = torch.zeros_like(x)
    for e in range(c["experts"]):
        share = torch.where(s["ids"] == e, s["weights"].double(), 0).sum(1)
        rows = (s["ids"] == e).any(1).nonzero()[:, 0]
        gu = x[rows] @ _wide(s["w1"][e], s["s1"][e].repeat_interleave(128, 0)).t()
        q, sa = _exact_tiles(_exact_act(gu[:, :i], c["act"])[0] * gu[:, i:], c["pow2"])
        a = q * sa.repeat_interleave(128, 1)
        y[rows] += share[rows, None] * (a @ _wide(s["w2"][e], s["s2"][e].repeat_interleave(128, 0)).t())
    return dict(y=y)
