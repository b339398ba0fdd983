"""The operators that surround the EQ-Linear layer in a transformer MLP block, as they are measured.

Layer norm over a row of C'*T features with one weight and bias per channel (shared by the
channel's T group elements), and 8-bit activation checkpoints with the passes that read them.
A case's "op" is one of

  norm         the norm's forward pass
  norm_step    forward and backward of the norm in a pre-norm block (the residual branch's
               gradient is added to the input's); keep = "x" keeps the input for the backward
               pass, keep = "8bit" the normalised row as an 8-bit checkpoint
  round_trip   a matrix into an 8-bit checkpoint and back
  gelu_grad    backward of the bias + GELU epilogue, GELU's input read from a checkpoint
  weight_grad  the EQ-Linear weight gradient, the layer's input read from a checkpoint of the
               norm's output (view = "affine"), of GELU's input ("gelu") or of itself ("none")

A checkpoint of an [N, R] matrix holds N rows of ceil(R / 32) * 32 signed bytes (zeros past R),
then N rows of ceil(R / 32) scale bytes s: 32 consecutive features share the step 2^(s - 127).
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 32


def _case(name, op, dtype, n, c, t, d=0, keep="", view=""):
    return {"name": name, "op": op, "dtype": dtype, "N": n, "C": c, "T": t, "D": d, "keep": keep, "view": view}


def listed():
    return [
        # One image's tokens (197) at the width of a small ViT: what a single request costs.
        _case("norm one image f16", "norm", "f16", 197, 96, 4),
        # A training batch at the width of the largest benchmarked layer, in inference form.
        _case("norm square f16", "norm", "f16", 65536, 1024, 4),
        # Full-precision training with eight rotations.
        _case("norm step C8 f32", "norm_step", "f32", 16384, 64, 8, keep="x"),
        # A small ViT's training batch (64 images).
        _case("norm step vit 8bit f16", "norm_step", "f16", 12608, 96, 4, keep="8bit"),
        # The widest block's training batch.
        _case("norm step square 8bit f16", "norm_step", "f16", 65536, 1024, 4, keep="8bit"),
        # Rows that end inside a block of 32 and that no vector load divides.
        _case("round trip odd f32", "round_trip", "f32", 3001, 133, 5),
        # The hidden activation of a small ViT's MLP.
        _case("round trip vit hidden f16", "round_trip", "f16", 12608, 384, 4),
        # The hidden gradient of a ragged three-fold layer: rows of 513 features.
        _case("gelu grad ragged f16", "gelu_grad", "f16", 5003, 171, 3),
        # The hidden gradient of the widest block.
        _case("gelu grad square f16", "gelu_grad", "f16", 65536, 1024, 4),
        # First layer of a small ViT's MLP: its input is the norm's output.
        _case("weight grad vit f16", "weight_grad", "f16", 12608, 96, 4, d=384, view="affine"),
        # Second layer of a full-precision block: its input is GELU of what was kept.
        _case("weight grad C8 f32", "weight_grad", "f32", 16384, 64, 8, d=64, view="gelu"),
        # The widest block's second layer.
        _case("weight grad square f16", "weight_grad", "f16", 65536, 1024, 4, d=1024, view="gelu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_step", "round_trip", "gelu_grad", "weight_grad"])
    dtype = rng.choice(["f16", "f32"])
    t = rng.choice([1, 2, 3, 4, 4, 5, 6, 8, 12])
    row = _log_int(rng, 24, 6000)
    c = max(1, row // t)
    n = max(1, min(_log_int(rng, 1, 60000), (1 << 26) // (c * t)))
    keep = rng.choice(["x", "8bit"]) if op == "norm_step" else ""
    if keep == "8bit":
        dtype = "f16"  # the full-precision step keeps x: its outputs are not held to 8 bits
    d, view = 0, ""
    if op == "weight_grad":
        view = rng.choice(["none", "affine", "gelu"])
        d = max(1, _log_int(rng, 16, 4096) // t)
        n = max(1, min(n, (1 << 36) // (c * t * d * t)))
    case = _case("", op, dtype, n, c, t, d, keep, view)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _dtype(case):
    return torch.float16 if case["dtype"] == "f16" else torch.float32


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32)


def _activations(gen, n, r):
    """Rows of a residual stream: features of different scale, an offset per row, and one row
    in a hundred sixteen times as large."""
    v = _randn(gen, n, r) * torch.exp(0.5 * _randn(gen, 1, r)) + 0.3 * _randn(gen, n, 1)
    big = torch.rand(n, 1, generator=gen, device=gen.device) < 0.01
    return torch.where(big, v * 16.0, v)


def _quantise(v):
    """Codes (as floats) and steps of a float32 matrix in blocks of 32 features."""
    n, r = v.shape
    b = -(-r // BLOCK)
    blocks = torch.zeros(n, b * BLOCK, dtype=torch.float32, device=v.device)
    blocks[:, :r] = v
    blocks = blocks.view(n, b, BLOCK)
    top = blocks.abs().amax(-1, keepdim=True)
    # Biased exponent of the smallest power of two that brings the block's largest magnitude
    # below 127.5: seven bits below the magnitude's own exponent, one more from 127.5 / 128 up.
    s = (((top.view(torch.int32) + 0x10000) >> 23) - 6).clamp(min=1)
    step = (s << 23).view(torch.float32)
    back = ((254 - s) << 23).view(torch.float32)
    return torch.round(blocks * back), step, s


def _checkpoint(v):
    codes, _, s = _quantise(v)
    n = v.shape[0]
    return torch.cat([codes.to(torch.int8).view(torch.uint8).reshape(-1), s.to(torch.uint8).reshape(-1)]) if n else \
        torch.empty(0, dtype=torch.uint8, device=v.device)


def prepare(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(int(seed))
    n, c, t, d, dt = case["N"], case["C"], case["T"], case["D"], _dtype(case)
    r = c * t
    s = {"case": case, "plan": None}
    if case["op"] in ("norm", "norm_step"):
        s["x"] = _activations(gen, n, r).to(dt)
        s["gamma"] = (1.0 + 0.2 * _randn(gen, c)).to(dt)
        s["beta"] = (0.1 * _randn(gen, c)).to(dt)
        if case["op"] == "norm_step":
            s["dy"] = (0.05 * _randn(gen, n, r)).to(dt)
            s["dres"] = (0.05 * _randn(gen, n, r)).to(dt)
    elif case["op"] == "round_trip":
        s["x"] = _activations(gen, n, r).to(dt)
    elif case["op"] == "gelu_grad":
        s["ckpt"] = _checkpoint(_randn(gen, n, r))
        s["dy"] = (0.05 * _randn(gen, n, r)).to(dt)
    else:
        s["ckpt"] = _checkpoint(_randn(gen, n, r))
        s["dy"] = (0.05 * _randn(gen, n, d * t)).to(dt)
        s["gamma"] = (1.0 + 0.2 * _randn(gen, c)).to(dt) if case["view"] == "affine" else None
        s["beta"] = (0.1 * _randn(gen, c)).to(dt) if case["view"] == "affine" else None
    return s


# ---------------------------------------------------------------------------
# The plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _decode(ckpt, n, r):
    b = -(-r // BLOCK)
    codes = ckpt[:n * b * BLOCK].view(torch.int8).view(n, b, BLOCK).float()
    step = (ckpt[n * b * BLOCK:].view(n, b, 1).to(torch.int32) << 23).view(torch.float32)
    return (codes * step).reshape(n, b * BLOCK)[:, :r]


def _normalise(x):
    x = x.float()
    centred = x - x.sum(-1, keepdim=True) / x.shape[-1]
    rstd = 1.0 / torch.sqrt((centred * centred).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return centred * rstd, rstd


def _per_feature(p, t):
    return p.float().repeat_interleave(t)


def _plain_norm(s):
    t, dt = s["case"]["T"], s["x"].dtype
    h, _ = _normalise(s["x"])
    return (h * _per_feature(s["gamma"], t) + _per_feature(s["beta"], t)).to(dt)


def _plain_norm_step(s):
    case, dt = s["case"], s["x"].dtype
    n, c, t = case["N"], case["C"], case["T"]
    h, rstd = _normalise(s["x"])
    gamma = _per_feature(s["gamma"], t)
    y = (h * gamma + _per_feature(s["beta"], t)).to(dt)
    if case["keep"] == "8bit":
        codes, step, _ = _quantise(h)
        h = (codes * step).reshape(n, -1)[:, :c * t]
    dy = s["dy"].float()
    g = dy * gamma
    r = c * t
    dx = rstd * (g - g.sum(-1, keepdim=True) / r - h * ((g * h).sum(-1, keepdim=True) / r)) + s["dres"].float()
    dgamma = (dy * h).view(n, c, t).sum((0, 2))
    dbeta = dy.view(n, c, t).sum((0, 2))
    return {"y": y, "dx": dx.to(dt), "dgamma": dgamma.to(dt), "dbeta": dbeta.to(dt)}


def _plain_round_trip(s):
    n, r = s["x"].shape
    codes, step, _ = _quantise(s["x"].float())
    return (codes * step).reshape(n, -1)[:, :r].to(s["x"].dtype)


def _plain_gelu_grad(s):
    case, dt = s["case"], s["dy"].dtype
    n, d, t = case["N"], case["C"], case["T"]
    v = _decode(s["ckpt"], n, d * t)
    slope = 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1.0 / math.sqrt(2.0 * math.pi))
    dpre = s["dy"].float() * slope
    return {"dpre": dpre.to(dt), "dbias": dpre.view(n, d, t).sum((0, 2)).to(dt)}


def _plain_weight_grad(s):
    case, dt = s["case"], s["dy"].dtype
    n, c, d, t = case["N"], case["C"], case["D"], case["T"]
    v = _decode(s["ckpt"], n, c * t)
    if case["view"] == "affine":
        v = v * _per_feature(s["gamma"], t) + _per_feature(s["beta"], t)
    elif case["view"] == "gelu":
        v = 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    # The unrolled layer's gradient, folded onto the entries that share a parameter:
    # dw[d, c, t] = sum over g of dense[d, g, c, (g - t) mod T].
    dense = (s["dy"].float().t() @ v).view(d, t, c, t).permute(1, 3, 0, 2)
    g = torch.arange(t, device=v.device)
    dw = dense[g[None, :], (g[None, :] - g[:, None]) % t].sum(1)
    return dw.permute(1, 2, 0).to(dt).contiguous()


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _plan(s):
    """The output buffers and workspaces a program keeps from step to step."""
    import group_circulant_linear_p4_amd as eql
    case = s["case"]
    n, c, t, d, dt = case["N"], case["C"], case["T"], case["D"], _dtype(case)
    dev = (s["x"] if "x" in s else s["dy"]).device
    p = {"eql": eql}

    def scratch(nbytes):
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)

    if case["op"] == "norm":
        p["y"] = torch.empty_like(s["x"])
    elif case["op"] == "norm_step":
        p["y"], p["dx"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        p["dgamma"], p["dbeta"] = torch.empty_like(s["gamma"]), torch.empty_like(s["gamma"])
        p["mean"] = torch.empty(n, dtype=torch.float32, device=dev) if case["keep"] == "x" else None
        p["rstd"] = torch.empty(n, dtype=torch.float32, device=dev)
        p["ckpt"] = scratch(eql.eqlinear_ckpt8_bytes(n, c, t)) if case["keep"] == "8bit" else None
        p["bytes"] = eql.eqlinear_layernorm_bwd_workspace_bytes(n, c, t, dt)
        p["ws"] = scratch(p["bytes"])
    elif case["op"] == "round_trip":
        p["ckpt"], p["back"] = scratch(eql.eqlinear_ckpt8_bytes(n, c, t)), torch.empty_like(s["x"])
    elif case["op"] == "gelu_grad":
        p["dpre"], p["dbias"] = torch.empty_like(s["dy"]), torch.empty(c, dtype=dt, device=dev)
        p["bytes"] = eql.eqlinear_fused_epilogue_bwd_workspace_bytes(n, c, t, dt)
        p["ws"] = scratch(p["bytes"])
    else:
        p["dw"] = torch.empty(d, c, t, dtype=dt, device=dev)
        p["bytes"] = eql.eqlinear_bwd_w_workspace_bytes(n, c, d, t, dt)
        p["ws"] = scratch(p["bytes"])
    return p


def _own(s):
    if s["plan"] is None:
        s["plan"] = _plan(s)
    case, p = s["case"], s["plan"]
    n, c, t, d, dt, eql = case["N"], case["C"], case["T"], case["D"], _dtype(case), p["eql"]
    if case["op"] == "norm":
        eql.eqlinear_layernorm_fwd(s["x"], s["gamma"], s["beta"], p["y"], None, None, None, n, c, t, EPS, dt)
        return p["y"]
    if case["op"] == "norm_step":
        eql.eqlinear_layernorm_fwd(s["x"], s["gamma"], s["beta"], p["y"], p["ckpt"], p["mean"], p["rstd"], n, c, t, EPS, dt)
        if case["keep"] == "8bit":
            eql.eqlinear_layernorm_bwd_ckpt8(s["dy"], p["ckpt"], p["rstd"], s["gamma"], s["dres"], p["dx"], p["dgamma"],
                                             p["dbeta"], p["ws"], p["bytes"], n, c, t, dt)
        else:
            eql.eqlinear_layernorm_bwd(s["dy"], s["x"], p["mean"], p["rstd"], s["gamma"], s["dres"], p["dx"], p["dgamma"],
                                       p["dbeta"], p["ws"], p["bytes"], n, c, t, dt)
        return {"y": p["y"], "dx": p["dx"], "dgamma": p["dgamma"], "dbeta": p["dbeta"]}
    if case["op"] == "round_trip":
        eql.eqlinear_ckpt8_pack(s["x"], p["ckpt"], n, c, t, dt)
        eql.eqlinear_ckpt8_unpack(p["ckpt"], p["back"], n, c, t, dt)
        return p["back"]
    if case["op"] == "gelu_grad":
        eql.eqlinear_fused_epilogue_bwd_ckpt8(s["dy"], s["ckpt"], p["dpre"], p["dbias"], p["ws"], p["bytes"], n, c, t, dt)
        return {"dpre": p["dpre"], "dbias": p["dbias"]}
    act = eql.EQL_ACT_GELU if case["view"] == "gelu" else eql.EQL_ACT_NONE
    eql.eqlinear_bwd_w_ckpt8(s["ckpt"], s["gamma"], s["beta"], act, s["dy"], p["dw"], p["ws"], p["bytes"], n, c, d, t, dt)
    return p["dw"]


_PLAIN = {"norm": _plain_norm, "norm_step": _plain_norm_step, "round_trip": _plain_round_trip,
          "gelu_grad": _plain_gelu_grad, "weight_grad": _plain_weight_grad}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    n, c, t, d, op = case["N"], case["C"], case["T"], case["D"], case["op"]
    r, e = c * t, 2 if case["dtype"] == "f16" else 4
    kept = r + -(-r // BLOCK)  # bytes of a checkpoint's row
    if op == "norm":
        return {"bytes": n * r * e * 2 + 2 * c * e, "flops": 8 * n * r}
    if op == "norm_step":
        # Forward: x in, y out and what is kept out; backward: dy, dres and what was kept in,
        # dx out.
        keep = n * r * e if case["keep"] == "x" else 2 * n * kept
        return {"bytes": n * r * e * 5 + keep + 4 * c * e, "flops": 24 * n * r}
    if op == "round_trip":
        return {"bytes": n * r * e * 2 + 2 * n * kept, "flops": 4 * n * r}
    if op == "gelu_grad":
        return {"bytes": n * r * e * 2 + n * kept + c * e, "flops": 30 * n * r}
    # One product per real frequency and four per complex pair of the half spectrum.
    real = 2 if t % 2 == 0 and t > 1 else 1
    return {"bytes": n * kept + n * d * t * e + d * c * t * e, "flops": 2 * (real + 2 * (t - real)) * n * c * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _power64(exponent):
    """2^exponent in 64 bits, from its bits."""
    return ((exponent.to(torch.int64) + 1023) << 52).view(torch.float64)


def _read64(ckpt, n, r):
    width = (r + BLOCK - 1) // BLOCK * BLOCK
    codes = ckpt[:n * width].view(torch.int8).reshape(n, width)[:, :r].double()
    unit = _power64(ckpt[n * width:].reshape(n, width // BLOCK).to(torch.int64) - 127)
    return codes * unit.repeat_interleave(BLOCK, 1)[:, :r]


def _round8_64(v):
    """Each value rounded to the step of its block of 32: the largest magnitude takes at most
    127 steps, a step being the smallest power of two that allows it."""
    n, r = v.shape
    pad = (-r) % BLOCK
    w = torch.nn.functional.pad(v, (0, pad)).reshape(n, -1, BLOCK)
    top = w.abs().amax(-1, keepdim=True)
    exponent = torch.frexp(top)[1] - 7  # top = f 2^(exponent + 7), f in [1/2, 1)
    unit = _power64(exponent.clamp(min=-126))
    unit = torch.where(top >= 127.5 * unit, 2.0 * unit, unit)
    return (torch.round(w / unit) * unit).reshape(n, -1)[:, :r]


def exact(case, seed):
    s = prepare(case, seed)
    n, c, t, d, op = case["N"], case["C"], case["T"], case["D"], case["op"]
    if op == "round_trip":
        return _round8_64(s["x"].double())
    if op in ("norm", "norm_step"):
        x = s["x"].double().view(n, c, t)
        gamma, beta = s["gamma"].double()[:, None], s["beta"].double()[:, None]
        var, mean = torch.var_mean(x, dim=(1, 2), correction=0, keepdim=True)
        h = (x - mean) / torch.sqrt(var + EPS)
        y = (gamma * h + beta).view(n, c * t)
        if op == "norm":
            return y
        if case["keep"] == "8bit":
            h = _round8_64(h.reshape(n, c * t)).view(n, c, t)
        dy = s["dy"].double().view(n, c, t)
        g = dy * gamma
        dx = (g - g.mean((1, 2), keepdim=True) - h * (g * h).mean((1, 2), keepdim=True)) / torch.sqrt(var + EPS)
        return {"y": y, "dx": dx.view(n, c * t) + s["dres"].double(), "dgamma": (dy * h).sum(2).sum(0),
                "dbeta": dy.sum(2).sum(0)}
    kept = _read64(s["ckpt"], n, c * t)
    if op == "gelu_grad":
        phi = 0.5 * torch.erfc(-kept / math.sqrt(2.0))
        dpre = s["dy"].double() * (phi + kept * torch.exp(-kept * kept / 2.0) / math.sqrt(2.0 * math.pi))
        return {"dpre": dpre, "dbias": dpre.view(n, c, t).sum(2).sum(0)}
    if case["view"] == "affine":
        kept = (s["gamma"].double()[:, None] * kept.view(n, c, t) + s["beta"].double()[:, None]).view(n, c * t)
    elif case["view"] == "gelu":
        kept = kept * 0.5 * torch.erfc(-kept / math.sqrt(2.0))
    kept, dy = kept.view(n, c, t), s["dy"].double().view(n, d, t)
    dw = torch.empty(d, c, t, dtype=torch.float64, device=kept.device)
    for j in range(t):
        total = torch.zeros(d, c, dtype=torch.float64, device=kept.device)
        for g in range(t):
            total += dy[:, :, g].t().contiguous() @ kept[:, :, (g - j) % t].contiguous()
        dw[:, :, j] = total
    return dw
