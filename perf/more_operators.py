"""The EQ-Linear layer in 8-bit integers and the RMS norm in front of it, as they are measured.

A case's "op" is one of

  norm         residual addition and RMS norm of rows of C'*T features, one weight per channel
               (shared by the channel's T group elements)
  norm_step    that, and its backward pass in a pre-norm block (the residual stream's gradient is
               added to the input's)
  linear8      activations to 8 bits (half spectrum, one scale for each row and frequency), and the
               layer as a product of 8-bit integers with the packed weight (one scale for each
               output channel and frequency), with bias, GELU or a residual where the case says so
  norm_linear8 residual addition, RMS norm with its output in those 8 bits, and the layer

8-bit form of a row (or of one output channel's weights), from its planes
    V[0] = sum_g v_g,  V[T/2] = sum_g (-1)^g v_g (even T),  V[k] = sum_g v_g exp(-2 pi i g k / T):
each frequency has m = max |Re|, |Im| over the channels (at least 2^-100), codes
round(plane * (127 / m)), product and quotient rounded to 32 bits, and the scale m / 127.
"""
import math

import torch

own = False

EPS = 1e-6
FLOOR = 2.0 ** -100


def _case(name, op, dtype, n, c, t, d=0, act="none", residual=False):
    return {"name": name, "op": op, "dtype": dtype, "N": n, "C": c, "T": t, "D": d, "act": act, "residual": residual}


def listed():
    return [
        # One token at the width of the largest benchmarked layer: what a single step of serving pays.
        _case("norm one token f16", "norm", "f16", 1, 1024, 4),
        # A small ViT's batch (64 images) in inference form.
        _case("norm vit f16", "norm", "f16", 12608, 96, 4),
        # Full-precision training with eight rotations.
        _case("norm step C8 f32", "norm_step", "f32", 16384, 64, 8),
        # Rows of 513 features: a ragged three-fold layer.
        _case("norm step ragged f16", "norm_step", "f16", 5003, 171, 3),
        # The widest block's training batch.
        _case("norm step square f16", "norm_step", "f16", 65536, 1024, 4),
        # One token through the largest benchmarked layer.
        _case("linear8 one token f16", "linear8", "f16", 1, 1024, 4, d=1024),
        # Five-fold layer of sizes that nothing divides.
        _case("linear8 odd f16", "linear8", "f16", 3001, 133, 5, d=171),
        # An ordinary linear layer (one group element) in full precision outside of the product.
        _case("linear8 dense f32", "linear8", "f32", 4096, 1024, 1, d=1024),
        # Second layer of a small ViT's MLP, with the block's residual.
        _case("linear8 vit out f16", "linear8", "f16", 12608, 384, 4, d=96, residual=True),
        # The widest block's second layer.
        _case("linear8 square f16", "linear8", "f16", 65536, 1024, 4, d=1024, residual=True),
        # One image's tokens through the norm and first layer of a small ViT's MLP.
        _case("norm linear8 one image f16", "norm_linear8", "f16", 197, 96, 4, d=384, act="gelu"),
        # The same for a batch of a Swin block's width.
        _case("norm linear8 swin f16", "norm_linear8", "f16", 50176, 192, 4, d=192, act="gelu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_step", "linear8", "norm_linear8"])
    dtype = rng.choice(["f16", "f32"])
    t = rng.choice([1, 2, 3, 4, 4, 5, 6, 8, 12])
    if op in ("linear8", "norm_linear8") and dtype == "f32":
        # In full precision one group element: outputs of 32 bits are held closer together than two
        # ways to sum a spectrum are, next to a code's border.
        t = 1
    c = max(1, _log_int(rng, 24, 6000) // t)
    n = max(1, min(_log_int(rng, 1, 60000), (1 << 26) // (c * t)))
    d, act, residual = 0, "none", False
    if op in ("linear8", "norm_linear8"):
        d = max(1, _log_int(rng, 16, 4096) // t)
        n = max(1, min(n, (1 << 38) // (c * t * d * t)))
        act, residual = rng.choice([("none", False), ("gelu", False), ("none", True)])
    case = _case("", op, dtype, n, c, t, d, act, residual)
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


def prepare(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(int(seed))
    n, c, t, d, dt, op = case["N"], case["C"], case["T"], case["D"], _dtype(case), case["op"]
    r = c * t
    s = {"case": case, "plan": None, "x": _activations(gen, n, r).to(dt)}
    if op != "linear8":
        s["r"] = _randn(gen, n, r).to(dt)
        s["gamma"] = (1.0 + 0.2 * _randn(gen, c)).to(dt)
    if op == "norm_step":
        s["dy"] = (0.05 * _randn(gen, n, r)).to(dt)
        s["dres"] = (0.05 * _randn(gen, n, r)).to(dt)
    if op in ("linear8", "norm_linear8"):
        # A layer's weight is laid out once: in 8 bits for the plain form, and by the library's own
        # packing at the first call.
        s["w"] = (_randn(gen, d, c, t) / math.sqrt(r)).to(dt)
        s["transform"], s["back"] = _transforms(t, s["w"].device)
        s["w8"] = _eight_bits(_planes(s["w"], s["transform"]), t)
        s["bias"] = (0.1 * _randn(gen, d)).to(dt)
        s["res"] = _randn(gen, n, d * t).to(dt) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------
# The plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _real(t):
    """How many of the T planes belong to a real frequency (0, and T / 2)."""
    return 2 if t % 2 == 0 else 1


def _transforms(t, device):
    """The transform of T group elements into the half spectrum's T planes, and back, as matrices
    [T, T] in 32 bits, their angles in 64."""
    p = torch.arange(t, device=device)
    nr = _real(t)
    k = torch.where(p == 0, 0, torch.where(p < nr, t // 2, (p - nr) // 2 + 1))
    angle = 2.0 * math.pi * ((k[:, None] * p[None, :]) % t).double() / t
    imag = ((p >= nr) & ((p - nr) % 2 == 1))[:, None]
    m = torch.where(imag, -torch.sin(angle), torch.cos(angle))
    m = torch.where(m.abs() < 1e-12, 0.0, m)
    return m.float(), (m * torch.where(p < nr, 1.0, 2.0)[:, None] / t).float()


def _planes(v, transform):
    """[rows, C, T] -> the T real planes of the half spectrum, [T, rows, C]."""
    rows, c, t = v.shape
    return (v.float().reshape(-1, t) @ transform.t()).view(rows, c, t).permute(2, 0, 1).contiguous()


def _eight_bits(planes, t):
    """Codes (as floats, [T, rows, C]) and scales ([T, rows, 1], equal for a frequency's two planes)."""
    nr = _real(t)
    top = planes.abs().amax(-1, keepdim=True)
    both = top[nr:].view(-1, 2, *top.shape[1:]).amax(1).repeat_interleave(2, 0)
    top = torch.cat([top[:nr], both]).clamp(min=FLOOR)
    return torch.round(planes * (127.0 / top)), top / 127.0


def _plain_sum_norm(s):
    """The residual stream after the addition, its rows' 1 / rms, and both in 32 bits."""
    total = (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    v = total.float()
    rstd = 1.0 / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS)
    return total, v, rstd


def _plain_norm(s):
    t = s["case"]["T"]
    total, v, rstd = _plain_sum_norm(s)
    return {"sum": total, "y": (v * rstd * s["gamma"].float().repeat_interleave(t)).to(total.dtype)}


def _plain_norm_step(s):
    case, dt = s["case"], s["x"].dtype
    n, c, t = case["N"], case["C"], case["T"]
    total, v, rstd = _plain_sum_norm(s)
    gamma = s["gamma"].float().repeat_interleave(t)
    h = v * rstd
    dy = s["dy"].float()
    g = dy * gamma
    dx = rstd * (g - h * ((g * h).sum(-1, keepdim=True) / (c * t))) + s["dres"].float()
    return {"sum": total, "y": (h * gamma).to(dt), "dx": dx.to(dt), "dgamma": (dy * h).view(n, c, t).sum((0, 2)).to(dt)}


def _plain_product(s, codes, scales):
    """The layer's output from the activations' codes and scales."""
    case, dt = s["case"], s["x"].dtype
    n, t, d, nr = case["N"], case["T"], case["D"], _real(case["T"])
    wc, ws = s["w8"]
    real = torch.bmm(codes[:nr], wc[:nr].transpose(1, 2).contiguous())
    # A complex frequency's product as a real one: [Xr, Xi] times [[Wr, Wi], [-Wi, Wr]].
    x2 = codes[nr:].view(-1, 2, n, codes.shape[-1]).permute(0, 2, 1, 3).reshape(-1, n, 2 * codes.shape[-1])
    wr, wi = wc[nr::2], wc[nr + 1::2]
    w2 = torch.cat([torch.cat([wr, -wi], -1), torch.cat([wi, wr], -1)], 1).transpose(1, 2).contiguous()
    pair = torch.bmm(x2, w2).view(-1, n, 2, d).permute(0, 2, 1, 3).reshape(-1, n, d)
    planes = torch.cat([real, pair]) * scales * ws.transpose(1, 2)
    y = (planes.reshape(t, -1).t() @ s["back"]).view(n, d, t)
    y = y + s["bias"].float()[:, None]
    if case["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    y = y.view(n, d * t)
    return (y if s["res"] is None else y + s["res"].float()).to(dt)


def _plain_linear8(s):
    case = s["case"]
    planes = _planes(s["x"].view(case["N"], case["C"], case["T"]), s["transform"])
    return _plain_product(s, *_eight_bits(planes, case["T"]))


def _plain_norm_linear8(s):
    case = s["case"]
    total, v, rstd = _plain_sum_norm(s)
    planes = _planes(v.view(case["N"], case["C"], case["T"]), s["transform"]) * s["gamma"].float()
    codes, scales = _eight_bits(planes, case["T"])
    return {"sum": total, "y": _plain_product(s, codes, scales * rstd)}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _plan(s):
    """The packed weight, output buffers and workspaces a program keeps from step to step."""
    import group_circulant_linear_p4_amd as eql
    case = s["case"]
    n, c, t, d, dt, dev = case["N"], case["C"], case["T"], case["D"], _dtype(case), s["x"].device
    p = {"eql": eql}

    def scratch(nbytes):
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)

    if case["op"] != "linear8":
        p["sum"] = torch.empty_like(s["x"])
    if case["op"] in ("norm", "norm_step"):
        p["y"] = torch.empty_like(s["x"])
    if case["op"] == "norm_step":
        p["dx"], p["dgamma"] = torch.empty_like(s["x"]), torch.empty_like(s["gamma"])
        p["rstd"] = torch.empty(n, dtype=torch.float32, device=dev)
        p["bytes"] = eql.eqlinear_rmsnorm_bwd_workspace_bytes(n, c, t, dt)
        p["ws"] = scratch(p["bytes"])
    if d:
        p["rows8"], p["w8"] = scratch(eql.eqlinear_q8_rows_bytes(n, c, t)), scratch(eql.eqlinear_q8_weight_bytes(d, c, t))
        p["y"] = torch.empty(n, d * t, dtype=dt, device=dev)
        eql.eqlinear_q8_pack_weight(s["w"], p["w8"], d, c, t, dt)
    return p


def _own(s):
    if s["plan"] is None:
        s["plan"] = _plan(s)
    case, p = s["case"], s["plan"]
    n, c, t, d, dt, eql = case["N"], case["C"], case["T"], case["D"], _dtype(case), p["eql"]
    if case["op"] == "norm":
        eql.eqlinear_rmsnorm_fwd(s["x"], s["r"], s["gamma"], p["sum"], p["y"], None, n, c, t, EPS, dt)
        return {"sum": p["sum"], "y": p["y"]}
    if case["op"] == "norm_step":
        eql.eqlinear_rmsnorm_fwd(s["x"], s["r"], s["gamma"], p["sum"], p["y"], p["rstd"], n, c, t, EPS, dt)
        eql.eqlinear_rmsnorm_bwd(s["dy"], p["sum"], p["rstd"], s["gamma"], s["dres"], p["dx"], p["dgamma"], p["ws"],
                                 p["bytes"], n, c, t, dt)
        return {"sum": p["sum"], "y": p["y"], "dx": p["dx"], "dgamma": p["dgamma"]}
    if case["op"] == "linear8":
        eql.eqlinear_q8_quantize(s["x"], p["rows8"], n, c, t, dt)
    else:
        eql.eqlinear_q8_rmsnorm(s["x"], s["r"], s["gamma"], p["sum"], p["rows8"], n, c, t, EPS, dt)
    act = eql.EQL_ACT_GELU if case["act"] == "gelu" else eql.EQL_ACT_NONE
    eql.eqlinear_q8_fwd(p["rows8"], p["w8"], s["bias"], s["res"], p["y"], n, c, d, t, dt, act)
    return p["y"] if case["op"] == "linear8" else {"sum": p["sum"], "y": p["y"]}


_PLAIN = {"norm": _plain_norm, "norm_step": _plain_norm_step, "linear8": _plain_linear8,
          "norm_linear8": _plain_norm_linear8}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    n, c, t, d, op = case["N"], case["C"], case["T"], case["D"], case["op"]
    r, e = c * t, 2 if case["dtype"] == "f16" else 4
    if op == "norm":
        return {"bytes": 4 * n * r * e + c * e, "flops": 6 * n * r}
    if op == "norm_step":
        # Forward: x and the residual in, sum and y out; backward: dy, sum and dres in, dx out.
        return {"bytes": 8 * n * r * e + 3 * c * e, "flops": 18 * n * r}
    # The activations in (with the norm: and the residual, and the sum out), the weight's codes in, the
    # output out.  One product per real frequency and four per complex one.
    rows = n * r * e * (1 if op == "linear8" else 3)
    out = n * d * t * e * (2 if case["residual"] else 1)
    nr = _real(t) if t > 1 else 1
    return {"bytes": rows + d * r + out, "flops": 2 * (nr + 2 * (t - nr)) * n * c * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _read_back64(v):
    """The values that the 8-bit form of [rows, C, T] stands for, in 64 bits."""
    t = v.shape[-1]
    grid = torch.arange(t, device=v.device, dtype=torch.float64)
    back = torch.zeros_like(v)
    for k in range(t // 2 + 1):
        cos, sin = torch.cos(2 * math.pi / t * (k * grid % t)), torch.sin(2 * math.pi / t * (k * grid % t))
        re, im = (v * cos).sum(-1), -(v * sin).sum(-1)
        if 2 * k % t == 0:
            im = torch.zeros_like(im)
        # The codes are whole numbers, defined by two operations in 32 bits.
        re, im = re.float(), im.float()
        top = torch.maximum(re.abs(), im.abs()).amax(1, keepdim=True).clamp(min=FLOOR)
        re, im = (torch.round(u * (127.0 / top)).double() * (top.double() / 127.0) for u in (re, im))
        back += (1 if 2 * k % t == 0 else 2) / t * (re[..., None] * cos - im[..., None] * sin)
    return back


def _layer64(s, x):
    """The layer on rows [N, C, T] that are read back from 8 bits already."""
    n, d, t = x.shape[0], s["case"]["D"], s["case"]["T"]
    w = _read_back64(s["w"].double())
    y = torch.zeros(n, d, t, dtype=torch.float64, device=x.device)
    for g in range(t):
        for h in range(t):
            y[:, :, g] += x[:, :, h].contiguous() @ w[:, :, (g - h) % t].t().contiguous()
    y += s["bias"].double()[:, None]
    if s["case"]["act"] == "gelu":
        y = y * 0.5 * torch.erfc(-y / math.sqrt(2.0))
    y = y.reshape(n, d * t)
    return y if s["res"] is None else y + s["res"].double()


def exact(case, seed):
    s = prepare(case, seed)
    n, c, t, op = case["N"], case["C"], case["T"], case["op"]
    if op == "linear8":
        return _layer64(s, _read_back64(s["x"].double().view(n, c, t)))
    total = s["x"].double() + s["r"].double()
    x = total.to(s["x"].dtype).double().view(n, c, t)  # the stream is kept in its own type
    rms = torch.sqrt((x * x).mean((1, 2), keepdim=True) + EPS)
    gamma = s["gamma"].double()[:, None]
    if op == "norm_linear8":
        return {"sum": total, "y": _layer64(s, _read_back64(gamma * x) / rms)}
    h = x / rms
    y = (gamma * h).reshape(n, c * t)
    if op == "norm":
        return {"sum": total, "y": y}
    dy = s["dy"].double().view(n, c, t)
    g = dy * gamma
    dx = (g - h * (g * h).mean((1, 2), keepdim=True)) / rms
    return {"sum": total, "y": y, "dx": dx.reshape(n, c * t) + s["dres"].double(), "dgamma": (dy * h).sum(2).sum(0)}
