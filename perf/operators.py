"""Measured cases of the floating-point layers of a transformer block: layer
norm and the linear layer (bias, activation and residual in one call), each
with its backward pass.

``prepare`` makes what a program has in hand before the call, ``run`` makes
one call (``own``: the framework's; otherwise the same mathematics in
elementary torch operations in 32 bits, rounded once at the end), ``exact``
is the operator's definition in 64 bits.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------
def _ln(name, rows, d, x, y):
    return {"name": name, "op": "layer_norm", "rows": rows, "d": d, "x": x, "y": y}


def _ln_bwd(name, rows, d, x, y, add):
    return {"name": name, "op": "layer_norm_backward", "rows": rows, "d": d, "x": x, "y": y, "add": add}


def _lin(name, m, n, k, t, out, act, bias, res, pre):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "t": t, "out": out, "act": act,
            "bias": bias, "res": res, "pre": pre}


def _lin_bwd(name, m, n, k, t, dout, act):
    return {"name": name, "op": "linear_backward", "m": m, "n": n, "k": k, "t": t, "out": dout, "act": act}


def listed():
    return [
        # one image through a block: 257 tokens, latency
        _ln("ln_image", 257, 1024, "bf16", "bf16"),
        # a batch of 256 images kept in fp32 between the layers, normalised for a bf16 linear
        _ln("ln_batch", 65792, 1024, "f32", "bf16"),
        # an odd width: rows that no vector load fits; the fp32 result goes on to the quantiser
        _ln("ln_odd", 4099, 997, "bf16", "f32"),
        # fine-tuning, 16 images, with the skipped branch's gradient added
        _ln_bwd("ln_bwd_block", 4112, 1024, "bf16", "bf16", True),
        # fine-tuning, 128 images kept in fp32
        _ln_bwd("ln_bwd_batch", 32896, 1024, "f32", "f32", False),
        # one image's class token into the classifier
        _lin("head_single", 1, 1000, 1024, "bf16", "f32", "none", True, False, False),
        # one image's projection with its residual, all in fp32
        _lin("proj_image_f32", 257, 1024, 1024, "f32", "f32", "none", True, True, False),
        # MLP fc1 of 16 images in training: the pre-activation is kept
        _lin("fc1_train", 4112, 4096, 1024, "bf16", "bf16", "gelu", True, False, True),
        # MLP fc2 of 128 images, added to an fp32 residual
        _lin("fc2_batch", 32896, 1024, 4096, "bf16", "f32", "none", True, True, False),
        # MLP fc1's gradients, 16 images
        _lin_bwd("fc1_bwd", 4112, 4096, 1024, "bf16", "bf16", "gelu"),
        # gradients of a small adapter with odd sizes
        _lin_bwd("adapter_bwd_odd", 1285, 333, 1022, "f16", "f16", "relu"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi):
    """A width over [lo, hi]: half of them any number, half multiples of 64, as models have."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.5 or v < 64 else v // 64 * 64


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "linear", "linear", "linear_backward"])
    if op == "layer_norm" or op == "layer_norm_backward":
        d = _width(rng, 16, 8192)
        rows = _log(rng, 1, min(65792, 33_000_000 // d))
        x = rng.choice(["f32", "bf16", "f16"])
        y = rng.choice([x, "f32"] if x != "f32" else ["f32", "bf16", "f16"])
        case = {"op": op, "rows": rows, "d": d, "x": x, "y": y}
        if op == "layer_norm_backward":
            case["add"] = rng.random() < 0.5
        return case
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    n, k = _width(rng, 16, 4096), _width(rng, 16, 4096)
    m = _log(rng, 1, 32896)
    # no larger than the largest listed cases
    m = max(1, min(m, (130_000_000_000 if t != "f32" else 16_000_000_000) // (2 * n * k)))
    act = rng.choice(["none", "gelu", "gelu_tanh", "relu", "silu"])
    out = rng.choice([t, "f32"])
    if op == "linear_backward":
        return {"op": op, "m": m, "n": n, "k": k, "t": t, "out": out, "act": act}
    return {"op": op, "m": m, "n": n, "k": k, "t": t, "out": out, "act": act, "bias": rng.random() < 0.8,
            "res": rng.random() < 0.5, "pre": act != "none" and rng.random() < 0.5}


# ---- inputs --------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def heavy(*shape):
        """Student-t(4) activations, the tails that a block's inputs have."""
        z = torch.randn(*shape, device="cuda", generator=g)
        chi = torch.zeros_like(z)
        for _ in range(4):
            chi.addcmul_(*(2 * [torch.randn(*shape, device="cuda", generator=g)]))
        return z.div_(chi.mul_(0.25).sqrt_().clamp_(min=1e-2))

    s = dict(case)
    op = case["op"]
    if op.startswith("layer_norm"):
        rows, d = case["rows"], case["d"]
        s["x_"] = heavy(rows, d).add_(0.3 * normal(rows, 1)).to(DT[case["x"]])
        s["w_"] = 1 + 0.2 * normal(d)
        s["b_"] = 0.1 * normal(d)
        if op == "layer_norm_backward":
            xf = s["x_"].float()
            s["dy_"] = (0.05 * normal(rows, d)).to(DT[case["y"]])
            s["mean_"] = xf.mean(1)
            s["rstd_"] = (xf.var(1, unbiased=False) + EPS).rsqrt()
            s["add_"] = (0.05 * normal(rows, d)).to(DT[case["x"]]) if case["add"] else None
        return s
    m, n, k, t, o = case["m"], case["n"], case["k"], DT[case["t"]], DT[case["out"]]
    s["x_"] = heavy(m, k).to(t)
    s["w_"] = (0.02 * normal(n, k)).to(t)
    if op == "linear":
        s["b_"] = 0.1 * normal(n) if case["bias"] else None
        s["r_"] = normal(m, n).to(o) if case["res"] else None
    else:
        s["dout_"] = (0.05 * normal(m, n)).to(o)
        s["pre_"] = normal(m, n).to(t) if case["act"] != "none" else None
    return s


# ---- the calls -----------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain_layer_norm(s):
    x = s["x_"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + EPS)
    return (c * rstd[:, None] * s["w_"] + s["b_"]).to(DT[s["y"]]), mean, rstd


def _plain_layer_norm_backward(s):
    dy, h = s["dy_"].float(), (s["x_"].float() - s["mean_"][:, None]) * s["rstd_"][:, None]
    g = dy * s["w_"]
    dx = (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True)) * s["rstd_"][:, None]
    if s["add_"] is not None:
        dx = dx + s["add_"].float()
    return dx.to(s["x_"].dtype), (dy * h).sum(0), dy.sum(0)


def _plain_linear(s):
    z = s["x_"].float() @ s["w_"].float().t()
    if s["b_"] is not None:
        z = z + s["b_"]
    out = _act(z, s["act"])
    if s["r_"] is not None:
        out = out + s["r_"].float()
    out = out.to(DT[s["out"]])
    return (out, z.to(DT[s["t"]])) if s["pre"] else out


def _plain_linear_backward(s):
    t = DT[s["t"]]
    dz = s["dout_"].float()
    if s["act"] != "none":
        dz = dz * _act_grad(s["pre_"].float(), s["act"])
    return (dz @ s["w_"].float()).to(t), (dz.t() @ s["x_"].float()).to(t), dz.sum(0).to(t)


_plain = {"layer_norm": _plain_layer_norm, "layer_norm_backward": _plain_layer_norm_backward,
          "linear": _plain_linear, "linear_backward": _plain_linear_backward}


def _own_layer_norm(s):
    from mixed_precision_vit_b200 import sc
    return sc.layer_norm(s["x_"], s["w_"], s["b_"], EPS, out_dtype=DT[s["y"]], want_stats=True)


def _own_layer_norm_backward(s):
    from mixed_precision_vit_b200 import sc
    return sc.layer_norm_backward(s["dy_"], s["x_"], s["mean_"], s["rstd_"], s["w_"], dx_add=s["add_"])


def _own_linear(s):
    from mixed_precision_vit_b200 import sc
    out, pre = sc.linear(s["x_"], s["w_"], s["b_"], s["r_"], s["act"], out_dtype=DT[s["out"]],
                         want_pre=s["pre"])
    return (out, pre) if s["pre"] else out


def _own_linear_backward(s):
    from mixed_precision_vit_b200 import sc
    return sc.linear_backward(s["dout_"], s["x_"], s["w_"], s["pre_"], s["act"])


_own = {"layer_norm": _own_layer_norm, "layer_norm_backward": _own_layer_norm_backward,
        "linear": _own_linear, "linear_backward": _own_linear_backward}


# ---- what a pass cannot do without ---------------------------------------------------------
def work(case):
    op = case["op"]
    if op.startswith("layer_norm"):
        rows, d, sx, sy = case["rows"], case["d"], SIZE[case["x"]], SIZE[case["y"]]
        if op == "layer_norm":
            return {"bytes": rows * d * (sx + sy) + 8 * d + 8 * rows, "flops": 8 * rows * d}
        return {"bytes": rows * d * ((3 if case["add"] else 2) * sx + sy) + 12 * d + 8 * rows,
                "flops": 14 * rows * d}
    m, n, k, st, so = case["m"], case["n"], case["k"], SIZE[case["t"]], SIZE[case["out"]]
    if op == "linear":
        b = (m * k + n * k) * st + m * n * so * (2 if case["res"] else 1)
        return {"bytes": b + (4 * n if case["bias"] else 0) + (m * n * st if case["pre"] else 0),
                "flops": 2 * m * n * k}
    b = m * n * so + (m * n * st if case["act"] != "none" else 0) + 2 * (m * k + n * k) * st + n * st
    return {"bytes": b, "flops": 4 * m * n * k}


# ---- the definitions in 64 bits ------------------------------------------------------------
def _phi(z):
    """The normal distribution's cumulative function, accurate in its lower tail."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d64 = {k: v.double() for k, v in s.items() if torch.is_tensor(v)}
    x, w = d64["x_"], d64["w_"]
    if op == "layer_norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        return torch.einsum("ij,i,j->ij", x - mean.unsqueeze(1), rstd, w) + d64["b_"], mean, rstd
    if op == "layer_norm_backward":
        mean, rstd, dy = d64["mean_"].unsqueeze(1), d64["rstd_"].unsqueeze(1), d64["dy_"]
        h = (x - mean) * rstd
        n = x.shape[1]
        s1 = (dy @ w).unsqueeze(1)
        s2 = ((dy * h) @ w).unsqueeze(1)
        dx = rstd * (dy * w - (s1 + h * s2) / n)
        if "add_" in d64:
            dx = dx + d64["add_"]
        return dx, torch.einsum("ij,ij->j", dy, h), dy.sum(dim=0)
    act = case["act"]
    k0 = math.sqrt(2.0 / math.pi)
    if op == "linear":
        z = torch.nn.functional.linear(x, w, d64.get("b_"))
        if act == "gelu":
            a = z * _phi(z)
        elif act == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
            a = z * torch.sigmoid(2 * k0 * z * (1 + 0.044715 * z ** 2))
        elif act == "silu":
            a = z * torch.sigmoid(z)
        elif act == "relu":
            a = z.clamp(min=0)
        else:
            a = z
        if "r_" in d64:
            a = a + d64["r_"]
        return (a, z) if case["pre"] else a
    dz = d64["dout_"]
    if act != "none":
        z = d64["pre_"]
        if act == "gelu":
            d = _phi(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
        elif act == "gelu_tanh":
            q = torch.sigmoid(2 * k0 * z * (1 + 0.044715 * z ** 2))
            d = q + z * q * (1 - q) * 2 * k0 * (1 + 0.134145 * z ** 2)
        elif act == "silu":
            q = torch.sigmoid(z)
            d = q + z * q * (1 - q)
        else:
            d = torch.heaviside(z, torch.zeros_like(z))
        dz = dz * d
    return dz.matmul(w), torch.einsum("mn,mk->nk", dz, x), dz.sum(dim=0)
