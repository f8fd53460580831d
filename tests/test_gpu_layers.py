"""The floating-point layers against their definitions in 64 bits.

Tolerances are error bounds, elementwise.  u = 2^-24 is half a step of fp32 and
h(t) = finfo(t).eps / 2 half a step of the output's type t.  A sum of n fp32
terms in any order with d additions on the longest path is off by at most
d u sum|terms|; the tensor cores may cut where fp32 rounds, so there d is the
number of terms.  Every bound is the first-order sum of the roundings on the
way, with the counts written beside it."""
import math
import os
import subprocess
import sys

import pytest
import torch

from mixed_precision_vit_b200 import _lib as L
from mixed_precision_vit_b200 import sc

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


def h(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half a step below the normal range."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def close(got, ref, bound, what=""):
    assert got.shape == ref.shape, (got.shape, ref.shape)
    err = (got.double() - ref).abs()
    lim = bound + h(got.dtype) * (ref.abs() + bound) + tiny(got.dtype)
    bad = ~(err <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(err / lim).max().item():.3g} of the bound"


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def strided(t, pad):
    """The same matrix inside a wider one filled with NaN: (view, wider)."""
    big = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device=t.device)
    big[..., : t.shape[-1]] = t
    return big[..., : t.shape[-1]], big


# ---- layer norm ------------------------------------------------------------------------
def ln_ref(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    y = (x - mean) * rstd
    return (y * w.double() if w is not None else y) + (b.double() if b is not None else 0), mean, rstd


def ln_depth(D):
    """Additions on the longest path of a row sum: at most 32 values in a thread (D / 512 in
    rows too wide for registers), 5 shuffles and 16 warps; and 8 roundings around it."""
    return max(32, D / 512) + 21 + 8


def check_ln(x, w, b, out_dtype, eps=1e-6, out=None):
    y, mean, rstd = sc.layer_norm(x, w, b, eps, out_dtype=out_dtype, want_stats=True, out=out)
    ry, rm, rr = ln_ref(x, w, b, eps)
    xd, d = x.double().abs(), ln_depth(x.shape[-1])
    mabs = xd.mean(-1, keepdim=True)
    close(mean, rm[..., 0], d * U * mabs[..., 0], "mean")
    close(rstd, rr[..., 0], d * U * rr[..., 0] * (1 + (rr * mabs)[..., 0] * d * U * 2), "rstd")
    # the mean is off by d u mean|x|, r by d u relative, and the product and sum round
    wa = w.double().abs() if w is not None else 1.0
    ba = b.double().abs() if b is not None else 0.0
    close(y, ry, d * U * (wa * rr * (xd + mabs) + ba), "y")
    return y, mean, rstd


PAIRS = [(F32, F32), (F32, BF16), (F32, F16), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)]


@pytest.mark.parametrize("xt,yt", PAIRS)
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 64), (257, 1024), (33, 997), (9, 1000), (6, 4096),
                                    (5, 4100), (3, 8192), (2, 16384), (2, 20000), (2, 16391)])
def test_layer_norm(rows, D, xt, yt):
    g = gen(rows * 7919 + D)
    x = rnd(g, rows, D, dtype=xt, scale=2.0) + 1
    w, b = 1 + rnd(g, D, scale=0.2), rnd(g, D)
    check_ln(x, w, b, yt)


@pytest.mark.parametrize("wt", [F32, BF16, F16])
def test_layer_norm_params(wt):
    g = gen(1)
    x = rnd(g, 2, 17, 256, dtype=BF16)
    w, b = rnd(g, 256, dtype=wt), rnd(g, 256, dtype=wt)
    for ww, bb in ((w, b), (w, None), (None, b), (None, None)):
        check_ln(x, ww, bb, F32)


@pytest.mark.parametrize("D,pad", [(1024, 8), (1024, 3), (333, 1), (40, 24)])
def test_layer_norm_strided_rows_and_untouched_padding(D, pad):
    g = gen(2)
    x, _ = strided(rnd(g, 11, D, dtype=BF16), pad)
    w, b = rnd(g, D), rnd(g, D)
    check_ln(x, w, b, BF16)
    # rows on other boundaries may be summed in another order, so not the same bits as contiguous
    # ones: the same bound against the definition
    out, big = strided(torch.zeros(11, D, dtype=BF16, device="cuda"), pad)
    y, _, _ = check_ln(x, w, b, BF16, out=out)
    assert y.data_ptr() == out.data_ptr()
    assert big[:, D:].isnan().all()


def test_layer_norm_views():
    g = gen(3)
    t = rnd(g, 4, 9, 128, dtype=F16)
    w = rnd(g, 128)
    assert torch.equal(sc.layer_norm(t[:, 0], w)[0], sc.layer_norm(t[:, 0].contiguous(), w)[0])
    assert torch.equal(sc.layer_norm(t[1], w)[0], sc.layer_norm(t, w)[0][1])
    one = t[0, 0]
    assert torch.equal(sc.layer_norm(one, w)[0], sc.layer_norm(t, w)[0][0, 0])
    for bad in (t[:, 1:], t.transpose(1, 2), t[:1, :1].expand(4, 9, 128), t[..., ::2]):
        with pytest.raises(ValueError):
            sc.layer_norm(bad, None)
    y = t.clone()
    sc.layer_norm(y, w, out=y)  # in place
    assert torch.equal(y, sc.layer_norm(t, w)[0])


def test_layer_norm_rows_are_independent_of_nonfinite_ones():
    g = gen(4)
    for D in (64, 1000, 5000, 20001):
        x = rnd(g, 6, D)
        clean = sc.layer_norm(x)[0]
        x[1, D // 2] = float("nan")
        x[3, 0] = float("inf")
        y = sc.layer_norm(x)[0]
        assert y[1].isnan().all() and y[3].isnan().all()
        for r in (0, 2, 4, 5):
            assert torch.equal(y[r], clean[r])


def test_layer_norm_extremes():
    x = torch.full((3, 64), 5.0, device="cuda")
    y, mean, rstd = sc.layer_norm(x, eps=1e-6, want_stats=True)
    assert (y == 0).all() and (mean == 5).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=4 * U)
    assert sc.layer_norm(x, eps=0.0)[0].isnan().all()
    # a mean far above the spread: the variance is taken about the mean
    g = gen(5)
    big = 4096 + rnd(g, 4, 1024)
    check_ln(big, None, None, F32)
    e = torch.empty(0, 64, device="cuda")
    y, m, r = sc.layer_norm(e, want_stats=True)
    assert y.shape == (0, 64) and m.shape == (0,)


def lnb_ref(dy, x, mean, rstd, w, add):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[..., None], rstd.double()[..., None]
    hh = (x - mean) * rstd
    gg = dy * w.double() if w is not None else dy
    dx = rstd * (gg - gg.mean(-1, keepdim=True) - hh * (gg * hh).mean(-1, keepdim=True))
    lim = rstd * (gg.abs() + gg.abs().mean(-1, keepdim=True) + hh.abs() * (gg * hh).abs().mean(-1, keepdim=True))
    if add is not None:
        dx = dx + add.double()
        lim = lim + add.double().abs()
    f = lambda t: t.reshape(-1, t.shape[-1])
    return dx, lim, f(dy * hh).sum(0), f(dy * hh).abs().sum(0), f(dy).sum(0), f(dy).abs().sum(0)


def check_lnb(dy, x, mean, rstd, w, add, **kw):
    dx, dw, db = sc.layer_norm_backward(dy, x, mean, rstd, w, dx_add=add, **kw)
    rx, lx, rw, lw, rb, lb = lnb_ref(dy, x, mean, rstd, w, add)
    D, rows = x.shape[-1], x.numel() // x.shape[-1]
    close(dx, rx, (ln_depth(D) + 4) * U * lx, "dx")
    if dw is not None:
        # at most rows / 8 rows in one thread, then 64 partial sums and roundings
        d = 64 + rows / 8
        close(dw, rw, d * U * lw, "dw")
        close(db, rb, d * U * lb, "db")
    return dx, dw, db


@pytest.mark.parametrize("xt,yt", PAIRS)
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 64), (257, 1024), (33, 997), (2000, 200), (6, 4096),
                                    (5, 4100), (600, 1536), (3, 8192), (2, 16384), (21, 20000), (2, 16391)])
def test_layer_norm_backward(rows, D, xt, yt):
    g = gen(rows * 31 + D)
    x = rnd(g, rows, D, dtype=xt, scale=2.0) + 1
    w = 1 + rnd(g, D, scale=0.2)
    dy = rnd(g, rows, D, dtype=yt)
    _, mean, rstd = sc.layer_norm(x, w, want_stats=True)
    check_lnb(dy, x, mean, rstd, w, None)
    check_lnb(dy, x, mean, rstd, w, rnd(g, rows, D, dtype=xt))


def test_layer_norm_backward_options():
    g = gen(6)
    x, dy = rnd(g, 40, 384, dtype=BF16), rnd(g, 40, 384, dtype=BF16)
    w = rnd(g, 384, dtype=BF16)
    _, mean, rstd = sc.layer_norm(x, w, want_stats=True)
    dx, dw, db = check_lnb(dy, x, mean, rstd, w, None)
    assert dw.dtype == BF16
    one = sc.layer_norm_backward(dy, x, mean, rstd, w, want_params=False)
    assert torch.equal(one[0], dx) and one[1] is None and one[2] is None
    two = sc.layer_norm_backward(dy, x, mean, rstd, w, want_dx=False)
    assert two[0] is None and torch.equal(two[1], dw) and torch.equal(two[2], db)
    assert sc.layer_norm_backward(dy, x, mean, rstd)[1] is None
    _, dw32, _ = check_lnb(dy, x, mean, rstd, None, None, want_params=True)
    assert dw32.dtype == F32
    xs, _ = strided(x, 5)
    dys, _ = strided(dy, 3)
    assert torch.equal(sc.layer_norm_backward(dys, xs, mean, rstd, w)[0].float().isfinite(), dx.isfinite())
    check_lnb(dys, xs, mean, rstd, w, xs)
    e = torch.empty(0, 384, dtype=BF16, device="cuda")
    z = torch.empty(0, device="cuda")
    dx, dw, db = sc.layer_norm_backward(e, e, z, z, w)
    assert dx.shape == (0, 384) and (dw == 0).all() and (db == 0).all()
    with pytest.raises(L.ScError):
        sc.layer_norm_backward(dy, x, mean, rstd, w, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_layer_norm_backward_same_bits():
    g = gen(7)
    x, dy = rnd(g, 1500, 768), rnd(g, 1500, 768)
    w = rnd(g, 768)
    _, mean, rstd = sc.layer_norm(x, w, want_stats=True)
    a = sc.layer_norm_backward(dy, x, mean, rstd, w)
    for _ in range(3):
        b = sc.layer_norm_backward(dy, x, mean, rstd, w)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_layer_norm_gradients_against_differences():
    """Central differences of sum(y * G) along a random direction, h = 2^-7: the outputs
    (|y| < 8, off by 2^-18 at most) contribute 2^-18 sum|G| / 2h as a worst case, 1e-3 of
    sum|G| |dir| as a bound here; curvature h^2 / 6 with third derivatives below 8."""
    g = gen(8)
    x, w, b, G = rnd(g, 8, 96), 1 + rnd(g, 96, scale=0.1), rnd(g, 96), rnd(g, 8, 96)
    _, mean, rstd = sc.layer_norm(x, w, b, want_stats=True)
    dx, dw, db = sc.layer_norm_backward(G, x, mean, rstd, w)
    f = lambda x, w, b: (sc.layer_norm(x, w, b)[0].double() * G.double()).sum().item()
    e = 2.0 ** -7
    for k, (t, grad) in enumerate(((x, dx), (w, dw), (b, db))):
        v = rnd(g, *t.shape)
        args = [x, w, b]
        hi, lo = list(args), list(args)
        hi[k], lo[k] = t + e * v, t - e * v
        num = (f(*hi) - f(*lo)) / (2 * e)
        ana = (grad.double() * v.double()).sum().item()
        lim = (2.0 ** -18 / (2 * e) + 8 * e * e / 6) * (G.abs().double().sum().item())
        assert abs(num - ana) <= lim, (k, num, ana, lim)


@pytest.mark.parametrize("D", [64, 1000, 4096, 8200, 20000])
@pytest.mark.parametrize("wt", [F32, BF16])
def test_layer_norm_params_off_their_boundary(D, wt):
    g = gen(9)
    x, dy = rnd(g, 5, D), rnd(g, 5, D)
    w, b = rnd(g, D + 1, dtype=wt)[1:], rnd(g, D + 3, dtype=wt)[3:]
    _, mean, rstd = check_ln(x, w, b, F32)
    check_lnb(dy, x, mean, rstd, w, None)


@pytest.mark.parametrize("xt,yt", [(BF16, F32), (F32, F32), (F16, F16)])
@pytest.mark.parametrize("D,pads", [(331, (0, 2, 4, 6)), (331, (0, 1, 0, 2)), (512, (1, 3, 5, 7)), (1023, (0, 0, 2, 2))])
def test_layer_norm_odd_strides(D, pads, xt, yt):
    """Strides of one parity (accesses of two elements) and of both (one element)."""
    g = gen(10)
    px, py, pa, po = pads
    x, _ = strided(rnd(g, 61, D, dtype=xt), px)
    dy, _ = strided(rnd(g, 61, D, dtype=yt), py)
    add, _ = strided(rnd(g, 61, D, dtype=xt), pa)
    out, big = strided(torch.zeros(61, D, dtype=yt, device="cuda"), po)
    w, b = 1 + rnd(g, D, scale=0.2), rnd(g, D)
    _, mean, rstd = check_ln(x, w, b, yt, out=out)
    assert big[:, D:].isnan().all()
    check_lnb(dy, x, mean, rstd, w, add)
    off = torch.zeros(61 * D + 1, dtype=xt, device="cuda")[1:].view(61, D).copy_(x)
    check_ln(off, w, b, yt)
    check_lnb(dy, off, mean, rstd, w, off)


def test_offsets_beyond_32_bits():
    """Rows that start more than 2^31 elements into their buffer."""
    g = gen(35)
    rows, ld = 70000, 32768
    big = torch.empty(rows, ld, dtype=BF16, device="cuda")
    x = big[:, :72]
    x.copy_(rnd(g, rows, 72, dtype=BF16))
    w = rnd(g, 72)
    tail = x[-300:].contiguous()
    y, mean, rstd = sc.layer_norm(x, w, want_stats=True)
    assert torch.equal(y[-300:], sc.layer_norm(tail, w)[0])
    out = big[:, 16384:16384 + 72]
    sc.layer_norm(x, w, out=out)
    assert torch.equal(out, y)
    dx, _, _ = sc.layer_norm_backward(out, x, mean, rstd, w)
    assert torch.equal(dx[-300:], sc.layer_norm_backward(y[-300:], tail, mean[-300:], rstd[-300:], w)[0])
    wl = rnd(g, 40, 72, dtype=BF16, scale=0.1)
    sc.linear(x, wl, out=big[:, 8192:8192 + 40])
    assert torch.equal(big[-300:, 8192:8192 + 40], sc.linear(tail, wl)[0])
    dl = big[:, 8192:8192 + 40]
    dx, dw, _ = sc.linear_backward(dl, x, wl, grad_dtype=F32)
    assert torch.equal(dx[-300:], sc.linear_backward(dl[-300:].contiguous(), tail, wl)[0])
    ref = dl.double().t() @ x.double()
    close(dw, ref, (rows + 16) * U * (dl.double().abs().t() @ x.double().abs()), "dw")


# ---- linear ----------------------------------------------------------------------------
def phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2))


def act_ref(z, act):
    c = math.sqrt(2 / math.pi)
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "gelu": lambda: z * phi(z),
            "gelu_tanh": lambda: z * torch.sigmoid(2 * c * (z + 0.044715 * z ** 3)),
            "silu": lambda: z * torch.sigmoid(z)}[act]()


def act_grad_ref(z, act):
    z = z.detach().clone().requires_grad_(True)
    act_ref(z, act).sum().backward()
    return z.grad


def terms(t):
    """Error of one product: exact for 16-bit operands; fp32 operands leave out three of nine
    partial products, 2 * 2^-24 |x w| and less, and round nothing else."""
    return 4 if t == F32 else 0


def check_linear(x, w, bias=None, res=None, act="none", out_dtype=None, want_pre=False, **kw):
    out, pre = sc.linear(x, w, bias, res, act, out_dtype=out_dtype, want_pre=want_pre, **kw)
    xd, wd = x.double(), w.double()
    K = x.shape[-1]
    z = xd @ wd.t()
    mag = xd.abs() @ wd.abs().t()
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    ez = (K + 16 + terms(x.dtype)) * U * mag
    assert (pre is not None) == want_pre
    if want_pre:
        close(pre, z, ez, "pre")
    ref = act_ref(z, act)
    # |act'| < 1.2; the activation itself is off by 16 u |z| at most
    lim = 1.2 * ez + (16 * U * z.abs() if act not in ("none", "relu") else 0)
    if res is not None:
        ref = ref + res.double()
        lim = lim + U * ref.abs()
    close(out, ref, lim, f"out {act}")
    return out, pre


LIN_TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)]
SHAPES = [(1, 1, 1), (1, 1000, 1024), (3, 5, 7), (16, 1000, 384), (17, 64, 64), (128, 128, 64), (129, 257, 72),
          (257, 384, 1024), (300, 130, 1000), (64, 1024, 4096), (513, 520, 33), (1000, 16, 16)]


@pytest.mark.parametrize("t,ot", LIN_TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, t, ot):
    g = gen(M * 131 + N * 17 + K)
    x, w = rnd(g, M, K, dtype=t), rnd(g, N, K, dtype=t, scale=K ** -0.5)
    check_linear(x, w, out_dtype=ot)
    check_linear(x, w, rnd(g, N), rnd(g, M, N, dtype=ot), "gelu", ot, want_pre=True)


@pytest.mark.parametrize("t,ot", LIN_TYPES)
@pytest.mark.parametrize("M,N,K", [(700, 1536, 512), (2100, 768, 256), (4112, 512, 264), (4112, 1600, 136),
                                   (2600, 2051, 1250)])
def test_linear_many_tiles(M, N, K, t, ot):
    g = gen(M + N + K)
    x, w = rnd(g, M, K, dtype=t), rnd(g, N, K, dtype=t, scale=K ** -0.5)
    check_linear(x, w, rnd(g, N, dtype=t), rnd(g, M, N, dtype=ot), "none", ot)


@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_activations(act, t):
    g = gen(11)
    x, w = rnd(g, 77, 160, dtype=t, scale=3), rnd(g, 96, 160, dtype=t, scale=0.1)
    for bias in (None, rnd(g, 96), rnd(g, 96, dtype=BF16), rnd(g, 96, dtype=F16)):
        check_linear(x, w, bias, None, act, F32, want_pre=True)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N,K,t,ot", [(4112, 1600, 1100, BF16, F32), (4112, 1601, 200, F16, F16),
                                        (4112, 1603, 1100, F16, F32), (1300, 1290, 90, BF16, BF16)])
def test_linear_activations_of_many_tiles(M, N, K, t, ot, act):
    g = gen(15)
    x, w = rnd(g, M, K, dtype=t), rnd(g, N, K, dtype=t, scale=2 * K ** -0.5)
    check_linear(x, w, rnd(g, N), rnd(g, M, N, dtype=ot), act, ot, want_pre=True)


@pytest.mark.parametrize("t,ot", [(BF16, BF16), (F16, F32)])
def test_linear_rows_on_different_boundaries(t, ot):
    """Results, residuals and pre-activations whose rows begin on other boundaries than each
    other's, and a residual that is the result."""
    g = gen(16)
    M, N, K = 700, 333, 96
    x, w = rnd(g, M, K, dtype=t), rnd(g, N, K, dtype=t, scale=0.1)
    b = rnd(g, N + 1, dtype=t)[1:]
    for po, pr in ((0, 0), (1, 0), (3, 8), (19, 2)):
        res, _ = strided(rnd(g, M, N, dtype=ot), pr)
        out, big = strided(torch.zeros(M, N, dtype=ot, device="cuda"), po)
        a, _ = check_linear(x, w, b, res, "gelu", ot, want_pre=True, out=out)
        assert big[:, N:].isnan().all()
        keep, _ = strided(res, po)
        sc.linear(x, w, b, keep, "gelu", out_dtype=ot, out=keep)
        assert torch.equal(keep, a)


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("pad", [1, 8])
def test_linear_strided_and_untouched_padding(t, pad):
    g = gen(12)
    M, N, K = 150, 200, 136
    x, _ = strided(rnd(g, M, K, dtype=t), pad)
    w, _ = strided(rnd(g, N, K, dtype=t), pad)
    res, _ = strided(rnd(g, M, N, dtype=t), pad)
    out, big = strided(torch.zeros(M, N, dtype=t, device="cuda"), pad)
    check_linear(x, w, None, res, "gelu", out=out)
    assert big[:, N:].isnan().all()
    a = sc.linear(x, w, None, res, "gelu")[0]
    keep = res.contiguous()
    sc.linear(x, w, None, keep, "gelu", out=keep)  # the residual's own memory
    assert torch.equal(keep, a)
    m = torch.randn(M * K + 1, device="cuda", generator=g).to(t)[1:].view(M, K)  # rows off their boundary
    check_linear(m, w, None, None, "none")


def test_linear_views_and_refusals():
    g = gen(13)
    t, w = rnd(g, 4, 9, 64, dtype=BF16), rnd(g, 24, 64, dtype=BF16)
    full = sc.linear(t, w)[0]
    assert full.shape == (4, 9, 24)
    assert torch.equal(sc.linear(t[:, 0], w)[0], sc.linear(t[:, 0].contiguous(), w)[0])
    assert sc.linear(t[0, 0], w)[0].shape == (24,)
    assert sc.linear(t[:0], w)[0].shape == (0, 9, 24)
    assert sc.linear(t, w[:0])[0].shape == (4, 9, 0)
    bad = [dict(x=t.transpose(1, 2)), dict(w=w.half()), dict(w=w[:, :32]), dict(bias=w[0, :23]), dict(act="tanh"),
           dict(residual=full.float()), dict(residual=full[:2]), dict(out_dtype=F16), dict(out_dtype=torch.float64),
           dict(x=t.double()), dict(residual=full[:1].expand(4, 9, 24)), dict(out=full[..., :12])]
    for kw in bad:
        a = {**dict(x=t, w=w), **kw}
        with pytest.raises((ValueError, L.ScError)):
            sc.linear(a.pop("x"), a.pop("w"), **a)


def test_linear_nonfinite_values_stay_in_their_rows_and_columns():
    g = gen(14)
    for t in (BF16, F32):
        x, w = rnd(g, 200, 96, dtype=t), rnd(g, 140, 96, dtype=t)
        clean = sc.linear(x, w)[0]
        x[5, 3] = float("nan")
        x[150, 95] = float("inf")
        w[139, 0] = float("-inf")
        y = sc.linear(x, w)[0]
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[[5, 150]] = True
        hit[:, 139] = True
        assert not y[hit].isfinite().any()
        assert torch.equal(y[~hit], clean[~hit])


def test_linear_f32_range():
    """The three parts of an fp32 operand keep its range: the largest and very small values."""
    big = torch.finfo(F32).max
    x = torch.tensor([[big, 1.0, 0.0], [-big, 0.0, 1.0], [2.0 ** -100, 0.0, 0.0]], device="cuda")
    w = torch.tensor([[0.5, 0.0, 0.0], [0.0, 3.0, 1 + 2.0 ** -23]], device="cuda")
    y = sc.linear(x, w)[0]
    ref = x.double() @ w.double().t()
    assert torch.all((y.double() - ref).abs() <= 8 * U * ref.abs()), (y, ref)


def check_linear_backward(dout, x, w, pre=None, act="none", **kw):
    dx, dw, db = sc.linear_backward(dout, x, w, pre, act, **kw)
    t, M, N = x.dtype, x.shape[0], w.shape[0]
    do, xd, wd = dout.double(), x.double(), w.double()
    dz = do if act == "none" else do * act_grad_ref(pre.double(), act)
    # act' (below 1.2, made of values below 8) off by 16 u; dz rounded to its type
    ez = (0 if act in ("none", "relu") else 16 * U) * do.abs() + h(t) * dz.abs() + tiny(t)
    if act == "none" and dout.dtype == t:
        ez = torch.zeros_like(dz)
    n = terms(t)
    if dx is not None:
        close(dx, dz @ wd, ez @ wd.abs() + (N + 16 + n) * U * ((dz.abs() + ez) @ wd.abs()), "dx")
    if dw is not None:
        close(dw, dz.t() @ xd, ez.t() @ xd.abs() + (M + 16 + n) * U * ((dz.abs() + ez).t() @ xd.abs()), "dw")
    if db is not None:
        # from the unrounded dz: at most M / 8 rows in one thread, then 64 sums and roundings
        close(db, dz.sum(0), (16 * U * do.abs() + (64 + M / 8) * U * dz.abs()).sum(0), "db")
    return dx, dw, db


@pytest.mark.parametrize("t,ot", LIN_TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_backward(M, N, K, t, ot):
    g = gen(M * 131 + N * 17 + K + 1)
    x, w = rnd(g, M, K, dtype=t), rnd(g, N, K, dtype=t, scale=0.05)
    dout, pre = rnd(g, M, N, dtype=ot), rnd(g, M, N, dtype=t)
    check_linear_backward(dout, x, w)
    check_linear_backward(dout, x, w, pre, "gelu", grad_dtype=F32)


@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_backward_activations(act, t):
    g = gen(21)
    x, w = rnd(g, 300, 160, dtype=t), rnd(g, 96, 160, dtype=t, scale=0.1)
    dout, pre = rnd(g, 300, 96, dtype=t), rnd(g, 300, 96, dtype=t, scale=2)
    check_linear_backward(dout, x, w, pre, act)


@pytest.mark.parametrize("t,ot", LIN_TYPES)
@pytest.mark.parametrize("M,N,K", [(2056, 1536, 768), (2313, 2304, 2050)])
def test_linear_backward_many_tiles(M, N, K, t, ot):
    g = gen(22)
    x, w = rnd(g, M, K, dtype=t), rnd(g, N, K, dtype=t, scale=0.05)
    check_linear_backward(rnd(g, M, N, dtype=ot), x, w, rnd(g, M, N, dtype=t), "gelu_tanh")


@pytest.mark.parametrize("gt", [BF16, F16, F32])
@pytest.mark.parametrize("M,N,K", [(1300, 3000, 2300), (1300, 1300, 1300), (4300, 130, 70), (65, 520, 1030), (1, 64, 64)])
def test_linear_backward_f32_operands(M, N, K, gt):
    """The parts' two accumulators: over several tiles, tiles of either width, shared contractions;
    weight gradients of 16 bits too."""
    g = gen(25)
    x, w = rnd(g, M, K, dtype=F32), rnd(g, N, K, dtype=F32, scale=0.05)
    check_linear(x, w, rnd(g, N, dtype=F32))
    check_linear_backward(rnd(g, M, N, dtype=F32), x, w, grad_dtype=gt)


def test_linear_backward_options():
    g = gen(23)
    x, w = rnd(g, 130, 72, dtype=BF16), rnd(g, 88, 72, dtype=BF16)
    dout, pre = rnd(g, 130, 88, dtype=BF16), rnd(g, 130, 88, dtype=BF16)
    full = check_linear_backward(dout, x, w, pre, "silu")
    for k, name in enumerate(("want_dx", "want_dw", "want_db")):
        part = sc.linear_backward(dout, x, w, pre, "silu", **{n: n == name for n in ("want_dx", "want_dw", "want_db")})
        assert all((p is None) if i != k else torch.equal(p, full[k]) for i, p in enumerate(part))
    xs, ws, ds, ps = (strided(t, 3)[0] for t in (x, w, dout, pre))
    check_linear_backward(ds, xs, ws, ps, "silu")
    xs, ws, ds, ps = (strided(t, 8)[0] for t in (x, w, dout, pre))
    check_linear_backward(ds, xs, ws, ps, "none")
    dx, dw, db = sc.linear_backward(dout[:0], x[:0], w, pre[:0], "silu")
    assert dx.shape == (0, 72) and (dw == 0).all() and (db == 0).all()
    dx, dw, db = sc.linear_backward(dout[:, :0].contiguous(), x, w[:0])
    assert (dx == 0).all() and dw.shape == (0, 72) and db.shape == (0,)
    for bad in (dict(pre=None), dict(pre=pre.float()), dict(dout=dout[:64]), dict(dout=dout.half()),
                dict(dout=dout[:1].expand(130, 88)), dict(grad_dtype=torch.float64),
                dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        a = {**dict(dout=dout, pre=pre), **bad}
        with pytest.raises((ValueError, L.ScError)):
            sc.linear_backward(a.pop("dout"), x, w, a.pop("pre"), "silu", **a)


def test_linear_gradients_against_differences():
    """Central differences of sum(out * G) with fp32 operands, h = 2^-6: outputs below 32 are off
    by 2^-14 at most (bound above), so 2^-14 / 2h of sum|G|; curvature h^2 / 6 of the third
    derivative along a unit-scale direction, below 2 for silu."""
    g = gen(24)
    x, w, b, G = rnd(g, 24, 40), rnd(g, 16, 40, scale=0.15), rnd(g, 16), rnd(g, 24, 16)
    _, pre = sc.linear(x, w, b, None, "silu", want_pre=True)
    dx, dw, db = sc.linear_backward(G, x, w, pre, "silu")
    f = lambda x, w, b: (sc.linear(x, w, b, None, "silu")[0].double() * G.double()).sum().item()
    e = 2.0 ** -6
    for k, (t, grad) in enumerate(((x, dx), (w, dw), (b, db))):
        v = rnd(g, *t.shape, scale=0.2)
        hi, lo = [x, w, b], [x, w, b]
        hi[k], lo[k] = t + e * v, t - e * v
        num = (f(*hi) - f(*lo)) / (2 * e)
        ana = (grad.double() * v.double()).sum().item()
        lim = (2.0 ** -14 / (2 * e) + 2 * e * e / 6) * G.abs().double().sum().item()
        assert abs(num - ana) <= lim, (k, num, ana, lim)


# ---- together, streams, graphs ----------------------------------------------------------
def mlp(x, p, stream=None):
    """A pre-norm MLP block and its gradients for dout = x0 + 1: every output."""
    kw = dict(stream=stream)
    y, mean, rstd = sc.layer_norm(x, p["lw"], p["lb"], want_stats=True, out_dtype=BF16, **kw)
    a, pre = sc.linear(y, p["w1"], p["b1"], None, "gelu", want_pre=True, **kw)
    out, _ = sc.linear(a, p["w2"], p["b2"], x, out_dtype=F32, **kw)
    da, dw2, db2 = sc.linear_backward(p["g"], a, p["w2"], **kw)
    dy, dw1, db1 = sc.linear_backward(da, y, p["w1"], pre, "gelu", **kw)
    dx, dlw, dlb = sc.layer_norm_backward(dy, x, mean, rstd, p["lw"], dx_add=p["g"], **kw)
    return out, dx, dlw, dlb, dw1, db1, dw2, db2


def mlp_case(seed, rows=300):
    g = gen(seed)
    D, H = 192, 768
    p = {"lw": 1 + rnd(g, D, scale=0.1), "lb": rnd(g, D, scale=0.1), "w1": rnd(g, H, D, dtype=BF16, scale=0.05),
         "b1": rnd(g, H, scale=0.1), "w2": rnd(g, D, H, dtype=BF16, scale=0.03), "b2": rnd(g, D, scale=0.1),
         "g": rnd(g, rows, D)}
    return rnd(g, rows, D), p


def test_block_and_its_gradients():
    """An MLP block in the framework's layers against torch autograd in 64 bits.  Each bf16
    rounding on the way (y, a, pre and their gradients: at most 6 in a chain, 2^-8 relative to
    the largest values that meet) moves an output by less than 6 * 2^-8 of its tensor's
    largest magnitude."""
    x, p = mlp_case(31)
    got = mlp(x, p)
    q = {k: v.double().requires_grad_(True) for k, v in p.items() if k != "g"}
    xd = x.double().requires_grad_(True)
    y = torch.nn.functional.layer_norm(xd, (192,), q["lw"], q["lb"], 1e-6)
    a = torch.nn.functional.gelu(y @ q["w1"].t() + q["b1"])
    out = xd + a @ q["w2"].t() + q["b2"]
    out.backward(p["g"].double())
    refs = [out.detach(), xd.grad] + [q[k].grad for k in ("lw", "lb", "w1", "b1", "w2", "b2")]
    for name, a, r in zip("out dx dlw dlb dw1 db1 dw2 db2".split(), got, refs):
        assert (a.double() - r).abs().max() <= 6 * 2.0 ** -8 * r.abs().max(), name


def test_norm_feeds_the_quantiser():
    g = gen(32)
    x = rnd(g, 2, 65, 256, dtype=BF16)
    y = sc.layer_norm(x, rnd(g, 256), None, out_dtype=F32)[0]
    lv, s, _ = sc.quantize(y, axis=0)
    back = (lv.float() - 128) * s[..., None]
    assert ((back - y).abs() <= 0.5001 * s[..., None]).all()


def test_first_call_inside_a_capture():
    """A fresh process whose first calls of every layer are captured."""
    code = """
import sys, torch
sys.path.insert(0, %r)
from mixed_precision_vit_b200 import sc
x = torch.randn(300, 72, device="cuda").bfloat16()
w = torch.randn(40, 72, device="cuda").bfloat16()
f = torch.randn(5, 64, device="cuda")
lw = torch.randn(72, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
def calls():
    y, m, r = sc.layer_norm(x, lw, want_stats=True)
    o, pre = sc.linear(y, w, None, None, "gelu", want_pre=True)
    dx, dw, db = sc.linear_backward(o, y, w, pre, "gelu")
    return (y, o, dx, dw, db, *sc.layer_norm_backward(dx, x, m, r, lw), sc.linear(f, f)[0])
with torch.cuda.graph(g):
    held = calls()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(held, calls()))
print("captured")
""" % ROOT
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_graphs_replayed_in_turn():
    x, p = mlp_case(36, rows=520)
    graphs, held = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(mlp(x, p))
        graphs.append(g)
    ref = mlp(x, p)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for h in held:
        assert all(torch.equal(a, b) for a, b in zip(h, ref))


def test_streams_and_graphs():
    x, p = mlp_case(33)
    ref = mlp(x, p)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in (s1, s2):  # two streams at once
        outs.append(mlp(x, p, stream=s))
    with torch.cuda.stream(s1):
        outs.append(mlp(x, p))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = mlp(x, p)
    x2, _ = mlp_case(34)
    x.copy_(x2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, mlp(x2, p)))
