"""Accuracy of the floating-point layers where elementwise bounds on random sums are too
wide to see it: activations' tails, exact sums, long sums of one sign.

u = 2^-24 is half a step of fp32, h(t) half a step of a type; every tolerance is the sum of
the roundings on the way, derived beside it."""
import math

import pytest
import torch

from mixed_precision_vit_b200 import sc
from test_gpu_layers import BF16, F16, F32, U, check_linear, close, gen, phi, rnd

pytestmark = pytest.mark.gpu


# ---- activations -----------------------------------------------------------------------
def on_values(z, act, out_dtype=None):
    """act(z) of a vector by a layer with one input and the weight 1: z reaches the activation
    exactly (one product, nothing to round)."""
    one = torch.ones(1, 1, dtype=z.dtype, device=z.device)
    return sc.linear(z[:, None], one, None, None, act, out_dtype=out_dtype)[0][:, 0]


def gelu_tail_bound(z):
    """gelu(z) = z exp(-z^2 / 2) Q, relative to itself: the exponent is rounded three times
    (3 u z^2 log2(e) / 2 of it, times ln 2), ex2 and rcp are off by 4 u and 2 u, Q moves by its
    argument's relative error at most 3.2-fold, 7 steps of a polynomial with falling weights
    round below 8 u, its fit is off by 16 u, and two products round."""
    return (1.5 * z * z + 4 + 3.2 * 2 + 8 + 16 + 2) * U


@pytest.mark.parametrize("t,ot", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
def test_gelu_keeps_its_lower_tail(t, ot):
    z = torch.linspace(-12.5, 0, 40001, device="cuda").to(t)
    y = on_values(z, "gelu", ot)
    zd = z.double()
    ref = zd * phi(zd)
    close(y, ref, gelu_tail_bound(zd) * ref.abs(), "gelu")


@pytest.mark.parametrize("t", [F32, BF16, F16])
def test_gelu_gradient_keeps_its_lower_tail(t):
    """dbias of one row is dz itself, in fp32: dout gelu'(z) with dout = 1."""
    z = torch.linspace(-12.5, 0, 40001, device="cuda").to(t)
    one = torch.ones(1, z.numel(), dtype=t, device="cuda")
    x, w = torch.ones(1, 8, dtype=t, device="cuda"), torch.ones(z.numel(), 8, dtype=t, device="cuda")
    db = sc.linear_backward(one, x, w, z[None], "gelu", want_dx=False, want_dw=False, grad_dtype=F32)[2]
    zd = z.double()
    p, d = phi(zd), zd * torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    close(db, p + d, gelu_tail_bound(zd) * (p + d.abs()), "gelu'")


def test_gelu_over_the_whole_range():
    """Off by 16 u |z| at most in Phi's 1 - q, and right at both ends.  (An infinity comes as a
    bias: an infinite fp32 operand is an infinity times the other's zero parts, a NaN.)"""
    ends = torch.tensor([-3e38, 3e38, 1e20, -1e20, 0.0], device="cuda")
    z = torch.cat([torch.linspace(-20, 20, 60001, device="cuda"), ends])
    y = on_values(z, "gelu")
    zd = z.double()
    assert torch.equal(y[-5:], torch.tensor([0.0, 3e38, 1e20, 0.0, 0.0], device="cuda"))
    close(y, zd * phi(zd), 16 * U * zd.abs(), "gelu")
    one = torch.ones(1, 1, device="cuda")
    assert on_values(torch.tensor([float("nan")], device="cuda"), "gelu").isnan().all()
    assert sc.linear(one, one, torch.full((1,), math.inf, device="cuda"), None, "gelu")[0].item() == math.inf


@pytest.mark.parametrize("t", [F32, BF16, F16])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_gradients_of_saturated_activations(act, t):
    """Far from 0 the derivative is 0 or 1, also where a pre-activation was kept as an infinity
    (fp16 from 65520 on)."""
    top = torch.finfo(t).max
    z = torch.tensor([200.0, 6e4, top, math.inf, -200.0, -6e4, -top, -math.inf, 1e20, -1e20, math.nan], device="cuda").to(t)
    one = torch.ones(1, z.numel(), dtype=t, device="cuda")
    x, w = torch.ones(1, 8, dtype=t, device="cuda"), torch.ones(z.numel(), 8, dtype=t, device="cuda")
    db = sc.linear_backward(one, x, w, z[None], act, want_dx=False, want_dw=False, grad_dtype=F32)[2]
    assert torch.equal(db[:-1], (z[:-1] > 0).float()) and db[-1].isnan()


# ---- long sums -------------------------------------------------------------------------
def pos(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g).abs_() * scale).to(dtype)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("N,K", [(2048, 1024), (4096, 1024)])
def test_long_sums_of_16_bit_results_do_not_drift(N, K, t):
    """A weight gradient over 262144 rows of one sign, in tiles of either width.  The tensor
    cores cut at every 16 products, below 2^-22 of the sum so far for all of them together:
    (1 + .. + 48) / 48 * 2^-22 < 2^-17.3 in a chunk of 768 or less; 512 chunks add up with
    u (1 + .. + 512) / 512 at most = 2^-16.  In one accumulation the cuts come to about 2^-11."""
    g = gen(51)
    M = 262144
    x, dout = pos(g, M, K, dtype=t), pos(g, M, N, dtype=t, scale=0.25)
    w = torch.zeros(N, K, dtype=t, device="cuda")
    dw = sc.linear_backward(dout, x, w, want_dx=False, want_db=False)[1]
    n, k = slice(0, N, N // 64 + 1), slice(0, K, K // 64 + 1)
    ref = dout[:, n].double().t() @ x[:, k].double()
    close(dw[n, k], ref, (2.0 ** -17.3 + 2.0 ** -16) * ref, "dw")


@pytest.mark.parametrize("gt", [F16, BF16])
def test_long_weight_gradients_of_fp32_operands(gt):
    g = gen(52)
    M, N, K = 20000, 2048, 1024
    x, dout = rnd(g, M, K), rnd(g, M, N, scale=0.05)
    w = torch.zeros(N, K, device="cuda")
    dw = sc.linear_backward(dout, x, w, want_dx=False, want_db=False, grad_dtype=gt)[1]
    ref, mag = dout.double().t() @ x.double(), dout.double().abs().t() @ x.double().abs()
    # chunks of 512 products: 32 cuts, (1 + .. + 32) / 32 * 2^-22; the six products leave 3 u out
    close(dw, ref, (16.5 * 2.0 ** -22 + 20 * U + 4 * U) * mag, "dw")


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,N", [(2100, 1296), (2100, 1291), (4112, 2048)])
def test_long_contractions_with_16_bit_results(M, N, t):
    """Past the longest single accumulation, with every part of the epilogue: aligned and ragged
    rows, both tile widths."""
    g = gen(53)
    K = 16448
    x, w = rnd(g, M, K, dtype=t), rnd(g, N, K, dtype=t, scale=K ** -0.5)
    check_linear(x, w, rnd(g, N), rnd(g, M, N, dtype=t), "gelu", want_pre=True)
    check_linear(x, w)


# tiles of CTA pairs, of single CTAs, and contractions shared by a cluster
KERNELS = [(4112, 1024), (1300, 1290), (257, 384), (1, 40)]


@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("M,N", KERNELS)
def test_long_sums_of_fp32_results_do_not_drift(M, N, t):
    """65536 products of one sign.  As above, at most 2^-22 of the sum so far is cut at every 16
    products: 24.5 * 2^-22 in a chunk of 768, 16.5 * 2^-22 in one of 512, of which there are 126
    (so together below 17 * 2^-22; fp32 operands' left-out products add 4 u); 128
    chunks, or a cluster's parts of them, are added with a u each at most.  In one accumulation
    the cuts come to 2^-13."""
    g = gen(54)
    K = 65536
    x, w = pos(g, M, K, dtype=t), pos(g, N, K, dtype=t)
    y = sc.linear(x, w, out_dtype=F32)[0]
    m, n = slice(0, M, M // 64 + 1), slice(0, N, N // 64 + 1)
    ref = x[m].double() @ w[n].double().t()
    close(y[m, n], ref, (17 * 2.0 ** -22 + (128 + 4 * (t == F32)) * U) * ref, "out")


@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("K,at,steps", [(4096, 0, 12), (4096, 1536, 8), (1024, 0, 8)])
@pytest.mark.parametrize("M,N", KERNELS)
def test_what_one_accumulation_can_lose(M, N, t, K, at, steps):
    """One product of 2^23 makes the accumulator's last place 1; 16 others together are 15/16, which
    a cut drops.  So at most the 64 * 15/256 = 3.75 of every step that shares the large product's
    accumulation are lost: 12 steps at the beginning of a long sum, else 8.  The other
    accumulations are exact, and their sums (45 or 30) too."""
    x, w = torch.full((M, K), 15 / 16, device="cuda"), torch.full((N, K), 1 / 16, device="cuda")
    x[:, at], w[:, at] = 4096, 2048
    y = sc.linear(x.to(t), w.to(t), out_dtype=F32)[0].double()
    lost = 2.0 ** 23 + (K - 1) * 15 / 256 - y
    assert (lost >= -1).all() and (lost <= steps * 3.75 + 1).all(), (lost.min().item(), lost.max().item())


def parts(g, shape, n):
    """fp32 values of n bf16 parts, steps of 2^-9 apart, each -1, 0 or 1 of its step; the leading
    parts of neighbours in the last axis are equal."""
    v = [torch.randint(-1, 2, shape, device="cuda", generator=g).double() * 2.0 ** (-9 * i) for i in range(n)]
    v[0][..., 1::2] = v[0][..., ::2]
    return sum(v).float()


@pytest.mark.parametrize("nx,nw", [(3, 1), (1, 3), (2, 2)])
@pytest.mark.parametrize("M,N", KERNELS)
def test_every_part_of_fp32_operands_counts(M, N, nx, nw):
    """Sums that no rounding touches: the products are multiples of 2^-18; the leading parts' run in
    pairs of opposite signs, so that their sums stay below 2^6, and the others' stay below
    2048 * 2^-8.  Both fit 24 bits together, so the result is exact, unless a part or one of the
    six products is left out."""
    g = gen(55)
    K = 2048
    x, w = parts(g, (M, K), nx), parts(g, (N, K), nw)
    sign = torch.ones(K, device="cuda")
    sign[1::2] = -1
    w = w * sign
    y = sc.linear(x, w)[0]
    assert torch.equal(y.double(), x.double() @ w.double().t())
    # the same sums as an input gradient (w^T in place of w) and as a weight gradient
    dx = sc.linear_backward(x, torch.zeros(M, N, device="cuda"), w.t().contiguous(), want_dw=False, want_db=False)[0]
    assert torch.equal(dx, y)
    dw = sc.linear_backward(x.t().contiguous(), w.t().contiguous(), torch.zeros(M, N, device="cuda"), want_dx=False,
                            want_db=False)[1]
    assert torch.equal(dw, y)
