"""Layer norm of rows that vary little about a large mean."""
import pytest
import torch

from mixed_precision_vit_b200 import sc
from test_gpu_layers import BF16, F16, F32, U, close, gen, ln_depth, rnd

pytestmark = pytest.mark.gpu
# widths of every kernel: one warp and whole blocks per row, rows on no boundary, rows too wide for registers
WIDTHS = [1, 64, 200, 768, 997, 1000, 1024, 4096, 5001, 16384, 20000, 16391]


@pytest.mark.parametrize("t", [F32, BF16, F16])
@pytest.mark.parametrize("D", WIDTHS)
def test_constant_rows(D, t):
    """Their variance is 0: the bias with an eps, 0 / 0 without."""
    c = torch.tensor([5.0, 0.1, 1000.1, -3.7e4, 1 / 3, 1e-3, 59999.0, 0.0], device="cuda").to(t)
    x = c[:, None].expand(-1, D).contiguous()
    b = rnd(gen(81), D)
    y, mean, rstd = sc.layer_norm(x, None, b, 1e-6, out_dtype=F32, want_stats=True)
    assert torch.equal(y, b.expand_as(y)) and torch.equal(mean, c.float())
    assert ((rstd - 1e3).abs() <= 4 * U * 1e3).all()
    assert sc.layer_norm(x, None, b, 0.0)[0].isnan().all()


@pytest.mark.parametrize("mean", [100.0, -1000.0, 30000.0])
@pytest.mark.parametrize("D", [w for w in WIDTHS if w > 1])
def test_rows_about_a_large_mean(D, mean):
    """c = x - m is exact, so y sees the roundings of sums of c, not of x: d u mean|c| in the
    rest of the mean, d u relative in r (and the rest squared, below (d u |mean| r)^2 of it), a few
    of the result itself."""
    g = gen(82)
    x = mean + rnd(g, 9, D)
    w, b = 1 + rnd(g, D, scale=0.2), rnd(g, D)
    xd = x.double()
    m = xd.mean(-1, keepdim=True)
    c = xd - m
    r = (c.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
    ref = c * r * w.double() + b.double()
    d = ln_depth(D) + 8
    lost = d * U + (d * U * abs(mean) * r) ** 2 * d * U
    y, mu, rstd = sc.layer_norm(x, w, b, 1e-6, want_stats=True)
    close(y, ref, w.double().abs() * r * (c.abs() + c.abs().mean(-1, keepdim=True)) * (lost + 4 * U) + 2 * U * b.double().abs())
    close(mu, m[:, 0], d * U * c.abs().mean(-1))
    close(rstd, r[:, 0], (lost * r)[:, 0])


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("D", [64, 997, 4096, 20000, 16391])
def test_statistics_of_nonfinite_rows(D, t):
    x = rnd(gen(83), 5, D, dtype=t)
    clean = sc.layer_norm(x, want_stats=True)
    x[1, D // 2], x[3, 0] = float("nan"), float("-inf")
    got = sc.layer_norm(x, want_stats=True)
    for a, b in zip(got, clean):
        assert torch.equal(a[[0, 2, 4]], b[[0, 2, 4]])
    assert got[0][[1, 3]].isnan().all() and got[2][[1, 3]].isnan().all()
    assert got[1][1].isnan() and got[1][3] == float("-inf")
