"""layer_norm_forward of rows whose offset is far larger than their spread, or that have no spread at all, against 64 bits.

Bounds, u = 2^-24, for sums in which a term passes at most A = 64 additions (the forms used here have 8 elements or fewer a thread,
16 where 1024 threads share a row, at most 32 warps and 5 exchanges).  The first mean is off by e0 = (A + 2) u mean|h|.  The differences from it, d,
have u (|d| + e0) each, and their mean, which is added to it, (A + 4) u (mean|d| + e0) = e1: what is left of e0.  The mean
squares lose (A + 8) u (var + e0^2) + 2 e0 e1 + e1^2 and the squares of two such sums as much; the root has half of that relative to
var + eps, counted whole, and 4 u.  An output carries e1, the root's error and four roundings, then one to its type."""
import pytest
import torch

import serving_util as util
import sparse_attention_kv_csa_gb300 as csa

pytestmark = pytest.mark.gpu
U, A = 2.0 ** -24, 64


def check(x, bias, eps, r=None):
    out, total, mean, rstd = csa.layer_norm_forward(x, None, bias, eps, residual=r)
    h = (x if r is None else total).double()
    m = h.mean(1, keepdim=True)
    d = h - m
    var = d.square().mean(1, keepdim=True)
    root = (var + eps).rsqrt()
    want = d * root + bias.double()
    e0 = (A + 2) * U * h.abs().mean(1, keepdim=True)
    e1 = (A + 4) * U * (d.abs().mean(1, keepdim=True) + e0)
    rel = (2 * (A + 8) * U * (var + e0 * e0) + 2 * e0 * e1 + e1 * e1) / (var + eps) + 4 * U
    tol = (e1 + 4 * U * (d.abs() + e0)) * root + d.abs() * root * (rel + 2 * U) + 2 * U * want.abs()
    assert ((mean.double()[:, None] - m).abs() <= e1 + U * m.abs()).all()
    assert ((rstd.double()[:, None] - root).abs() <= rel * root).all()
    half = util.HALF[x.dtype]
    worst = ((out.double() - want).abs() / (tol + half * (want.abs() + tol) + 2.0 ** -40)).max().item()
    assert worst <= 1, worst
    return mean


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim", [3, 96, 1000, 1001, 2000, 4100, 9001])
@pytest.mark.parametrize("n", [1, 40, 4000])
def test_rows_of_one_value(dtype, dim, n):
    # out is the bias, whatever the value, and the mean the value itself
    values = torch.linspace(-2.0, 4.0, n).exp2() * 1000.1
    x = values.to(dtype).cuda()[:, None].expand(n, dim).contiguous()
    bias = torch.linspace(-1e-3, 1e-3, dim).cuda()
    mean = check(x, bias, 1e-5)
    assert torch.equal(mean, x[:, 0].float())


@pytest.mark.parametrize("dim", [96, 1000, 1001, 4100])
@pytest.mark.parametrize("offset", [1e3, -3e4, 1e6])
@pytest.mark.parametrize("residual", [False, True])
def test_small_spreads(dim, offset, residual):
    g = torch.Generator().manual_seed(dim)
    x = (torch.randn((300, dim), generator=g) + offset).cuda()
    r = torch.randn((300, dim), generator=g).cuda() if residual else None
    check(x, torch.zeros(dim, device="cuda"), 1e-5, r)
