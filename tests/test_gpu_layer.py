"""layer_norm forward and backward against 64 bits.

Bounds, u = 2^-24.  The mean sums dim terms (any order): E = (dim + 2) u mean|h|.  The variance sums dim squares of differences from
that mean: (dim + 8) u (var + E^2) + E^2; its root has half of that relative to var + eps, counted whole, and 4 u.  An output carries
the mean's error, the root's and four roundings, then one to its type.  The gradient's two means sum dim products:
(dim + 8) u of the mean of magnitudes; eight roundings on top."""
import pytest
import torch

import serving_util as util
import sparse_attention_kv_csa_gb300 as csa
from sparse_attention_kv_csa_gb300.autograd import layer_norm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def rand(shape, dtype, seed, spread=0.5, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[-1:], generator=g)) + offset
    return x.to(dtype).cuda()


def forward64(x, w, b, eps, r=None, additions=None):
    """(h, y, mean, rstd, bounds on y, mean, rstd).  additions: how many a term of a sum passes at most (any order: dim)."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    hd = h.double()
    dim = hd.shape[1]
    mean = hd.mean(1, keepdim=True)
    d = hd - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    w64 = torch.ones(dim, dtype=torch.float64, device=x.device) if w is None else w.double()
    y = d * rstd * w64 + (0.0 if b is None else b.double())
    additions = dim if additions is None else additions
    e = (additions + 2) * U * hd.abs().mean(1, keepdim=True)
    rel = ((additions + 8) * U * (var + e * e) + e * e) / (var + eps) + 4 * U
    tol = ((e + 2 * U * d.abs()) * rstd + d.abs() * rstd * (rel + 2 * U)) * w64.abs() + 2 * U * (y.abs() + (d * rstd * w64).abs())
    return h, y, mean[:, 0], rstd[:, 0], tol, e[:, 0], (rstd * rel)[:, 0]


def rounded(tol, want, dtype):
    return tol + util.HALF[dtype] * (want.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0)


SIZES = [(1, 1), (1, 2), (1, 8), (3, 7), (5, 64), (257, 256), (300, 512), (2, 1000), (700, 1001), (33, 2048), (9, 4096), (3, 4100),
         (2, 8192), (2, 16384), (2, 16383), (1, 1025), (5000, 96), (6000, 4096), (30000, 512), (2000, 640)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,dim", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(dtype, n, dim, residual):
    x, w, b = rand((n, dim), dtype, 1, offset=0.5), rand((dim,), torch.float32, 2), rand((dim,), torch.float32, 3)
    r = rand((n, dim), dtype, 4) if residual else None
    out, total, mean, rstd = csa.layer_norm_forward(x, w, b, 1e-5, residual=r)
    h, y, m64, r64, tol, tol_m, tol_r = forward64(x, w, b, 1e-5, r)
    assert (total is None) == (not residual)
    if residual:
        assert torch.equal(total, h)
    assert ((mean.double() - m64).abs() <= tol_m).all() and ((rstd.double() - r64).abs() <= tol_r).all()
    assert ((out.double() - y).abs() <= rounded(tol, y, dtype)).all()


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_without_parameters(weight, bias):
    x = rand((37, 512), torch.bfloat16, 5)
    w, b = rand((512,), torch.float32, 6) if weight else None, rand((512,), torch.float32, 7) if bias else None
    out, _, mean, rstd = csa.layer_norm_forward(x, w, b)
    _, y, _, _, tol, _, _ = forward64(x, w, b, 1e-5)
    assert ((out.double() - y).abs() <= rounded(tol, y, x.dtype)).all()
    dx, dw, db = csa.layer_norm_backward(x, x, w, mean, rstd)
    ones = torch.ones(512, device="cuda")
    again = csa.layer_norm_backward(x, x, ones if w is None else w, mean, rstd)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1]) and torch.equal(db, again[2])


def test_an_offset_far_larger_than_the_spread():
    # mean 4096, spread 1: mean(x^2) - mean^2 in fp32 would leave nothing of the variance.  128 threads with two vectors of four
    # each: a term passes fewer than 64 additions.
    x = (torch.randn((64, 1024), generator=torch.Generator().manual_seed(8)) + 4096).cuda()
    out, _, mean, rstd = csa.layer_norm_forward(x)
    _, y, m64, r64, tol, tol_m, tol_r = forward64(x, None, None, 1e-5, additions=64)
    assert ((out.double() - y).abs() <= rounded(tol, y, x.dtype)).all()
    assert ((rstd.double() - r64).abs() <= tol_r).all() and tol_r.max() < 1e-2


def test_constant_rows():
    # no spread: out is the bias whatever the constant, and rstd 1 / sqrt(eps)
    x = torch.full((5, 512), 3.0, device="cuda", dtype=torch.bfloat16)
    b = rand((512,), torch.float32, 9)
    out, _, mean, rstd = csa.layer_norm_forward(x, None, b, 1e-4)
    assert (mean == 3).all() and torch.equal(out, b.bfloat16().expand(5, -1)) and ((rstd - 100).abs() <= 1e-4).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_bases_and_places(dtype):
    big = rand((20, 1100), dtype, 10)
    for first, dim in ((0, 512), (8, 512), (1, 512), (3, 333), (2, 444)):
        x, r = big[2:17, first:first + dim], big[1:16, first + 64:first + 64 + dim]
        _, y, _, _, tol, _, _ = forward64(x, None, None, 1e-5, r)
        a = csa.layer_norm_forward(x, residual=r)
        wide = torch.zeros(15, dim + 24, dtype=dtype, device="cuda")
        csa.layer_norm_forward(x, residual=r, out=wide[:, :dim])
        for o in (a[0], wide[:, :dim]):
            assert ((o.double() - y).abs() <= rounded(tol, y, dtype)).all()
        assert (wide[:, dim:] == 0).all()
        own = x.contiguous()
        out, total, _, _ = csa.layer_norm_forward(own, residual=r.contiguous(), out=own)
        assert out is own and torch.equal(total, a[1]) and ((own.double() - y).abs() <= rounded(tol, y, dtype)).all()


def test_nan_and_infinity_stay_in_their_row():
    x = rand((4, 512), torch.bfloat16, 11)
    clean = csa.layer_norm_forward(x)[0]
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    out = csa.layer_norm_forward(x)[0]
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3]) and out[1].isnan().all() and out[2].isnan().any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,dim", SIZES + [(700, 256), (65, 1024), (3, 9001), (40000, 64)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward(dtype, n, dim, residual):
    h, w = rand((n, dim), dtype, 12, offset=0.5), rand((dim,), torch.float32, 13)
    dy = rand((n, dim), dtype, 14)
    dh = rand((n, dim), dtype, 15) if residual else None
    mean = h.double().mean(1).float()
    rstd = (h.double().var(1, unbiased=False) + 1e-5).rsqrt().float()
    dx, dw, db = csa.layer_norm_backward(dy, h, w, mean, rstd, grad_residual=dh)
    hd, gd, wd, rd = h.double(), dy.double(), w.double(), rstd.double()[:, None]
    unit, g = (hd - mean.double()[:, None]) * rd, wd * gd
    through, level = (g * unit).mean(1, keepdim=True), g.mean(1, keepdim=True)
    want = rd * (g - level - unit * through)
    e_t, e_l = (dim + 8) * U * (g * unit).abs().mean(1, keepdim=True), (dim + 8) * U * g.abs().mean(1, keepdim=True)
    tol = rd * (8 * U * (g.abs() + (unit * through).abs() + level.abs()) + unit.abs() * e_t + e_l)
    if residual:
        want, tol = want + dh.double(), tol + 2 * U * dh.double().abs()
    assert ((dx.double() - want).abs() <= rounded(tol, want, dtype)).all()
    assert ((dw.double() - (gd * unit).sum(0)).abs() <= (n + 8) * U * (gd * unit).abs().sum(0) + 1e-30).all()
    assert ((db.double() - gd.sum(0)).abs() <= (n + 8) * U * gd.abs().sum(0) + 1e-30).all()
    again = csa.layer_norm_backward(dy, h, w, mean, rstd, grad_residual=dh)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))


def test_backward_strides():
    big, grads = rand((40, 1200), torch.bfloat16, 16), rand((40, 1200), torch.bfloat16, 17)
    w = rand((512,), torch.float32, 18)
    for first in (0, 8, 2, 3):
        h, dy, dh = big[3:39, first:first + 512], grads[1:37, first:first + 512], grads[2:38, first + 600:first + 1112]
        _, _, mean, rstd = csa.layer_norm_forward(h, w)
        got = csa.layer_norm_backward(dy, h, w, mean, rstd, grad_residual=dh)
        want = csa.layer_norm_backward(dy.contiguous().float(), h.contiguous().float(), w, mean, rstd, grad_residual=dh.contiguous().float())
        assert ((got[0].float() - want[0]).abs() <= 2.0 ** -8 * want[0].abs() + 1e-5).all()
        assert torch.allclose(got[1], want[1], rtol=0, atol=1e-3) and torch.allclose(got[2], want[2], rtol=0, atol=1e-3)


def test_backward_against_differences():
    n, dim, step = 3, 24, 1e-4
    x, w, b = rand((n, dim), torch.float32, 19), rand((dim,), torch.float32, 20), rand((dim,), torch.float32, 21)
    dy = rand((n, dim), torch.float32, 22)
    _, _, mean, rstd = csa.layer_norm_forward(x, w, b)
    dx, dw, db = csa.layer_norm_backward(dy, x, w, mean, rstd)
    loss = lambda a, v, c: (forward64(a, v, c, 1e-5)[1] * dy.double()).sum()  # noqa: E731
    for i, j in ((0, 0), (1, 7), (2, 23)):
        d = torch.zeros(n, dim, dtype=torch.float64, device="cuda")
        d[i, j] = step
        e = torch.zeros(dim, dtype=torch.float64, device="cuda")
        e[j] = step
        xd, wd, bd = x.double(), w.double(), b.double()
        for got, hi, lo in ((dx[i, j], loss(xd + d, wd, bd), loss(xd - d, wd, bd)), (dw[j], loss(xd, wd + e, bd), loss(xd, wd - e, bd)),
                            (db[j], loss(xd, wd, bd + e), loss(xd, wd, bd - e))):
            num = ((hi - lo) / (2 * step)).item()
            assert abs(num - got.item()) <= 1e-5 * (1 + abs(num))


def test_no_rows():
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    out, _, mean, rstd = csa.layer_norm_forward(x)
    assert out.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = csa.layer_norm_backward(x, x, None, mean, rstd)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("use", ["both", "out", "total"])
@pytest.mark.parametrize("parameters", [False, True])
def test_autograd(residual, use, parameters):
    if use != "out" and not residual:
        pytest.skip("no second output")
    g = torch.Generator(device="cuda").manual_seed(23)
    leaf = lambda *s: torch.randn(s, device="cuda", generator=g).requires_grad_()  # noqa: E731
    x, r = leaf(2, 3, 64), leaf(2, 3, 64) if residual else None
    w, b = (leaf(64), leaf(64)) if parameters else (None, None)
    p, q = torch.randn(2, 3, 64, device="cuda", generator=g), torch.randn(2, 3, 64, device="cuda", generator=g)

    def loss(out, total):
        return (0 if use == "total" else (out * p).sum()) + (0 if use == "out" else (total * q).sum())

    got = layer_norm(x, w, b, r, 1e-5)
    leaves = [t for t in (x, w, b, r) if t is not None]
    grads = torch.autograd.grad(loss(*(got if residual else (got, None))), leaves, allow_unused=True)
    ref = [t.detach().double().requires_grad_() for t in leaves]
    h = ref[0] + (ref[-1] if residual else 0)
    y = (h - h.mean(-1, keepdim=True)) * (h.var(-1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    if parameters:
        y = y * ref[1] + ref[2]
    want = torch.autograd.grad(loss(y, h), ref, allow_unused=True)
    for got_, want_ in zip(grads, want):
        if want_ is None:
            assert got_ is None
        else:
            assert (got_.double() - want_).abs().max() <= 1e-5 * want_.abs().max()


def test_side_stream_and_graph():
    x, w, b = rand((2000, 512), torch.bfloat16, 24), rand((512,), torch.float32, 25), rand((512,), torch.float32, 26)
    want = csa.layer_norm_forward(x, w, b)
    grads = csa.layer_norm_backward(x, x, w, want[2], want[3])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = csa.layer_norm_forward(x, w, b, stream=s)
    back = csa.layer_norm_backward(x, x, w, got[2], got[3], stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and all(torch.equal(p, q) for p, q in zip(back, grads))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    results = []
    for g in graphs:
        with torch.cuda.graph(g):
            o = csa.layer_norm_forward(x, w, b)
            results.append((o, csa.layer_norm_backward(x, x, w, o[2], o[3])))
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, d in results:
        assert torch.equal(o[0], want[0]) and all(torch.equal(p, q) for p, q in zip(d, grads))


def test_captured_backward_while_an_eager_graph_lives():
    g = torch.Generator(device="cuda").manual_seed(27)
    x = torch.randn((33, 512), device="cuda", generator=g).bfloat16().requires_grad_()
    w, b = torch.ones(512, device="cuda", requires_grad=True), torch.zeros(512, device="cuda", requires_grad=True)
    eager = layer_norm(x, w, b).float().square().sum()  # kept alive across the capture
    want = torch.autograd.grad(eager, [x, w, b], retain_graph=True)
    leaves = [t.detach().clone().requires_grad_() for t in (x, w, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(layer_norm(*leaves).float().square().sum(), leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(layer_norm(*leaves).float().square().sum(), leaves)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.isfinite(eager)
