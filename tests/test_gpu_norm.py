"""rms_norm forward and backward against 64 bits.

Bounds, u = 2^-24: rstd from a sum of dim squares (any order: relative dim u, halved by the root) and five roundings:
(dim / 2 + 8) u.  y adds three roundings; out one rounding to its type.  The gradient's mean sums dim products of
relative error (rstd's + 6 u): dim u of the sum of magnitudes on top; grad_weight sums n_rows products."""
import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def rand(shape, dtype, seed, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[-1:], generator=g))
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,dim", [(1, 1), (1, 8), (3, 7), (5, 64), (257, 256), (300, 512), (2, 1000), (700, 1001),
                                   (33, 2048), (9, 4096), (3, 4100), (2, 8192), (2, 16384), (2, 16383), (1, 1025)])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(dtype, n, dim, residual):
    x, w = rand((n, dim), dtype, 1), rand((dim,), torch.float32, 2)
    r = rand((n, dim), dtype, 3) if residual else None
    out, scales, total, rstd = csa.rms_norm_forward(x, w, 1e-5, residual=r)
    h, y, rs = u.norm64(x, w, 1e-5, r)
    assert scales is None and (total is None) == (not residual)
    if residual:
        assert torch.equal(total, h)
    e = (dim / 2 + 8) * U
    assert ((rstd.double() - rs).abs() <= e * rs).all()
    assert ((out.double() - y).abs() <= (u.HALF[dtype] * (1 + e) + e + 3 * U) * y.abs() + 1e-7 * (dtype == torch.float16)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,dim,group", [(1, 128, 128), (300, 512, 0), (300, 512, 128), (7, 1024, 128), (5, 4096, 128),
                                         (5, 4096, 0), (4, 1001, 0), (3, 7, 0), (2, 16384, 128), (2, 640, 128), (2, 100, 0)])
def test_eight_bits(dtype, n, dim, group):
    x, w = rand((n, dim), dtype, 4), rand((dim,), torch.float32, 5)
    x[n // 2] = 0  # a row of zeros: scale 0, values 0
    out, scales, _, _ = csa.rms_norm_forward(x, w, 1e-6, out_dtype=torch.float8_e4m3fn, scale_group=group)
    _, y, _ = u.norm64(x, w, 1e-6)
    groups = y.view(n, -1, group or dim)
    want = groups.abs().amax(2) / 448
    e = (dim / 2 + 16) * U
    assert scales.shape == want.shape and ((scales.double() - want).abs() <= e * want).all()
    assert (scales[n // 2] == 0).all() and (out[n // 2].float() == 0).all()
    got = out.double().view_as(groups) * scales.double()[..., None]
    # half a step of e4m3: 2^-4 of the value, at least half of its smallest step (2^-10 of the scale)
    tol = (2.0 ** -4 + 2 * e) * groups.abs() + (2.0 ** -10 + 2 * e) * want[..., None]
    assert ((got - groups).abs() <= tol).all()


def test_slots_leave_other_rows_alone():
    n, dim, total = 37, 512, 64
    x = rand((n, dim), torch.bfloat16, 6)
    slots = torch.randperm(total, generator=torch.Generator().manual_seed(1))[:n].cuda()
    slots[3], slots[20], slots[36] = -1, total, 1 << 40  # nowhere
    keep = (slots >= 0) & (slots < total)
    plain, ps, _, _ = csa.rms_norm_forward(x, out_dtype=torch.float8_e4m3fn)
    out = torch.full((total, dim), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((total,), -7.0, device="cuda")
    csa.rms_norm_forward(x, slots=slots, out=out.view(torch.float8_e4m3fn), scales=scales)
    want, want_s = torch.full_like(out, 0x55), torch.full_like(scales, -7.0)
    want[slots[keep]] = plain.view(torch.uint8)[keep]
    want_s[slots[keep]] = ps[keep, 0]
    assert torch.equal(out, want) and torch.equal(scales, want_s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_bases(dtype):
    big = rand((20, 1100), dtype, 7)
    for first, dim in ((0, 512), (8, 512), (1, 512), (3, 333)):
        x = big[2:17, first:first + dim]
        r = big[1:16, first + 64:first + 64 + dim]
        a = csa.rms_norm_forward(x, None, residual=r)
        b = csa.rms_norm_forward(x.contiguous(), None, residual=r.contiguous())
        _, y, _ = u.norm64(x, None, 1e-6, r)
        assert torch.equal(a[2], b[2])
        e = (dim / 2 + 16) * U
        for o in (a[0], b[0]):
            assert ((o.double() - y).abs() <= (u.HALF[dtype] + 2 * e) * y.abs()).all()
        out = torch.zeros(15, dim + 24, dtype=dtype, device="cuda")
        csa.rms_norm_forward(x, None, residual=r, out=out[:, :dim])
        assert torch.equal(out[:, :dim], a[0]) or dtype == torch.float32 or first == 1
        assert (out[:, dim:] == 0).all()


def test_nan_and_infinity_stay_in_their_row():
    x = rand((4, 512), torch.bfloat16, 8)
    clean = csa.rms_norm_forward(x)[0]
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    out, s, _, _ = csa.rms_norm_forward(x, out_dtype=torch.float8_e4m3fn)
    assert s[1].isnan().all()
    out = csa.rms_norm_forward(x)[0]
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    assert out[1].isnan().all() and out[2, 7].isnan()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,dim", [(1, 1), (1, 64), (3, 7), (700, 256), (300, 512), (65, 1024), (20, 1001), (9, 2048),
                                   (9, 4096), (3, 8192), (2, 16384), (2, 9001), (5000, 96)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward(dtype, n, dim, residual):
    h, w = rand((n, dim), dtype, 9), rand((dim,), torch.float32, 10)
    dy = rand((n, dim), dtype, 11)
    dh = rand((n, dim), dtype, 12) if residual else None
    rstd = h.float().square().mean(1).add(1e-6).rsqrt()
    dx, dw = csa.rms_norm_backward(dy, h, w, rstd, grad_residual=dh)
    hd, gd, wd, rd = h.double(), dy.double(), w.double(), rstd.double()[:, None]
    unit = hd * rd
    c = (wd * gd * unit).mean(1, keepdim=True)
    want = rd * (wd * gd - unit * c)
    # magnitudes before cancellation, and the mean's error through the sum of magnitudes
    mag = rd * ((wd * gd).abs() + unit.abs() * (wd * gd * unit).abs().mean(1, keepdim=True) * (dim + 8) / 4)
    tol = 8 * U * mag
    if residual:
        want = want + dh.double()
        tol = tol + 2 * U * dh.double().abs()
    tol = tol + u.HALF[dtype] * (want.abs() + tol) + 1e-7 * (dtype == torch.float16)
    assert ((dx.double() - want).abs() <= tol).all()
    terms = (gd * unit).abs().sum(0)
    assert ((dw.double() - (gd * unit).sum(0)).abs() <= (n + 8) * U * terms + 1e-30).all()
    dx2, dw2 = csa.rms_norm_backward(dy, h, w, rstd, grad_residual=dh)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_backward_against_differences():
    # fp32 inputs, central differences of the 64-bit form
    n, dim, step = 3, 24, 1e-4
    x, w = rand((n, dim), torch.float32, 13), rand((dim,), torch.float32, 14)
    dy = rand((n, dim), torch.float32, 15)
    _, _, _, rstd = csa.rms_norm_forward(x, w, 1e-6)
    dx, dw = csa.rms_norm_backward(dy, x, w, rstd)
    loss = lambda a, b: (u.norm64(a, b, 1e-6)[1] * dy.double()).sum()  # noqa: E731
    for i, j in ((0, 0), (1, 7), (2, 23)):
        d = torch.zeros(n, dim, dtype=torch.float64, device="cuda")
        d[i, j] = step
        num = (loss(x.double() + d, w) - loss(x.double() - d, w)) / (2 * step)
        assert abs(num.item() - dx[i, j].item()) <= 1e-5 * (1 + abs(num.item()))
        num = (loss(x.double(), w.double() + d[i]) - loss(x.double(), w.double() - d[i])) / (2 * step)
        assert abs(num.item() - dw[j].item()) <= 1e-5 * (1 + abs(num.item()))


def test_no_rows():
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    out, _, _, rstd = csa.rms_norm_forward(x)
    assert out.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = csa.rms_norm_backward(x, x, None, rstd)
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_side_stream_and_graph():
    x, w = rand((513, 512), torch.bfloat16, 16), rand((512,), torch.float32, 17)
    want = csa.rms_norm_forward(x, w)
    grads = csa.rms_norm_backward(x, x, w, want[3])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = csa.rms_norm_forward(x, w, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = csa.rms_norm_forward(x, w)
        d = csa.rms_norm_backward(x, x, w, o[3])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o[0], want[0]) and torch.equal(d[0], grads[0]) and torch.equal(d[1], grads[1])


@pytest.mark.parametrize("dim,bits8,group,dtype",
                         [(128, False, 0, torch.bfloat16), (128, True, 0, torch.bfloat16), (136, False, 0, torch.float16),
                          (256, True, 128, torch.bfloat16), (512, True, 0, torch.bfloat16), (512, True, 128, torch.float16),
                          (504, True, 0, torch.bfloat16), (128, True, 128, torch.float32), (256, True, 128, torch.float32),
                          (256, False, 0, torch.float32), (33, False, 0, torch.bfloat16), (576, True, 0, torch.bfloat16)])
def test_many_narrow_rows(dim, bits8, group, dtype):
    # two rows a warp, where 16-bit types and whole vectors allow it
    n = 33001
    x, r, w = rand((n, dim), dtype, 20), rand((n, dim), dtype, 21), rand((dim,), torch.float32, 22)
    x[17], r[17] = 0, 0
    out, scales, total, rstd = csa.rms_norm_forward(x, w, 1e-6, residual=r, scale_group=group,
                                                    out_dtype=torch.float8_e4m3fn if bits8 else None)
    h, y, rs = u.norm64(x, w, 1e-6, r)
    e = (dim / 2 + 16) * U
    assert torch.equal(total, h) and ((rstd.double() - rs).abs() <= e * rs).all()
    if not bits8:
        assert ((out.double() - y).abs() <= (u.HALF[dtype] + 2 * e) * y.abs() + (2.0 ** -25 if dtype == torch.float16 else 0)).all()
        return
    groups = y.view(n, -1, group or dim)
    want = groups.abs().amax(2) / 448
    assert ((scales.double() - want).abs() <= e * want).all()
    got = out.double().view_as(groups) * scales.double()[..., None]
    assert ((got - groups).abs() <= (2.0 ** -4 + 2 * e) * groups.abs() + (2.0 ** -10 + 2 * e) * want[..., None]).all()
