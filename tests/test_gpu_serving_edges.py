"""The serving operators where they are most likely to go wrong: totals and offsets past 32 bits, the kernels that only large
calls reach, values that are not finite, calls in place.  Each test ends with the device's status word clear."""
import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa
from test_gpu_latent import check, made

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def status_stays_clear():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_status() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n", [2, 3, 5, 33, 600])
def test_page_totals_past_31_bits_are_held(n):
    most = 2 ** 31 - 1
    free = i32([11, 12, 13, 14, 15, 16, 17, 18])
    table, cu, slots, counts = csa.page_tables(i32([0] * n), i32([most] * n), 1, 1, free, i32([[-1] * 4] * n), 6)
    assert table.tolist() == [[11, 12, 13, 14]] + [[-1] * 4] * (n - 1)
    assert cu.tolist() == [0] + [most] * n
    assert slots.tolist() == [11, 12, 13, 14, -1, -1]
    assert counts.tolist() == [most, 8, most - 8, most]
    # the totals pass 2^31 only with the last requests: those before are served as ever
    before, after = [0] * (n - 1) + [0], [1] * (n - 1) + [most]
    ids = i32(list(range(1000, 1000 + n + 3)))
    table, cu, slots, counts = csa.page_tables(i32(before), i32(after), 1, 1, ids, i32([[-1] * 4] * n), n + 5)
    want = [[1000 + r, -1, -1, -1] for r in range(n - 1)] + [[1000 + n - 1 + c for c in range(4)]]
    assert table.tolist() == want and cu.tolist() == list(range(n)) + [most]
    assert slots.tolist() == [1000 + i for i in range(n + 3)] + [-1, -1]
    assert counts.tolist() == [most, n + 3, most - n - 3, most]


# (narrow and wide teams, odd widths, two rows a warp, and rows enough for the ring)
NORMS = [(5, 512, 0, torch.bfloat16), (5, 512, 128, torch.bfloat16), (3, 1001, 0, torch.float16), (4, 4096, 128, torch.float32),
         (33001, 128, 0, torch.bfloat16), (33001, 256, 128, torch.float16), (4000, 4096, 128, torch.bfloat16),
         (4000, 2048, 0, torch.float32)]


@pytest.mark.parametrize("n,dim,group,dtype", NORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_weights_that_are_not_finite_reach_the_scales_of_eight_bits(n, dim, group, dtype, bad):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((n, dim), device="cuda", generator=g).to(dtype)
    w = torch.rand(dim, device="cuda", generator=g) + 0.5
    clean, clean_scales, _, _ = csa.rms_norm_forward(x, w, out_dtype=torch.float8_e4m3fn, scale_group=group)
    col = dim - 3
    x[n - 1, col] = 0  # an infinite weight times 0
    w[col] = bad
    out, scales, _, _ = csa.rms_norm_forward(x, w, out_dtype=torch.float8_e4m3fn, scale_group=group)
    x64 = x.double()
    y = x64 * (x64.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.double()
    want = y.view(n, -1, group or dim).abs().amax(2)  # NaN where there is one, else infinite
    hit = ~want.isfinite()
    assert hit.any(1).all()
    assert torch.equal(scales.isnan(), want.isnan()) and torch.equal(scales.isinf(), want.isinf())
    # the groups without that column stay as they were
    same = ~hit & (torch.arange(n, device="cuda") < n - 1)[:, None]
    assert torch.equal(scales[same], clean_scales[same])
    bytes_of = lambda t: t.view(torch.uint8).view(n, -1, group or dim)[same]  # noqa: E731
    assert torch.equal(bytes_of(out), bytes_of(clean))


@pytest.mark.parametrize("n,dim,group,dtype", NORMS)
def test_rows_of_zeros_without_eps(n, dim, group, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((n, dim), device="cuda", generator=g).to(dtype)
    x[n // 2] = 0
    out, scales, _, rstd = csa.rms_norm_forward(x, None, 0.0, out_dtype=torch.float8_e4m3fn, scale_group=group)
    assert rstd[n // 2].isinf() and scales[n // 2].isnan().all() and out[n // 2].float().isnan().all()
    rest = torch.arange(n, device="cuda") != n // 2
    assert scales[rest].isfinite().all() and rstd[rest].isfinite().all() and out[rest].float().isfinite().all()


def test_helpers_without_csa_torch_give_the_same(monkeypatch):
    from sparse_attention_kv_csa_gb300 import serving
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((50, 128), device="cuda", generator=g).bfloat16()
    w = torch.rand(128, device="cuda", generator=g)
    cache = torch.randn((6, 16, 128), device="cuda", generator=g).bfloat16()
    scales = torch.rand((6, 16), device="cuda", generator=g)
    q = torch.randn((3, 8, 128), device="cuda", generator=g).bfloat16()
    table, cu, lens = i32([[4, 1, -1], [0, 2, 5]]), i32([0, 1, 3]), i32([20, 48])

    def calls():
        a = csa.rms_norm_forward(x, w, residual=x)
        b = csa.rms_norm_forward(x, w, out_dtype=torch.float8_e4m3fn, scale_group=128)
        c = csa.rms_norm_backward(x, x, w, a[3], grad_residual=x)
        d = csa.page_tables(i32([0, 9]), i32([70, 30]), 4, 4, i32(list(range(9))), i32([[7] * 5] * 2), 30)
        e = csa.latent_attention(q, cache, table, cu, lens, 1, 0.1)
        f = csa.latent_attention(q, cache.to(torch.float8_e4m3fn), table, cu, lens, 1, 0.1, 64, scales, torch.zeros(8, device="cuda"))
        return [t if t is None or t.dtype != torch.float8_e4m3fn else t.view(torch.uint8) for r in (a, b, c, d, e, f) for t in r]

    short = calls()
    assert serving._short is not None
    monkeypatch.setattr(serving, "_short", None)
    for s, p in zip(short, calls()):
        assert (s is None and p is None) or torch.equal(s, p)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("held", [0, 2, 3, 5])
def test_too_narrow_a_table_is_widened_and_the_call_repeated(in_place, held):
    page, width = 4, 3
    before, after = i32([held * page, 2, 0]), i32([30, 41, 3])
    ids = torch.randperm(64, generator=torch.Generator().manual_seed(held)).int().cuda()
    free, taken = ids[20:].contiguous(), i32([2])
    narrow = i32([[-1] * width] * 3)
    narrow[0, :min(held, width)] = ids[:min(held, width)]
    narrow[1, 0] = ids[9]
    got, _, _, counts = csa.page_tables(before, after, 1, page, free, narrow, 80, taken=taken, out=narrow if in_place else None)
    need = counts[3].item()
    assert need == 11 > width
    wide = torch.full((3, need), -7, dtype=torch.int32, device="cuda")
    wide[:, :width] = got
    # (the caller's own pages past the old width, which the narrow table could not hold)
    wide[0, width:max(held, width)] = ids[width:max(held, width)]
    again = csa.page_tables(before, after, 1, page, free, wide, 80, taken=taken)
    want = u.pages_plain(before.tolist(), after.tolist(), 1, page, free.tolist(),
                         [ids[:held].tolist() + [-1] * (need - held), [ids[9].item()] + [-1] * (need - 1), [-1] * need], 80, 2)
    for w, g in zip(want, again):
        assert list(w) == g.tolist()
    table = again[0]
    pages = table[table >= 0]
    assert pages.unique().numel() == pages.numel() == held + 1 + again[3][1].item()  # each held or taken page in one place


# ---- the norm's ring of rows: taken where the blocks that the rows need exceed three times the resident ones; these counts
# exceed three times what 152 SMs of 2048 threads can hold, whatever the registers.
#
# Bounds, u = 2^-24, as in test_gpu_norm.py: rstd from a sum of dim squares, (dim / 2 + 8) u; y three roundings more, 8-bit
# scales at most eight more; out one rounding to its type; the gradient's mean sums dim products.
U = 2.0 ** -24


def rows_of(n, dim, dtype, seed, stride=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, dim + stride), device="cuda", generator=g) * torch.exp(0.5 * torch.randn(dim + stride, device="cuda", generator=g))
    return x.to(dtype)[:, :dim]


@pytest.mark.parametrize("n,dim,dtype,residual,group,stride", [
    (30011, 512, torch.bfloat16, False, 0, 0), (30011, 512, torch.float16, True, None, 8), (30013, 384, torch.float32, True, 128, 4),
    (40009, 128, torch.bfloat16, True, 128, 64), (30011, 1024, torch.bfloat16, False, 128, 0),
    (7501, 2048, torch.bfloat16, True, None, 0), (7501, 4096, torch.bfloat16, True, 128, 0), (7501, 4096, torch.float16, False, 0, 24),
    (3701, 4096, torch.float32, True, 128, 0), (3701, 8192, torch.bfloat16, True, 0, 0), (1901, 16384, torch.bfloat16, True, 128, 8),
    (1901, 8192, torch.float32, False, None, 0), (1001, 16384, torch.float32, True, None, 0), (1001, 16384, torch.float32, True, 128, 0)])
def test_ring_forward(n, dim, dtype, residual, group, stride):
    """group None: output of x's type, else 8 bits."""
    x, w = rows_of(n, dim, dtype, 31, stride), rows_of(1, dim, torch.float32, 32)[0]
    r = rows_of(n, dim, dtype, 33, stride) if residual else None
    kw = {} if group is None else dict(out_dtype=torch.float8_e4m3fn, scale_group=group)
    out, scales, total, rstd = csa.rms_norm_forward(x, w, 1e-6, residual=r, **kw)
    h, y, rs = u.norm64(x, w, 1e-6, r)
    e = (dim / 2 + 16) * U
    assert total is None if r is None else torch.equal(total, h)
    assert ((rstd.double() - rs).abs() <= e * rs).all()
    if group is None:
        small = 1e-7 if dtype == torch.float16 else 0.0
        assert ((out.double() - y).abs() <= (u.HALF[dtype] * (1 + e) + 2 * e) * y.abs() + small).all()
    else:
        y = y.view(n, -1, group or dim)
        want = y.abs().amax(2) / 448
        assert ((scales.double() - want).abs() <= e * want).all()
        got = out.double().view_as(y) * scales.double()[..., None]
        assert ((got - y).abs() <= (2.0 ** -4 + 2 * e) * y.abs() + (2.0 ** -10 + 2 * e) * want[..., None]).all()
    again = csa.rms_norm_forward(x, w, 1e-6, residual=r, **kw)
    assert torch.equal(again[0].view(torch.uint8), out.view(torch.uint8)) and torch.equal(again[3], rstd)


@pytest.mark.parametrize("n,dim,dtype,residual,stride", [
    (30011, 512, torch.bfloat16, True, 0), (30011, 256, torch.float16, False, 8), (30011, 128, torch.float32, True, 0),
    (15013, 1024, torch.bfloat16, True, 16), (7501, 2048, torch.bfloat16, False, 0), (7501, 1024, torch.float32, True, 4),
    (3701, 4096, torch.bfloat16, True, 0), (3701, 4096, torch.float16, False, 40), (1901, 8192, torch.bfloat16, True, 0),
    (1001, 16384, torch.bfloat16, True, 0), (1001, 8192, torch.float32, True, 0), (1001, 16384, torch.float32, True, 0),
    (1001, 16384, torch.float32, False, 8)])
def test_ring_backward(n, dim, dtype, residual, stride):
    h, w = rows_of(n, dim, dtype, 41, stride), rows_of(1, dim, torch.float32, 42)[0]
    dy = rows_of(n, dim, dtype, 43, stride)
    dh = rows_of(n, dim, dtype, 44, stride) if residual else None
    rstd = h.float().square().mean(1).add(1e-6).rsqrt()
    dx, dw = csa.rms_norm_backward(dy, h, w, rstd, grad_residual=dh)
    gd, unit = dy.double(), h.double() * rstd.double()[:, None]
    wg, rd = w.double() * gd, rstd.double()[:, None]
    want = rd * (wg - unit * (wg * unit).mean(1, keepdim=True))
    tol = 8 * U * rd * (wg.abs() + unit.abs() * (wg * unit).abs().mean(1, keepdim=True) * (dim + 8) / 4)
    if residual:
        want = want + dh.double()
        tol = tol + 2 * U * dh.double().abs()
    tol = tol + u.HALF[dtype] * (want.abs() + tol) + (1e-7 if dtype == torch.float16 else 0.0)
    assert ((dx.double() - want).abs() <= tol).all()
    terms = gd * unit
    assert ((dw.double() - terms.sum(0)).abs() <= (n + 8) * U * terms.abs().sum(0)).all()
    again = csa.rms_norm_backward(dy, h, w, rstd, grad_residual=dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


IN_PLACE = [(1, 8, torch.bfloat16), (300, 1001, torch.bfloat16), (300, 1002, torch.float16), (33001, 128, torch.bfloat16),
            (30011, 512, torch.bfloat16), (7501, 4096, torch.bfloat16), (3701, 4096, torch.float32), (9, 16384, torch.float32),
            (1001, 16384, torch.float32), (40000, 333, torch.float32)]
CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


@pytest.mark.parametrize("n,dim,dtype", IN_PLACE)
def test_forward_in_place(n, dim, dtype):
    x, r, w = rows_of(n, dim, dtype, 51).contiguous(), rows_of(n, dim, dtype, 52).contiguous(), rows_of(1, dim, torch.float32, 53)[0]
    want = csa.rms_norm_forward(x, w, 1e-6, residual=r)
    alone = csa.rms_norm_forward(x, w, 1e-6)
    a = x.clone()
    assert torch.equal(csa.rms_norm_forward(a, w, 1e-6, out=a)[0], alone[0])
    for out_is_x in (True, False):
        a, b, rstd = x.clone(), r.clone(), torch.empty(n, device="cuda")
        out, total = (a, b) if out_is_x else (b, a)
        csa.csa_rms_norm_fwd(a, dim, b, dim, w, n, dim, 1e-6, CODES[dtype], None, 0, out, dim, CODES[dtype], None, 0, total, rstd)
        assert torch.equal(out, want[0]) and torch.equal(total, want[2]) and torch.equal(rstd, want[3])


@pytest.mark.parametrize("n,dim,dtype", IN_PLACE)
def test_backward_in_place(n, dim, dtype):
    h, dy, dh = (rows_of(n, dim, dtype, s).contiguous() for s in (54, 55, 56))
    w = rows_of(1, dim, torch.float32, 57)[0]
    rstd = h.float().square().mean(1).add(1e-6).rsqrt()
    want = csa.rms_norm_backward(dy, h, w, rstd, grad_residual=dh)
    for onto_dy in (True, False):
        a, b, dw = dy.clone(), dh.clone(), torch.empty(dim, device="cuda")
        dx = a if onto_dy else b
        csa.csa_rms_norm_bwd(h, dim, a, dim, b, dim, w, rstd, n, dim, CODES[dtype], dx, dw)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("first,dim", [(0, 512), (8, 512), (1, 512), (3, 333), (2, 334)])
def test_strided_output_holds_the_norm(dtype, first, dim):
    big = rows_of(20, 1100, dtype, 61)
    x, r = big[2:17, first:first + dim], big[1:16, first + 64:first + 64 + dim]
    for base in (0, 1, 8):
        room = torch.full((15, dim + 24), 7.0, dtype=dtype, device="cuda")
        csa.rms_norm_forward(x, None, residual=r, out=room[:, base:base + dim])
        _, y, _ = u.norm64(x, None, 1e-6, r)
        e, small = (dim / 2 + 16) * U, 1e-7 if dtype == torch.float16 else 0.0
        assert ((room[:, base:base + dim].double() - y).abs() <= (u.HALF[dtype] + 2 * e) * y.abs() + small).all()
        assert (room[:, :base] == 7).all() and (room[:, base + dim:] == 7).all()


# ---- attention: what only wide rows in odd pages, many requests, long requests among short ones, or large totals reach


@pytest.mark.parametrize("dim,v_dim", [(256, 256), (320, 320), (512, 512), (576, 512)])
@pytest.mark.parametrize("page", [1, 3, 50])
@pytest.mark.parametrize("bits8", [False, True])
def test_wide_rows_in_odd_pages(dim, v_dim, page, bits8):
    check(made([513, 64, 200, 3], [1, 1, 9, 3], 16, dim, 1, page, bits8, True, seed=dim + page), v_dim)


@pytest.mark.parametrize("dim,bits8", [(64, False), (128, True), (512, False), (200, False)])
def test_more_requests_than_the_division_keeps(dim, bits8):
    lens = [(7 * i) % 90 for i in range(3000)]
    check(made(lens, [min(1, a) for a in lens], 4, dim, 2, 16, bits8, seed=60))


@pytest.mark.parametrize("dim,page,bits8", [(512, 64, False), (512, 64, True), (128, 64, False), (576, 16, False), (256, 50, False)])
@pytest.mark.parametrize("where", [0, 9, 19])
def test_a_long_request_among_short_ones(dim, page, bits8, where):
    lens = [40 + i for i in range(20)]
    lens[where] = 12001
    check(made(lens, [1] * 20, 16, dim, 1, page, bits8, True, seed=61), min(dim, 512))


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("lens,news,ratio", [([900], [300], 4), ([5000, 131], [260, 130], 128)])
def test_prompts(lens, news, ratio, bits8):
    check(made(lens, news, 64, 512, ratio, 64, bits8, True, seed=62))


def test_units_past_2_to_the_20():
    # 5000 tokens of 64 heads, an item each, over 11384 to 16384 rows in tiles of 64: more than 5000 * (177 + 3) on average 220
    new, total, heads, dim, page = 5000, 16384, 64, 64, 64
    assert sum((total - new + i + 1 + 63) // 64 + 3 for i in range(new)) >= 1 << 20
    g = torch.Generator(device="cuda").manual_seed(63)
    cache = torch.randn((total // page, page, dim), device="cuda", generator=g).bfloat16()
    table = torch.randperm(total // page, device="cuda", generator=g).int()[None]
    q = torch.randn((new, heads, dim), device="cuda", generator=g).bfloat16()
    out, lse = csa.latent_attention(q, cache, table, i32([0, new]), i32([total]), 1, 0.125)
    torch.cuda.synchronize()
    for t in sorted({0, 1, new - 1, *range(17, new, 61)}):
        a = dict(q=q[t:t + 1], cache=cache, block_table=table, cu_q=i32([0, 1]), seq_lens=i32([total - new + t + 1]), ratio=1, scale=0.125)
        check(a, out=out[t:t + 1], lse=lse[t:t + 1])


@pytest.mark.parametrize("dim,bits8", [(512, False), (512, True), (128, False), (96, False), (96, True)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("row", [100, 128])
def test_every_query_that_sees_a_bad_row_shows_it(dim, bits8, bad, row):
    # of 130 rows the last four belong to the new tokens: token i sees rows up to 126 + i, so row 128 is seen by two of them
    a = made([130], [4], 8, dim, 1, 64, bits8, seed=8)
    out, lse = check(a)
    at = (a["block_table"][0, row // 64], row % 64)
    if bits8:
        a["row_scales"][at] = bad
    else:
        a["cache"][at][5] = bad
    sees = max(0, row - 126)
    out2, lse2 = csa.latent_attention(**a)
    assert torch.equal(out[:sees], out2[:sees]) and torch.equal(lse[:sees], lse2[:sees])
    assert not out2[sees:].isfinite().all(2).any()
