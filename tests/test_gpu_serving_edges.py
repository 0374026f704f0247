"""The serving operators where they are most likely to go wrong: totals and offsets past 32 bits, the kernels that only large
calls reach, values that are not finite, calls in place.  Each test ends with the device's status word clear."""
import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa

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
