"""latent_attention against 64 bits (serving_util.attention64 has the bounds)."""
import math
import random

import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa

pytestmark = pytest.mark.gpu


def made(lens, news, heads, dim, ratio, page, bits8=False, sink=False, seed=0, spare=2, q_scale=1.0, width=0):
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    used = [-(-(a // ratio) // page) for a in lens]
    pages = sum(used) + spare
    ids = list(range(pages))
    rng.shuffle(ids)
    width = width or max(used + [1])
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for r, k in enumerate(used):
        for c in range(min(k, width)):
            table[r, c] = ids.pop()
    rows = torch.randn((pages, page, dim), generator=g)
    a = {}
    if bits8:
        a["row_scales"] = (rows.abs().amax(2) / 448).cuda()
        a["cache"] = (rows / (rows.abs().amax(2) / 448)[..., None]).to(torch.float8_e4m3fn).cuda()
    else:
        a["cache"] = rows.bfloat16().cuda()
    a["q"] = (q_scale * torch.randn((sum(news), heads, dim), generator=g)).bfloat16().cuda()
    cu = [0]
    for b in news:
        cu.append(cu[-1] + b)
    a["block_table"] = table.cuda()
    a["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    a["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a["ratio"], a["scale"] = ratio, 1 / math.sqrt(dim)
    if sink:
        a["sink"] = torch.randn((heads,), generator=g).cuda()
    return a


def check(a, v_dim=None, out=None, lse=None):
    v_dim = a["q"].shape[2] if v_dim is None else v_dim
    if out is None:
        out, lse = csa.latent_attention(**a, v_dim=v_dim)
        torch.cuda.synchronize()
        assert csa.csa_device_status() == 0
    want, want_lse, tol, tol_lse = u.attention64(a["q"], a["cache"], a["block_table"], a["cu_q"].cpu(), a["seq_lens"].cpu(),
                                                 a["ratio"], a["scale"], v_dim, a.get("row_scales"), a.get("sink"))
    got, got_lse = out.cpu().double(), lse.cpu().double()
    worst = ((got - want).abs() / tol).max().item() if got.numel() else 0
    assert got.isfinite().all() and worst <= 1, worst
    inf = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(got_lse), inf)
    assert ((got_lse - want_lse).abs() <= tol_lse)[~inf].all()
    assert (got[inf] == 0).all()
    return out, lse


WIDTHS = [(512, 512), (576, 512), (256, 256), (192, 128), (128, 128), (64, 64), (576, 64), (320, 192)]
OTHER = [(8, 8), (96, 96), (200, 200), (104, 40), (640, 640), (1024, 1024), (576, 576), (264, 8)]


@pytest.mark.parametrize("dim,v_dim", WIDTHS + OTHER)
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("sink", [False, True])
def test_widths(dim, v_dim, bits8, sink):
    if bits8 and dim % 16:
        pytest.skip("8-bit rows are multiples of 16 bytes")
    check(made([300, 5, 777], [2, 1, 3], 8, dim, 3, 16, bits8, sink, seed=dim), v_dim)


@pytest.mark.parametrize("heads", [1, 3, 16, 24, 63, 64, 65, 128, 130])
@pytest.mark.parametrize("bits8", [False, True])
def test_heads(heads, bits8):
    check(made([260, 70, 4], [1, 5, 2], heads, 512, 1, 64, bits8, True, seed=heads))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 48, 50, 64, 100, 128, 256])
@pytest.mark.parametrize("bits8", [False, True])
def test_pages(page, bits8):
    check(made([513, 64, 200], [1, 1, 4], 16, 128, 1, page, bits8, seed=page))


@pytest.mark.parametrize("lens,news", [
    ([0], [0]), ([1], [1]), ([3], [3]), ([4], [1]), ([4], [4]), ([1, 0, 9, 0], [1, 0, 9, 0]), ([255, 256, 257], [1, 1, 1]),
    ([259, 260, 515], [4, 9, 1]), ([2000], [1]), ([2000], [70]), ([130], [130]), ([64, 1], [64, 1])])
@pytest.mark.parametrize("ratio", [1, 4])
@pytest.mark.parametrize("dim", [512, 96])
def test_lengths(lens, news, ratio, dim):
    a = made(lens, news, 16, dim, ratio, 16, sink=False, seed=len(lens))
    check(a)
    a["sink"] = torch.linspace(-3, 3, 16, device="cuda")
    check(a)


def test_more_new_tokens_than_the_request_has():
    # the first tokens lie before position 0: they see nothing
    a = made([5, 8], [9, 8], 4, 64, 2, 4, seed=3)
    out, lse = check(a)
    assert torch.isinf(lse[:4]).all()


@pytest.mark.parametrize("dim", [512, 128, 200])
def test_long_rows_split_over_blocks(dim):
    check(made([9001], [1], 4, dim, 1, 64, seed=4))
    check(made([9001, 3, 4000], [1, 1, 2], 64, dim, 1, 64, seed=4, sink=True))


def test_many_requests():
    rng = random.Random(1)
    lens = [rng.choice([0, 1, rng.randint(1, 40), rng.randint(1, 600)]) for _ in range(400)]
    news = [min(1, a) for a in lens]
    check(made(lens, news, 8, 128, 2, 16, seed=5))


@pytest.mark.parametrize("dim", [512, 96])
def test_peaked_and_large_logits(dim):
    # logits of several hundred: the running maximum has to move, the rest underflows
    check(made([700, 300], [1, 2], 8, dim, 1, 64, seed=6, q_scale=40.0))


@pytest.mark.parametrize("dim", [512, 96])
@pytest.mark.parametrize("bits8", [False, True])
def test_what_no_token_sees_may_hold_anything(dim, bits8):
    a = made([77, 130], [1, 3], 8, dim, 1, 64, bits8, seed=7, spare=3)
    out, lse = check(a)
    seen = torch.zeros(a["cache"].shape[:2], dtype=torch.bool)
    for r, length in enumerate([77, 130]):
        for j in range(length):
            seen[a["block_table"][r, j // 64], j % 64] = True
    raw = a["cache"].view(torch.uint8) if bits8 else a["cache"]
    raw[~seen.cuda()] = 0x7F if bits8 else float("nan")
    if bits8:
        a["row_scales"][~seen.cuda()] = float("nan")
    out2, lse2 = csa.latent_attention(**a)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dim", [512, 96])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_later_rows_do_not_reach_earlier_tokens(dim, bad):
    # rows 126..129 belong to the four new tokens: token i may read row 126 + i and no later one
    a = made([130], [4], 8, dim, 1, 64, seed=8)
    out, lse = check(a)
    a["cache"][a["block_table"][0, 2], 0, 5] = bad  # row 128
    out2, lse2 = csa.latent_attention(**a)
    assert torch.equal(out[:2], out2[:2]) and torch.equal(lse[:2], lse2[:2])
    assert not out2[2:].isfinite().all()


@pytest.mark.parametrize("dim", [512, 96])
def test_entries_outside_the_cache_hide_their_rows(dim):
    a = made([200, 90], [2, 1], 8, dim, 1, 16, seed=9)
    a["block_table"][0, 3], a["block_table"][0, 7], a["block_table"][1, 0] = -1, a["cache"].shape[0], 2 ** 31 - 1
    check(a)
    a["block_table"][1] = -5
    out, lse = check(a)
    assert torch.isinf(lse[2]).all()


def test_table_narrower_than_the_request():
    check(made([500], [3], 8, 128, 1, 16, seed=10, width=9))


def test_strides():
    a = made([150, 70], [2, 3], 8, 128, 1, 16, seed=11)
    base = check(a)
    q = torch.zeros(5, 12, 144, dtype=torch.bfloat16, device="cuda")
    q[:, 2:10, 8:136] = a["q"]
    cache = torch.full((a["cache"].shape[0] * 16, 160), float("nan"), dtype=torch.bfloat16, device="cuda")
    cache[:, 16:144] = a["cache"].view(-1, 128)
    table = torch.full((2, 40), 7, dtype=torch.int32, device="cuda")
    table[:, :a["block_table"].shape[1]] = a["block_table"]
    b = dict(a, q=q[:, 2:10, 8:136], cache=cache.view(-1, 16, 160)[:, :, 16:144], block_table=table[:, :a["block_table"].shape[1]])
    out, lse = csa.latent_attention(**b)
    assert torch.equal(out, base[0]) and torch.equal(lse, base[1])


@pytest.mark.parametrize("bits8", [False, True])
def test_offsets_past_32_bits(bits8):
    # rows past element 2^32 of the cache; only the table's pages are written
    dim, page = 512, 64
    pages = (2 ** 32 + 2 ** 24) // (dim * page)
    a = made([200], [1], 8, dim, 1, page, bits8, seed=12)
    big = torch.empty((pages, page, dim), dtype=torch.uint8 if bits8 else torch.bfloat16, device="cuda")
    scales = torch.empty((pages, page), device="cuda") if bits8 else None
    small = a["cache"].view(torch.uint8) if bits8 else a["cache"]
    n = small.shape[0]
    big[pages - n:] = small
    if bits8:
        scales[pages - n:] = a["row_scales"]
    base = check(a)
    b = dict(a, cache=big.view(torch.float8_e4m3fn) if bits8 else big, block_table=a["block_table"] + (pages - n))
    if bits8:
        b["row_scales"] = scales
    out, lse = csa.latent_attention(**b)
    assert torch.equal(out, base[0]) and torch.equal(lse, base[1])


def test_tokens_past_the_last_offset_are_left_alone():
    a = made([40, 20], [2, 1], 4, 128, 1, 16, seed=13)
    q = torch.cat([a["q"], torch.full_like(a["q"], float("nan"))])
    out = torch.full((6, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    got, _ = csa.latent_attention(**dict(a, q=q), out=out)
    assert (got[3:] == 3.0).all()
    base = csa.latent_attention(**a)
    assert torch.equal(got[:3], base[0])


@pytest.mark.parametrize("dim", [512, 96])
def test_repeats_side_stream_and_graph(dim):
    a = made([900, 17, 300], [1, 2, 1], 24, dim, 1, 64, seed=14, sink=True)
    out, lse = check(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = csa.latent_attention(**a, stream=s)
    s.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o3, l3 = csa.latent_attention(**a)
    a["q"].neg_()
    want = csa.latent_attention(**a)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o3, want[0]) and torch.equal(l3, want[1])


def test_cache_without_pages():
    a = made([40], [1], 8, 512, 1, 16, seed=15)
    a["cache"] = a["cache"][:0]
    out, lse = csa.latent_attention(**a)
    assert (out == 0).all() and torch.isinf(lse).all()


def test_items_in_a_row_with_few_live_rows():
    # one block takes both requests: the warp that writes the first one's output comes a tile later to the second
    for seed in range(6):
        a = made([77, 130], [1, 3], 8, 512, 1, 64, seed=seed)
        out, lse = check(a)
        for _ in range(5):
            o2, l2 = csa.latent_attention(**a)
            assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_scales_of_later_rows_may_hold_anything():
    # as test_later_rows...: a row that only later tokens see has a scale of NaN or infinity
    for bad in (float("nan"), float("inf")):
        a = made([130], [4], 8, 512, 1, 64, True, seed=8)
        out, lse = check(a)
        a["row_scales"][a["block_table"][0, 2], 0] = bad  # row 128
        out2, lse2 = csa.latent_attention(**a)
        assert torch.equal(out[:2], out2[:2]) and torch.equal(lse[:2], lse2[:2])
        assert not out2[2:].isfinite().all()
