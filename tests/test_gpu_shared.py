"""shared_attention against 64 bits (serving_util.attention64 has the bounds; joining the prefix's part and the requests' own adds a
few roundings of fp32 to sums that the bound counts one for each row)."""
import math
import random

import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa

pytestmark = pytest.mark.gpu


def made(groups, heads, dim, ratio, page, bits8=False, sink=False, seed=0, q_scale=1.0, spare=2, copies=False, width=None):
    """groups: a list of (shared rows, [(rows behind them, new tokens), ...]).  The shared rows' whole pages are in every table
    of the group; with copies each request has pages of its own with equal contents.  A table with room for 400000 rows, which
    these lengths do not use, makes the call worth the kernels for prefixes; one of just the pages in use (width 0) leaves most of
    these small calls to the attention by requests."""
    if width is None:
        width = 400000 // page + 1
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    lens, news, cu_groups, need = [], [], [0], 0
    for shared, members in groups:
        for behind, new in members:
            lens.append((shared + behind) * ratio + rng.randint(0, ratio - 1))
            news.append(new)
            need += -(-(shared + behind) // page)
        cu_groups.append(len(lens))
    ids = list(range(need + spare))
    rng.shuffle(ids)
    widest = max([-(-(n // ratio) // page) for n in lens] + [1])
    table = torch.full((len(lens), max(width, widest)), -1, dtype=torch.int32)
    rows = torch.randn((need + spare, page, dim), generator=g)
    r = 0
    for shared, members in groups:
        whole = shared // page
        first = None
        for behind, _ in members:
            count = -(-(shared + behind) // page)
            mine = [ids.pop() for _ in range(count)]
            if first is None:
                first = mine
            else:
                rows[mine[:whole]] = rows[first[:whole]]
                if whole < count and whole < len(first) and shared % page:
                    rows[mine[whole], :shared % page] = rows[first[whole], :shared % page]
                if not copies:
                    mine[:whole] = first[:whole]
            table[r, :count] = torch.tensor(mine, dtype=torch.int32)
            r += 1
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
    int32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    a["block_table"], a["cu_q"], a["seq_lens"], a["cu_groups"] = table.cuda(), int32(cu), int32(lens), int32(cu_groups)
    a["shared_rows"] = int32([s for s, _ in groups])
    a["ratio"], a["scale"] = ratio, 1 / math.sqrt(dim)
    if sink:
        a["sink"] = torch.randn((heads,), generator=g).cuda()
    return a


def alone(a):
    return {k: v for k, v in a.items() if k not in ("cu_groups", "shared_rows")}


def check(a, v_dim=None, out=None, lse=None):
    v_dim = a["q"].shape[2] if v_dim is None else v_dim
    if out is None:
        out, lse = csa.shared_attention(**a, v_dim=v_dim)
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


ONE = [(400, [(30, 1), (0, 1), (77, 2), (200, 1), (5, 3)])]
TWO = [(520, [(30, 1), (61, 1), (16, 2)]), (130, [(3, 1), (300, 1), (12, 1), (9, 2)])]


@pytest.mark.parametrize("dim,v_dim", [(512, 512), (576, 512), (256, 256), (192, 128), (128, 128), (64, 64), (576, 64), (320, 192),
                                       (384, 384), (448, 256), (96, 96), (640, 640), (576, 576), (264, 8)])
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("width", [0, None])
def test_widths(dim, v_dim, bits8, sink, width):
    if bits8 and dim % 16:
        pytest.skip("8-bit rows are multiples of 16 bytes")
    check(made(TWO, 24, dim, 3, 16, bits8, sink, seed=dim, width=width), v_dim)


@pytest.mark.parametrize("heads", [1, 3, 16, 24, 63, 64, 65, 128, 130])
@pytest.mark.parametrize("bits8", [False, True])
def test_heads(heads, bits8):
    check(made(ONE, heads, 512, 1, 64, bits8, True, seed=heads))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 48, 50, 64, 100, 128, 256])
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("copies", [False, True])
def test_pages(page, bits8, copies):
    check(made(ONE, 32, 128, 1, page, bits8, seed=page, copies=copies))


@pytest.mark.parametrize("shared", [0, 1, 7, 8, 63, 64, 127, 128, 129, 192, 255, 256, 257, 1000, 2049])
@pytest.mark.parametrize("dim", [512, 128])
def test_prefix_lengths(shared, dim):
    check(made([(shared, [(20, 1), (64, 1), (0, 1), (129, 1)])], 32, dim, 1, 8, sink=shared % 2 == 0, seed=shared))


@pytest.mark.parametrize("groups", [
    [(300, [(1, 1)])], [(300, [(1, 1)] * 9), (64, [(5, 1)]), (700, [(2, 2)] * 3)], [(0, [(9, 1), (0, 0)]), (256, [(9, 1), (33, 1)])],
    [(128, [(0, 0), (0, 0)]), (128, [(3, 1), (4, 0), (2, 1)])], [(640, [(0, 1), (0, 1), (0, 1)])], [(200, []), (300, [(3, 1), (8, 4)])],
    [(0, [(0, 1), (0, 1)])], [(96, [(k % 3, 1 + k % 2) for k in range(70)])]])
@pytest.mark.parametrize("ratio", [1, 4])
def test_groups(groups, ratio):
    a = made(groups, 16, 512, ratio, 32, seed=len(groups))
    check(a)
    a["sink"] = torch.linspace(-3, 3, 16, device="cuda")
    check(a)


def test_requests_outside_of_groups():
    a = made([(200, [(30, 1)] * 3), (128, [(7, 1)] * 4), (64, [(9, 2)] * 2)], 16, 512, 1, 16, sink=True, seed=3)
    for cu in ([3, 7], [0, 3], [7, 9], [2, 2], [0, 0], [9, 9]):
        a["cu_groups"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        a["shared_rows"] = torch.tensor([128 if cu == [3, 7] else 64 if cu[0] >= 7 else 200], dtype=torch.int32, device="cuda")
        check(a)
    a["cu_groups"], a["shared_rows"] = a["cu_groups"][:1], a["shared_rows"][:0]
    check(a)  # no groups at all


def test_rows_that_a_token_does_not_see_are_not_shared():
    # a prompt's tokens lie inside the prefix; shared_rows reaches past every length; and is negative
    a = made([(300, [(0, 40), (5, 1), (0, 290)])], 4, 512, 1, 16, seed=4)
    check(a)
    a["shared_rows"] = torch.tensor([1 << 30], dtype=torch.int32, device="cuda")
    a["block_table"][1:] = a["block_table"][:1]  # (every row of every request is the first one's)
    check(a)
    a["shared_rows"] = torch.tensor([-5], dtype=torch.int32, device="cuda")
    check(a)
    # more new tokens than the request has: the first see nothing
    a = made([(64, [(4, 1), (2, 1)])], 8, 512, 2, 8, seed=5)
    a["seq_lens"] = torch.tensor([136, 0], dtype=torch.int32, device="cuda")
    out, lse = check(a)
    assert torch.isinf(lse[1]).all()


def test_narrow_tables_and_bad_entries():
    a = made([(400, [(100, 1), (30, 1), (64, 1)])], 16, 512, 1, 16, seed=6)
    bad = dict(a, block_table=a["block_table"].clone())
    bad["block_table"][:, 7] = -1              # hides rows 112 to 127 of all
    bad["block_table"][1, 27] = 1 << 20        # and own rows of one
    check(bad)
    narrow = dict(a, block_table=a["block_table"][:, :20].contiguous())  # 320 rows at most
    check(narrow)
    wide = torch.full((3, 27000), -1, dtype=torch.int32, device="cuda")
    wide[:, :a["block_table"].shape[1]] = a["block_table"]
    check(dict(a, block_table=wide[:, :26000]))
    check(dict(a, block_table=wide[:, :40]))
    # tables narrower than the rows, with enough requests for the prefix's kernels
    a = made([(400, [(100 + k % 7, 1) for k in range(700)]), (300, [(k % 9, 1) for k in range(20)])], 16, 128, 1, 16, seed=21, width=0)
    check(a)
    check(dict(a, block_table=a["block_table"][:, :31].contiguous()))


@pytest.mark.parametrize("bits8", [False, True])
def test_peaked_and_large_logits(bits8):
    # logits of several hundred: the running maximum has to move, the rest underflows, and prefix and own rows far apart
    check(made(ONE, 32, 512, 1, 64, bits8, True, seed=7, q_scale=40.0))
    a = made(ONE, 32, 512, 1, 64, bits8, seed=8)
    a["cache"] = a["cache"].clone()
    first = a["block_table"][0, :6].long()
    if bits8:
        a["row_scales"][first] *= 1e-3  # the prefix's logits are near zero
    else:
        a["cache"][first] *= 1e-3
    check(a)


@pytest.mark.parametrize("dim", [512, 128])
@pytest.mark.parametrize("bits8", [False, True])
def test_what_no_token_sees_may_hold_anything(dim, bits8):
    a = made([(200, [(77, 1), (130, 3), (5, 1)])], 24, dim, 1, 64, bits8, seed=9, spare=3)
    out, lse = check(a)
    seen = torch.zeros(a["cache"].shape[:2], dtype=torch.bool)
    for r, n in enumerate(a["seq_lens"].tolist()):
        for j in range(n):
            seen[a["block_table"][r, j // 64].item(), j % 64] = True
    hidden = ~seen.cuda()
    assert hidden.any()
    raw = a["cache"].view(torch.uint8).clone()
    raw[hidden] = 0x7f if bits8 else 0xff  # NaN
    b = dict(a, cache=raw.view(a["cache"].dtype))
    if bits8:
        b["row_scales"] = torch.where(hidden, float("nan"), a["row_scales"])
    again = csa.shared_attention(**b)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_infinities_and_nan_reach_those_that_see_them():
    a = made([(256, [(40, 1), (50, 3), (20, 1)])], 16, 512, 1, 64, seed=10)
    clean = csa.shared_attention(**a)
    own = a["block_table"][1, 4].item()
    a["cache"][own, 49, 3] = float("nan")  # row 305 of the second request: its last token alone sees it
    out, lse = csa.shared_attention(**a)
    assert out[3].isnan().all() and lse[3].isnan().all()
    keep = [0, 1, 2, 4]
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])
    a["cache"][a["block_table"][0, 1].item(), 5, 7] = float("nan")  # a shared row
    out, lse = csa.shared_attention(**a)
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("bits8", [False, True])
def test_many_requests_and_groups(bits8):
    rng = random.Random(2)
    groups = [(rng.choice([0, 50, 300, 800]), [(rng.randint(0, 60), rng.choice([0, 1, 1, 2])) for _ in range(rng.randint(1, 40))])
              for _ in range(12)]
    check(made(groups, 8, 256, 1, 16, bits8, True, seed=11))


def test_long_prefix_split_over_blocks():
    check(made([(9000, [(100, 1), (3, 1)])], 8, 512, 1, 64, seed=12, sink=True))
    check(made([(5000, [(100, 1)] * 9), (3000, [(64, 1)] * 5)], 64, 512, 1, 64, seed=13))


def test_equals_latent_attention_and_is_bitwise_repeatable():
    a = made([(2000, [(100 + k, 1) for k in range(40)])], 64, 512, 1, 64, True, True, seed=14)
    first = csa.shared_attention(**a)
    plain = csa.latent_attention(**alone(a))
    assert ((first[0].float() - plain[0].float()).abs() <= 2.0 ** -6 * plain[0].float().abs().amax(-1, keepdim=True)).all()
    assert (first[1] - plain[1]).abs().max() <= 1e-4
    for _ in range(3):
        again = csa.shared_attention(**a)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_tokens_outside_are_left_alone():
    a = made(ONE, 16, 512, 1, 64, seed=15)
    n = a["q"].shape[0]
    wide = torch.cat([a["q"][:2], a["q"], a["q"][:3]])
    b = dict(a, q=wide, cu_q=a["cu_q"] + 2)
    out = torch.full((n + 5, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    got, lse = csa.shared_attention(**b, out=out)
    want, want_lse = csa.shared_attention(**a)
    assert got is out and (out[:2] == 7).all() and (out[n + 2:] == 7).all()
    assert torch.equal(out[2:n + 2], want) and torch.equal(lse[2:n + 2], want_lse)


def test_strided_queries_and_caches():
    a = made(TWO, 16, 512, 1, 16, seed=16)
    want = csa.shared_attention(**a)
    q = torch.zeros(a["q"].shape[0], 16, 640, dtype=torch.bfloat16, device="cuda")
    q[..., 64:576] = a["q"]
    heads_first = torch.zeros(16, a["q"].shape[0], 512, dtype=torch.bfloat16, device="cuda")
    heads_first.copy_(a["q"].transpose(0, 1))
    cache = torch.full((*a["cache"].shape[:2], 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    cache[..., :512] = a["cache"]
    for b in (dict(a, q=q[..., 64:576]), dict(a, q=heads_first.transpose(0, 1)), dict(a, cache=cache[..., :512])):
        got = csa.shared_attention(**b)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("bits8", [False, True])
def test_streams_and_two_graphs(bits8):
    a = made([(700, [(64, 1), (30, 2), (1, 1), (90, 1)])], 64, 512, 1, 64, bits8, True, seed=17)
    b = made([(300, [(10, 1)] * 5)], 64, 512, 1, 64, bits8, True, seed=18)
    want, want_b = csa.shared_attention(**a), csa.shared_attention(**b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [csa.shared_attention(**x, stream=s) for x, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], want[0]) and torch.equal(got[1][0], want_b[0])
    graphs, results = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, x in zip(graphs, (a, b)):
        with torch.cuda.graph(g):
            results.append(csa.shared_attention(**x))
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(results[0][0], want[0]) and torch.equal(results[1][0], want_b[0])
    # lengths and groups are read on the device: a replay follows them
    a["seq_lens"] -= 30
    a["shared_rows"] -= 64
    a["cu_groups"][0] += 1
    graphs[0].replay()
    torch.cuda.synchronize()
    check(a, None, *results[0])


def test_finished_requests_in_front():
    # the group's first requests have no new tokens and no pages any more
    a = made([(700, [(0, 0), (0, 0), (30, 1), (64, 2), (5, 1)])], 64, 512, 1, 64, seed=22)
    a["block_table"][:2] = -1
    a["seq_lens"][:2] = 0
    check(a)
    # nobody has
    b = dict(a, q=a["q"][:0], cu_q=torch.zeros_like(a["cu_q"]))
    out, lse = csa.shared_attention(**b)
    assert out.shape == (0, 64, 512)
    b = dict(a, cu_q=torch.zeros_like(a["cu_q"]), out=torch.full_like(a["q"], 7.0))  # tokens of no request
    assert (csa.shared_attention(**b)[0] == 7).all()


def test_many_calls_at_once():
    sets = [made([(600 + 64 * k, [(30 + k, 1)] * (3 + k))], 64, 512 if k % 2 else 576, 1, 64, k == 3, True, seed=30 + k) for k in range(4)]
    want = [csa.shared_attention(**a, v_dim=512) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(6):
        got += [(k, csa.shared_attention(**a, v_dim=512, stream=s)) for k, (a, s) in enumerate(zip(sets, streams))]
    torch.cuda.synchronize()
    assert csa.csa_device_status() == 0
    for k, (out, lse) in got:
        assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])


def test_nothing_to_do():
    a = made(ONE, 16, 512, 1, 64, seed=19)
    out, lse = csa.shared_attention(**dict(a, q=a["q"][:0]))
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
    empty = torch.zeros((0, 64, 512), dtype=torch.bfloat16, device="cuda")
    out, lse = csa.shared_attention(**dict(a, cache=empty))  # no pages: nobody sees anything
    assert (out == 0).all() and torch.isinf(lse).all()
