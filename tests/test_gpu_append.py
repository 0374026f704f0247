"""append_rows and rotate against 64 bits.

A rotated value a cos - b sin has at most three fp32 roundings: 3 2^-24 (|a cos| + |b sin|), then one to its type; the table's
fp32 values are the definition's.  8-bit rows as in the norm: half a step, 2^-4 of the value or 2^-10 of the scale."""
import pytest
import torch

import serving_util as util
import sparse_attention_kv_csa_gb300 as csa
from sparse_attention_kv_csa_gb300.autograd import rotate as rotate_grad

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def turned(x, table, positions, interleaved, inverse=False):
    """(value, bound) of x [..., rot] in 64 bits; positions broadcast over the heads."""
    half = x.shape[-1] // 2
    t = table.double()[positions.long()]
    t = t.view(t.shape[0], *([1] * (x.dim() - 2)), t.shape[1])
    cos, sin = t[..., :half], t[..., half:] * (-1 if inverse else 1)
    x = x.double()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    join = (lambda p, q: torch.stack([p, q], -1).flatten(-2)) if interleaved else (lambda p, q: torch.cat([p, q], -1))
    size = join((a * cos).abs() + (b * sin).abs(), (a * sin).abs() + (b * cos).abs())
    return join(a * cos - b * sin, a * sin + b * cos), 3 * U * size


def near(got, want, tol, dtype):
    return ((got.double() - want).abs() <= tol + util.HALF[dtype] * (want.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0)).all()


def test_table():
    t = csa.rotation_table(70000, 64, 10000.0).double()
    p = torch.tensor([0, 1, 4095, 69999], device="cuda")
    angle = p.double()[:, None] * 10000.0 ** (-torch.arange(32, device="cuda").double() / 32)
    assert (t[p] - torch.cat([angle.cos(), angle.sin()], 1)).abs().max() <= 2.0 ** -25 + 1e-9


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,rot", [(1, 1, 2), (1, 64, 64), (3, 5, 6), (77, 16, 64), (33, 3, 48), (9, 1, 1024), (5, 7, 130), (2, 24, 32),
                                         (300, 64, 128), (4, 2, 1022)])
def test_rotate(dtype, interleaved, n, heads, rot):
    table = csa.rotation_table(5000, rot)
    x = randn((n, heads, rot), dtype, 1)
    positions = torch.randint(0, 5000, (n,), generator=torch.Generator().manual_seed(2)).int().cuda()
    for inverse in (False, True):
        out = csa.rotate(x, positions, table, interleaved=interleaved, inverse=inverse)
        want, tol = turned(x, table, positions, interleaved, inverse)
        assert out.dtype == dtype and near(out, want, tol, dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("first,rot", [(64, 64), (8, 32), (1, 64), (3, 30), (448, 64)])
def test_strided_heads_and_in_place(interleaved, first, rot):
    x = randn((21, 8, 512), torch.bfloat16, 3)
    table, positions = csa.rotation_table(100, rot), torch.arange(21, dtype=torch.int32, device="cuda")
    view = x[..., first:first + rot]
    want, tol = turned(view, table, positions, interleaved)
    out = torch.zeros(21, 8, rot + 40, dtype=torch.bfloat16, device="cuda")
    csa.rotate(view, positions, table, interleaved=interleaved, out=out[..., 8:8 + rot])
    assert near(out[..., 8:8 + rot], want, tol, x.dtype) and (out[..., :8] == 0).all() and (out[..., 8 + rot:] == 0).all()
    before = x.clone()
    assert csa.rotate(view, positions, table, interleaved=interleaved, out=view) is view
    assert near(view, want, tol, x.dtype)
    keep = torch.ones(512, dtype=torch.bool)
    keep[first:first + rot] = False
    assert torch.equal(x[..., keep], before[..., keep])
    # heads before tokens
    t = randn((8, 21, rot), torch.bfloat16, 4).transpose(0, 1)
    want, tol = turned(t, table, positions, interleaved)
    assert near(csa.rotate(t, positions, table, interleaved=interleaved), want, tol, t.dtype)


def test_positions_past_the_table_give_nan():
    table = csa.rotation_table(10, 64)
    x = randn((4, 2, 64), torch.bfloat16, 5)
    positions = torch.tensor([9, 10, -1, 1 << 30], dtype=torch.int32, device="cuda")
    out = csa.rotate(x, positions, table)
    want, tol = turned(x[:1], table, positions[:1], False)
    assert near(out[:1], want, tol, x.dtype) and out[1:].isnan().all()
    store = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    rows = randn((4, 128), torch.bfloat16, 6)
    csa.append_rows(rows, positions, table, torch.arange(4, device="cuda"), store)
    assert torch.equal(store[:, :64], rows[:, :64]) and store[1:, 64:].isnan().all() and store[0].isfinite().all()


SHAPES = [(1, 512, 64, True), (37, 512, 64, True), (37, 512, 64, False), (300, 448, 64, False), (5, 64, 64, True), (9, 100, 30, True),
          (9, 7, 6, False), (4, 1024, 128, True), (4, 960, 64, False), (3, 1, 2, False), (6, 512, 512, True), (50, 192, 48, True),
          (12, 33, 32, True), (12, 1023, 64, True), (700, 576, 64, True)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,dim,rot,inside", SHAPES)
@pytest.mark.parametrize("bits8", [False, True])
def test_append(dtype, interleaved, n, dim, rot, inside, bits8):
    table = csa.rotation_table(3000, rot)
    g = torch.Generator().manual_seed(7)
    positions = torch.randint(0, 3000, (n,), generator=g).int().cuda()
    rows, part = randn((n, dim), dtype, 8), None if inside else randn((n, rot), dtype, 9)
    if n > 4:
        rows[2] = 0
        if part is not None:
            part[2] = 0
    total = n + 9
    slots = torch.randperm(total, generator=g)[:n].cuda()
    if n > 4:
        slots[1], slots[3] = -1, total  # nowhere
    keep = (slots >= 0) & (slots < total)
    width = dim if inside else dim + rot
    if bits8:
        store = torch.full((total, width), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.full((total,), -7.0, device="cuda")
    else:
        store, scales = torch.full((total, width), -3.0, dtype=dtype, device="cuda"), None
    got = csa.append_rows(rows, positions, table, slots, store, scales=scales, rotary=part, interleaved=interleaved)
    assert got[0] is store and got[1] is scales and got[2] is None
    plain, last = (rows[:, :dim - rot], rows[:, dim - rot:]) if inside else (rows, part)
    want, tol = turned(last, table, positions, interleaved)
    want, tol = torch.cat([plain.double(), want], 1)[keep], torch.cat([torch.zeros_like(plain).double(), tol], 1)[keep]
    touched = torch.zeros(total, dtype=torch.bool, device="cuda")
    touched[slots[keep]] = True
    if not bits8:
        out = store[slots[keep]]
        assert torch.equal(out[:, :width - rot], plain[keep]) and near(out, want, tol, dtype) and (store[~touched] == -3).all()
        return
    s = scales[slots[keep]].double()
    top = want.abs().amax(1) / 448
    assert ((s - top).abs() <= 8 * U * top + tol.amax(1) / 448).all()
    out = store.view(torch.uint8)[slots[keep]].view(torch.float8_e4m3fn).double() * s[:, None]
    assert ((out - want).abs() <= (2.0 ** -4 + 32 * U) * want.abs() + (2.0 ** -10 + 32 * U) * top[:, None] + 2 * tol).all()
    if n > 4:
        assert scales[slots[2]] == 0 and (store.view(torch.uint8)[slots[2]] & 0x7f == 0).all()
    assert (store.view(torch.uint8)[~touched] == 0x55).all() and (scales[~touched] == -7).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,tokens,heads", [(64, 64, 64), (3, 12, 5), (0, 7, 3), (5, 0, 2)])
def test_queries_beside_rows(interleaved, dtype, n, tokens, heads):
    rot, table = 64, csa.rotation_table(2000, 64)
    g = torch.Generator().manual_seed(10)
    positions, q_positions = torch.randint(0, 2000, (n,), generator=g).int().cuda(), torch.randint(0, 2000, (tokens,), generator=g).int().cuda()
    latent = randn((n, 576 + 8), dtype, 11)
    rows, part, q = latent[:, :512], latent[:, 512:576], randn((tokens, heads, 192), dtype, 12)
    store, wide = torch.zeros(n + 3, 576, dtype=dtype, device="cuda"), torch.zeros(tokens, heads, 576, dtype=dtype, device="cuda")
    slots = torch.randperm(n + 3, generator=g)[:n].cuda()
    _, _, out = csa.append_rows(rows, positions, table, slots, store, rotary=part, interleaved=interleaved, queries=q[..., 128:],
                                query_positions=q_positions, query_out=wide[..., 512:])
    want, tol = turned(q[..., 128:], table, q_positions, interleaved)
    assert near(wide[..., 512:], want, tol, dtype) and (wide[..., :512] == 0).all() and out.data_ptr() == wide[..., 512:].data_ptr()
    want, tol = turned(part, table, positions, interleaved)
    assert torch.equal(store[slots][:, :512], rows) and near(store[slots][:, 512:], want, tol, dtype)
    if n == tokens:  # positions by default, a new tensor by default
        again = csa.append_rows(rows, positions, table, slots, store, rotary=part, interleaved=interleaved, queries=q[..., 128:])[2]
        want, tol = turned(q[..., 128:], table, positions, interleaved)
        assert again.shape == (tokens, heads, rot) and near(again, want, tol, dtype)


def test_special_values():
    table = csa.rotation_table(10, 8)
    rows = randn((4, 16), torch.bfloat16, 13)
    rows[0, 3], rows[1, 2], rows[2, 9] = float("nan"), float("inf"), float("nan")
    positions, slots = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.arange(4, device="cuda")
    store = torch.zeros(4, 16, device="cuda").to(torch.float8_e4m3fn)
    scales = torch.zeros(4, device="cuda")
    csa.append_rows(rows, positions, table, slots, store, scales=scales)
    assert scales[0].isnan() and scales[1].isinf() and scales[2].isnan() and scales[3].isfinite()
    tiny = torch.full((1, 16), 1e-38, device="cuda")
    csa.append_rows(tiny, positions[:1], table, slots[:1], store, scales=scales)
    assert ((store[0].float() * scales[0] - 1e-38).abs() <= 2.0 ** -4 * 1e-38).all()


def test_far_rows_and_large_offsets():
    # a cache past 2^32 bytes: 8.4 million rows of 512 bytes; rows of fp32 whose strides pass 2^31 bytes
    table = csa.rotation_table(200000, 64)
    store = torch.zeros((8500000, 512), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros(8500000, device="cuda")
    rows = randn((3, 512), torch.bfloat16, 14)
    positions = torch.tensor([0, 150000, 199999], dtype=torch.int32, device="cuda")
    slots = torch.tensor([8499999, 0, 8400001], device="cuda")
    csa.append_rows(rows, positions, table, slots, store, scales=scales)
    want, tol = turned(rows[:, 448:], table, positions, False)
    for i, s in enumerate(slots.tolist()):
        got = store[s].double() * scales[s].double()
        full = torch.cat([rows[i, :448].double(), want[i]])
        assert ((got - full).abs() <= (2.0 ** -4 + 32 * U) * full.abs() + (2.0 ** -10 + 32 * U) * scales[s] + 1e-5).all()
    assert scales.count_nonzero() == 3


def test_rotate_autograd():
    table, positions = csa.rotation_table(50, 32), torch.tensor([0, 7, 49], dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        for inverse in (False, True):
            x = randn((3, 4, 32), torch.float32, 15).requires_grad_()
            g = randn((3, 4, 32), torch.float32, 16)
            out = rotate_grad(x, positions, table, interleaved, inverse)
            grad, = torch.autograd.grad(out, x, g)
            want, tol = turned(g, table, positions, interleaved, not inverse)
            assert near(grad, want, tol, torch.float32)
            # against differences
            d = torch.zeros_like(x)
            d[1, 2, 5] = 0.5
            hi, lo = turned(x.detach() + d, table, positions, interleaved, inverse)[0], turned(x.detach() - d, table, positions, interleaved, inverse)[0]
            assert abs(((hi - lo) * g.double()).sum().item() - grad[1, 2, 5].item()) <= 1e-5
    x = randn((3, 4, 32), torch.float32, 15).requires_grad_()
    grad, = torch.autograd.grad(rotate_grad(x, positions, table).sum(), x)  # an expanded gradient
    assert near(grad, *turned(torch.ones_like(x), table, positions, False, True), torch.float32)


def test_side_stream_and_graph():
    table = csa.rotation_table(3000, 64)
    rows, q = randn((129, 512), torch.bfloat16, 17), randn((129, 16, 64), torch.bfloat16, 18)
    positions, slots = torch.arange(129, dtype=torch.int32, device="cuda"), torch.arange(129, device="cuda").flip(0)

    def call(store, **kw):
        return csa.append_rows(rows, positions, table, slots, store, queries=q, **kw)[2]

    store = torch.zeros(129, 512, dtype=torch.bfloat16, device="cuda")
    want = call(store)
    torch.cuda.synchronize()
    s, other = torch.cuda.Stream(), torch.zeros_like(store)
    torch.cuda.synchronize()
    got = call(other, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(other, store)
    g, third = torch.cuda.CUDAGraph(), torch.zeros_like(store)
    with torch.cuda.graph(g):
        out = call(third)
        back = csa.rotate(out, positions, table, inverse=True)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(third, store)
    assert ((back.float() - q.float()).abs() <= 2.0 ** -7 * (q.float().abs() + q.float().roll(32, 2).abs()) + 1e-6).all()
