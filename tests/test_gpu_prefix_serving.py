"""A layer's serving step with the operators as they are used together: layer norm of the residual stream, rows appended to the
cache with the rotation (queries beside them), attention of requests behind one prompt, the output turned back; against the same in
64 bits from what each step was given."""
import math

import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa

pytestmark = pytest.mark.gpu

LATENT, ROT, HEADS, PAGE = 192, 64, 64, 16


def step(s, out=None):
    """The calls of one step; what a program has between them (projections) is a fixed product."""
    normed, stream, _, _ = csa.layer_norm_forward(s["x"], s["weight"], s["bias"], 1e-5, residual=s["residual"])
    rows, part = (normed @ s["down"]).split([LATENT, ROT], 1)
    q = (normed @ s["up"]).view(-1, HEADS, LATENT + ROT)
    csa.append_rows(rows, s["positions"], s["table"], s["slots"], s["cache"].view(-1, LATENT + ROT), scales=s["flat_scales"],
                    rotary=part, interleaved=True, queries=q[..., LATENT:], query_out=q[..., LATENT:])
    y, lse = csa.shared_attention(q, s["cache"], s["block_table"], s["cu_q"], s["seq_lens"], s["cu_groups"], s["shared_rows"], 1,
                                  1 / math.sqrt(LATENT + ROT), row_scales=s["scales"], sink=s["sink"])
    back = csa.rotate(y[..., LATENT:], s["positions"], s["table"], interleaved=True, inverse=True)
    return dict(normed=normed, stream=stream, rows=rows, part=part, q=q, y=y, lse=lse, back=back)


def made(bits8, requests=40, prefix=1000, dim=512):
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *a: torch.randn(a, device="cuda", generator=g)  # noqa: E731
    width, shared = LATENT + ROT, prefix // PAGE
    behind = [5 + 7 * k % 90 for k in range(requests)]  # rows behind the prefix before the step
    used = [-(-(prefix + b + 1) // PAGE) for b in behind]
    pages = shared + sum(n - shared for n in used) + 2
    ids = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((requests, 20000), -1, dtype=torch.int32, device="cuda")
    table[:, :shared] = ids[:shared]
    at = shared
    for r, n in enumerate(used):
        table[r, shared:n] = ids[at:at + n - shared]
        at += n - shared
    rows = randn(pages, PAGE, width)
    if prefix % PAGE:  # each request's own copy of the prefix's last rows
        rows[table[1:, shared].long(), :prefix % PAGE] = rows[table[0, shared].long(), :prefix % PAGE]
    int32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(x=randn(requests, dim).bfloat16(), residual=randn(requests, dim).bfloat16(), weight=1 + 0.1 * randn(dim), bias=0.1 * randn(dim),
             down=(randn(dim, width) / math.sqrt(dim)).bfloat16(), up=(randn(dim, HEADS * width) / math.sqrt(dim)).bfloat16(),
             table=csa.rotation_table(4096, ROT), positions=int32([prefix + b for b in behind]), block_table=table,
             cu_q=int32(list(range(requests + 1))), seq_lens=int32([prefix + b + 1 for b in behind]), cu_groups=int32([0, requests]),
             shared_rows=int32([prefix]), sink=randn(HEADS))
    s["slots"] = torch.stack([table[r, (prefix + b) // PAGE].long() * PAGE + (prefix + b) % PAGE for r, b in enumerate(behind)])
    if bits8:
        s["scales"] = rows.abs().amax(2) / 448
        s["cache"] = (rows / s["scales"][..., None]).to(torch.float8_e4m3fn)
    else:
        s["cache"], s["scales"] = rows.bfloat16(), None
    s["flat_scales"] = s["scales"].view(-1) if bits8 else None
    return s


@pytest.mark.parametrize("bits8", [False, True])
def test_step(bits8):
    s = made(bits8)
    r = step(s)
    torch.cuda.synchronize()
    assert csa.csa_device_status() == 0
    half = 2.0 ** -8  # a bf16 rounding
    # the norm
    h = (s["x"].float() + s["residual"].float()).bfloat16()
    assert torch.equal(r["stream"], h)
    h = h.double()
    unit = (h - h.mean(1, keepdim=True)) * torch.rsqrt(h.var(1, unbiased=False, keepdim=True) + 1e-5)
    want = unit * s["weight"].double() + s["bias"].double()
    assert ((r["normed"].double() - want).abs() <= half * want.abs() + 2.0 ** -18 * (unit.abs() + 1)).all()
    # the appended rows, turned by their positions
    turn = torch.polar(torch.ones((40, ROT // 2), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] * 10000.0 ** (-torch.arange(ROT // 2, device="cuda", dtype=torch.float64) / (ROT // 2)))
    part = torch.view_as_complex(r["part"].double().unflatten(-1, (-1, 2)).contiguous())
    want = torch.cat([r["rows"].double(), torch.view_as_real(part * turn).flatten(-2)], 1)
    got = s["cache"].view(-1, LATENT + ROT)[s["slots"]] if not bits8 else s["cache"].view(torch.uint8).view(-1, LATENT + ROT)[s["slots"]].view(
        torch.float8_e4m3fn)
    got = got.double()
    top = want.abs().amax(1, keepdim=True)
    if bits8:
        got = got * s["flat_scales"][s["slots"]].double()[:, None]
        # e4m3: half a step of 2^-4, or of its least number's 2^-10 of the scale; fp32 around it
        assert ((got - want).abs() <= (2.0 ** -4 + 2.0 ** -16) * want.abs() + (2.0 ** -10 + 2.0 ** -16) * top / 448 + 2.0 ** -20 * top).all()
    else:
        assert ((got - want).abs() <= half * want.abs() + 2.0 ** -20 * top).all()
    # the attention over what the cache now holds, and its output turned back
    want, want_lse, tol, tol_lse = u.attention64(r["q"], s["cache"], s["block_table"], s["cu_q"].cpu(), s["seq_lens"].cpu(), 1,
                                                 1 / math.sqrt(LATENT + ROT), LATENT + ROT, s["scales"], s["sink"])
    assert ((r["y"].cpu().double() - want).abs() <= tol).all() and ((r["lse"].cpu().double() - want_lse).abs() <= tol_lse).all()
    y = torch.view_as_complex(r["y"][..., LATENT:].double().unflatten(-1, (-1, 2)).contiguous())
    want = torch.view_as_real(y * turn.conj()[:, None]).flatten(-2)
    assert ((r["back"].double() - want).abs() <= half * want.abs() + 2.0 ** -20 * y.abs().amax()).all()


def test_captured_steps_give_what_single_ones_do():
    s = made(True)
    first = {k: v.clone() for k, v in step(s).items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step(s)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert csa.csa_device_status() == 0
    for k, v in first.items():
        assert torch.equal(again[k], v), k
