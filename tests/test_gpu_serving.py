"""The serving operators together: the example's loop against a dense computation, and the norm's autograd function."""
import math
import os
import sys

import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa
from sparse_attention_kv_csa_gb300.autograd import rms_norm

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_example_prompts_and_steps_match_one_dense_computation():
    import serve_rows as ex
    heads, dim, prompts, steps = 4, 128, [37, 8, 3, 130], 9
    server = ex.Server(len(prompts), heads, dim, 8, 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    all_kv, all_score = [[] for _ in prompts], [[] for _ in prompts]
    for new in [prompts] + [[1] * len(prompts)] * steps + [[5, 1, 2, 7]]:
        kv, score, q = ex.inputs(sum(new), heads, dim, g)
        out = server.step(kv, score, q, new)
        at = 0
        for r, n in enumerate(new):
            all_kv[r].append(kv[at:at + n])
            all_score[r].append(score[at:at + n])
            at += n
        # dense: every request compressed from its first token, normed, quantised as the cache holds it
        at = 0
        for r, n in enumerate(new):
            k, sc = torch.cat(all_kv[r]), torch.cat(all_score[r])
            total = k.shape[0]
            rows = total // ex.RATIO
            if rows:
                cu = torch.tensor([0, total], dtype=torch.int32, device="cuda")
                cc = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
                c = csa.compress_forward(k, sc, server.ape, cu, cc, ex.RATIO, ex.COFF, dim, rows)
                q8, scale, _, _ = csa.rms_norm_forward(c, server.norm, out_dtype=torch.float8_e4m3fn)
                cache, scales = q8.view(1, rows, dim), scale.view(1, rows)
            else:
                cache = torch.zeros((1, 1, dim), device="cuda").to(torch.float8_e4m3fn)
                scales = torch.zeros((1, 1), device="cuda")
            want, _, tol, _ = u.attention64(q[at:at + n], cache, torch.zeros((1, 1), dtype=torch.int32), torch.tensor([0, n]),
                                            torch.tensor([total]), ex.RATIO, 1 / math.sqrt(dim), dim, scales, server.sink)
            assert ((out[at:at + n].cpu().double() - want).abs() <= tol).all()
            at += n
    assert server.taken.item() == sum(-(-(n // ex.RATIO) // 8) for n in server.lens)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("use", ["both", "out", "total"])
def test_norm_autograd(residual, use):
    if use != "out" and not residual:
        pytest.skip("no second output")
    g = torch.Generator(device="cuda").manual_seed(4)
    leaf = lambda *s: torch.randn(s, device="cuda", generator=g).requires_grad_()  # noqa: E731
    x, w = leaf(2, 3, 64), leaf(64)
    r = leaf(2, 3, 64) if residual else None
    a, b = torch.randn(2, 3, 64, device="cuda", generator=g), torch.randn(2, 3, 64, device="cuda", generator=g)

    def loss(out, total):
        return (0 if use == "total" else (out * a).sum()) + (0 if use == "out" else (total * b).sum())

    got = rms_norm(x, w, r, 1e-5)
    leaves = [t for t in (x, w, r) if t is not None]
    grads = torch.autograd.grad(loss(*(got if residual else (got, None))), leaves, allow_unused=True)
    ref = [t.detach().double().requires_grad_() for t in leaves]
    h = ref[0] + (ref[2] if residual else 0)
    y = h * (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * ref[1]
    want = torch.autograd.grad(loss(y, h), ref, allow_unused=True)
    for p, q in zip(grads, want):
        if q is None:
            assert p is None
        else:
            assert (p.double() - q).abs().max() <= 1e-5 * q.abs().max()


def test_norm_forward_and_backward_captured_while_an_eager_graph_lives():
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((33, 512), device="cuda", generator=g).bfloat16().requires_grad_()
    w = torch.ones(512, device="cuda", requires_grad=True)
    eager = rms_norm(x, w).float().square().sum()  # kept alive across the capture
    want = torch.autograd.grad(eager, [x, w], retain_graph=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xs, ws = x.detach().clone().requires_grad_(), w.detach().clone().requires_grad_()
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(rms_norm(xs, ws).float().square().sum(), [xs, ws])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(rms_norm(xs, ws).float().square().sum(), [xs, ws])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isfinite(eager)
