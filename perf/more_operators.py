"""More serving and training operators' cases: what is measured, in plain torch operations and through the package.

The operators are the layer norm and its gradient, the append of rows to a paged cache with the position rotation on the
way (queries rotated beside it), the rotation alone, and the attention of a batch whose requests share a prefix.

Kinds of cases:
  norm     layer_norm_forward: residual addition, mean and variance, weight and bias
  grad     layer_norm_backward: the inputs' gradient, the weight's and the bias's
  append   append_rows: rows (their last columns rotated) to cache slots, bf16 or 8 bits; queries rotated beside them
  rotate   rotate, backwards or forwards, over part of each head
  shared   shared_attention over the paged cache, bf16 or 8-bit rows
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
BASE = 10000.0


def listed():
    return [
        # one token's residual stream in a decode step: latency
        dict(name="layer_token", kind="norm", rows=1, dim=4096, residual=True, type="bf16"),
        # a prompt's residual stream
        dict(name="layer_stream", kind="norm", rows=16411, dim=4096, residual=True, type="bf16"),
        # training: the gradient over a batch's residual stream
        dict(name="layer_grad_stream", kind="grad", rows=16384, dim=4096, residual=True, type="bf16"),
        # training: the gradient over rows of an odd width in fp16
        dict(name="layer_grad_odd", kind="grad", rows=5003, dim=1001, residual=False, type="f16"),
        # a decode step of 64 requests: latents of 512 columns and a rotary key of 64 to one row of 576, the queries of
        # 64 heads beside them
        dict(name="append_decode", kind="append", rows=64, dim=512, rotary=64, inside=False, bits8=False, tokens=64, heads=64,
             interleaved=True),
        # a long prompt's rows into an 8-bit cache, the last 64 of 512 columns rotated, no queries
        dict(name="append_rows8", kind="append", rows=65543, dim=512, rotary=64, inside=True, bits8=True, tokens=0, heads=1,
             interleaved=False),
        # the attention's output of a prompt of 4099 tokens turned back, the last 64 of 512 columns of 64 heads
        dict(name="rotate_back", kind="rotate", tokens=4099, heads=64, dim=512, rotary=64, inverse=True, interleaved=True),
        # a small batch behind one prompt: latency
        dict(name="shared_few", kind="shared", groups=1, requests=5, prefix=2048, most=256, new=1, heads=16, dim=576, vdim=512,
             ratio=1, page=64, bits8=False, sink=False),
        # a decode step of 128 requests behind one system prompt of 16384 tokens (4096 rows)
        dict(name="shared_decode", kind="shared", groups=1, requests=128, prefix=16384, most=4096, new=1, heads=64, dim=512,
             vdim=512, ratio=4, page=64, bits8=False, sink=True),
        # ragged groups behind three prompts, 128 heads over 8-bit rows
        dict(name="shared_groups8", kind="shared", groups=3, requests=97, prefix=12000, most=2000, new=1, heads=128, dim=512,
             vdim=512, ratio=4, page=64, bits8=True, sink=True),
        # speculative steps of up to three tokens, 16 heads, small pages, every token a row of 576
        dict(name="shared_steps", kind="shared", groups=2, requests=201, prefix=6000, most=500, new=3, heads=16, dim=576,
             vdim=512, ratio=1, page=16, bits8=False, sink=False),
        # a large batch behind one long document
        dict(name="shared_large", kind="shared", groups=1, requests=512, prefix=32768, most=2048, new=1, heads=64, dim=512,
             vdim=512, ratio=4, page=64, bits8=False, sink=True),
    ]


def _between(rng, low, high):
    """A whole number of [low, high], spread over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["norm", "grad", "append", "rotate", "shared", "shared", "shared"])
    if kind in ("norm", "grad"):
        dim = rng.choice([128, 512, 576, 1000, 1001, 2048, 4096, 4100, _between(rng, 64, 8192)])
        return dict(kind=kind, rows=_between(rng, 1, max(1, 16384 * 4096 // max(dim, 4096))), dim=dim, residual=rng.random() < 0.5,
                    type=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if kind == "append":
        inside = rng.random() < 0.5
        dim = rng.choice([128, 192, 256, 512, 512, 1024])
        rotary = rng.choice([32, 64, 64, 128, 48])
        rows = _between(rng, 1, 65543)
        with_queries = rng.random() < 0.5 and rows <= 8192
        return dict(kind="append", rows=rows, dim=dim, rotary=rotary, inside=inside, bits8=rng.random() < 0.5,
                    tokens=rows if with_queries else 0, heads=rng.choice([1, 16, 24, 64]), interleaved=rng.random() < 0.5)
    if kind == "rotate":
        heads = rng.choice([1, 8, 16, 24, 64, 128])
        rotary = rng.choice([32, 64, 64, 128, 48])
        return dict(kind="rotate", tokens=_between(rng, 1, 4099 * 64 // max(heads, 32)), heads=heads,
                    dim=rng.choice([rotary, 192, 512]), rotary=rotary, inverse=rng.random() < 0.5, interleaved=rng.random() < 0.5)
    dim, vdim = rng.choice([(512, 512), (512, 512), (576, 512), (256, 256), (128, 128), (192, 128)])
    heads = rng.choice([8, 16, 24, 64, 128])
    ratio = rng.choice([1, 4, 4, 16])
    new = rng.choice([1, 1, 1, 2, 4])
    requests = _between(rng, 2, max(2, 16384 // (heads * new)))
    case = dict(kind="shared", groups=min(requests, rng.choice([1, 1, 2, 5])), requests=requests,
                prefix=ratio * _between(rng, 64, 8192), most=ratio * _between(rng, 16, max(16, min(1024, 100000 // requests))) + new,
                new=new, heads=heads, dim=dim, vdim=vdim, ratio=ratio, page=rng.choice([16, 64, 64, 128, 50]),
                bits8=rng.random() < 0.3, sink=rng.random() < 0.5)
    while work(case)["flops"] > 5e11:
        case["prefix"] //= 2
    return case


# ---------------------------------------------------------------- inputs

def _lengths(case, seed):
    """What a shared case's requests hold: (first request of each group and the end, prefix tokens of each group, tokens of each
    request behind its prefix, new tokens of each).  Groups and new tokens go by the case alone, so that the outputs'
    shapes do."""
    n, groups, new = case["requests"], case["groups"], case["new"]
    rng = random.Random(n * 31 + new)
    cuts = sorted(rng.sample(range(1, n), groups - 1)) if groups > 1 else []
    news = [rng.randint(max(1, new // 2), new) for _ in range(n)]
    rng = random.Random(seed * 7919 + 17)
    # the first group has the longest prefix; prefixes end inside a block of the compression too
    prefix = [case["prefix"]] + [rng.randint(case["prefix"] // 2, case["prefix"]) for _ in range(groups - 1)]
    behind = [rng.randint(max(b, case["most"] // 8), max(b, case["most"])) for b in news]
    return [0] + cuts + [n], prefix, behind, news


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g):
    return torch.randn(shape, device="cuda", generator=g)


def _angles(case):
    half = case["rotary"] // 2
    frequency = BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    at = torch.arange(131072, device="cuda", dtype=torch.float64)[:, None] * frequency
    return torch.cat([at.cos(), at.sin()], 1).float()


def prepare(case, seed):
    g = _generator(seed)
    state = {"case": case}
    if case["kind"] in ("norm", "grad"):
        n, d = case["rows"], case["dim"]
        dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[case["type"]]
        # a residual stream has a few columns far larger than the rest, and an offset
        x = _randn((n, d), g) * torch.exp(0.5 * _randn((d,), g)) + 0.5
        state["x"] = x.to(dtype)
        state["weight"], state["bias"] = 1 + 0.2 * _randn((d,), g), 0.1 * _randn((d,), g)
        state["eps"] = 1e-5
        if case["kind"] == "grad":
            x = state["x"].double()
            state["mean"] = x.mean(1).float()
            state["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + 1e-5).float()
            state["dy"] = (0.01 * _randn((n, d), g)).to(dtype)
            state["dh"] = (0.01 * _randn((n, d), g)).to(dtype) if case["residual"] else None
        else:
            state["residual"] = _randn((n, d), g).to(dtype) if case["residual"] else None
        return state
    if case["kind"] == "append":
        n, d, rot = case["rows"], case["dim"], case["rotary"]
        state["rotation"] = _angles(case)
        # prompts and single tokens of many requests: positions run on within a stretch
        start = torch.randint(0, 65000, (n // 512 + 1,), device="cuda", generator=g)
        at = torch.arange(n, device="cuda")
        state["positions"] = (start[at // 512] + at % 512).int()
        state["rows"] = _randn((n, d), g).bfloat16()
        state["part"] = None if case["inside"] else _randn((n, d + rot), g).bfloat16()[:, d:]
        width = d if case["inside"] else d + rot
        total = n + n // 2 + 64
        slots = torch.randperm(total, device="cuda", generator=g)[:n]
        state["slots"] = torch.where(torch.rand(n, device="cuda", generator=g) < 0.01, -1, slots)
        # one row past the cache, where the plain form puts rows that have no slot
        state["store"] = torch.zeros((total + 1, width), dtype=torch.uint8 if case["bits8"] else torch.bfloat16, device="cuda")
        if case["bits8"]:
            state["store"] = state["store"].view(torch.float8_e4m3fn)
            state["store_scales"] = torch.zeros(total + 1, device="cuda")
        if case["tokens"]:
            # the projection gives a head's plain and rotary columns side by side; the attention's queries are wider
            q = _randn((case["tokens"], case["heads"], 128 + rot), g).bfloat16()
            state["q"] = q[..., 128:]
            state["q_wide"] = torch.zeros((case["tokens"], case["heads"], width), dtype=torch.bfloat16, device="cuda")
        return state
    if case["kind"] == "rotate":
        state["rotation"] = _angles(case)
        state["x"] = _randn((case["tokens"], case["heads"], case["dim"]), g).bfloat16()
        state["positions"] = torch.randint(0, 131072 - case["tokens"], (1,), device="cuda", generator=g).int() + torch.arange(
            case["tokens"], device="cuda", dtype=torch.int32)
        return state
    cuts, prefix, behind, news = _lengths(case, seed)
    page, ratio, d, h, n = case["page"], case["ratio"], case["dim"], case["heads"], case["requests"]
    group = [g_ for g_ in range(case["groups"]) for _ in range(cuts[g_], cuts[g_ + 1])]
    lens = [prefix[group[r]] + behind[r] for r in range(n)]
    # a prefix's pages are shared as far as they are whole; its last page's rows are each request's own copy
    shared_pages = [p // ratio // page for p in prefix]
    used = [-(-(a // ratio) // page) for a in lens]
    mine = [u - shared_pages[group[r]] for r, u in enumerate(used)]
    n_pages = sum(shared_pages) + sum(mine) + 3
    ids = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((n, max(used + [1])), -1, dtype=torch.int32)
    at = 0
    for k, count in enumerate(shared_pages):
        table[cuts[k]:cuts[k + 1], :count] = ids[at:at + count]
        at += count
    for r in range(n):
        table[r, used[r] - mine[r]:used[r]] = ids[at:at + mine[r]]
        at += mine[r]
    state["table"] = table.cuda()
    rows = torch.randn((n_pages, page, d), device="cuda", generator=g, dtype=torch.bfloat16)
    if case["bits8"]:
        scales = rows.float().abs().amax(2) / E4M3_MAX
        state["cache"] = (rows.float() / scales[..., None]).to(torch.float8_e4m3fn)
        state["scales"] = scales.contiguous()
    else:
        state["cache"], state["scales"] = rows, None
    state["q"] = (1.5 * _randn((sum(news), h, d), g)).bfloat16()
    cu = [0]
    for b in news:
        cu.append(cu[-1] + b)
    state["cu_q"], state["lens"], state["cu_groups"] = _int32(cu), _int32(lens), _int32(cuts)
    state["shared_rows"] = _int32([p * page for p in shared_pages])
    state["sink"] = _randn((h,), g) if case["sink"] else None
    state["cuts"], state["shared"], state["longest"] = cuts, [p * page for p in shared_pages], max(news)
    state["widest"] = max(b // ratio + 2 + page for b in behind)
    return state


# ---------------------------------------------------------------- plain forms

def _norm_plain(s):
    dtype = s["x"].dtype
    x = s["x"].float()
    stream = None
    if s["residual"] is not None:
        stream = (x + s["residual"].float()).to(dtype)
        x = stream.float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"])
    answer = {"out": (x * rstd * s["weight"] + s["bias"]).to(dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if stream is not None:
        answer["stream"] = stream
    return answer


def _grad_plain(s):
    h, dy = s["x"].float(), s["dy"].float()
    unit = (h - s["mean"][:, None]) * s["rstd"][:, None]
    wdy = dy * s["weight"]
    dx = s["rstd"][:, None] * (wdy - wdy.mean(1, keepdim=True) - unit * (wdy * unit).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * unit).sum(0), "dbias": dy.sum(0)}


def _turned(x, angles, interleaved, inverse):
    """x [..., rot] in fp32, angles [..., rot] (cosines, then sines, of the pairs)."""
    half = x.shape[-1] // 2
    cos, sin = angles[..., :half], angles[..., half:]
    if inverse:
        sin = -sin
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _append_plain(s):
    case = s["case"]
    rot = case["rotary"]
    angles = s["rotation"][s["positions"].long()]
    rows = s["rows"].float()
    plain, part = (rows[:, :-rot], rows[:, -rot:]) if s["part"] is None else (rows, s["part"].float())
    y = torch.cat([plain, _turned(part, angles, case["interleaved"], False)], 1)
    at = torch.where(s["slots"] < 0, s["store"].shape[0] - 1, s["slots"])
    answer = {}
    if case["bits8"]:
        scales = y.abs().amax(1) / E4M3_MAX
        step = torch.where(scales > 0, scales, torch.ones_like(scales))
        s["store"].view(torch.uint8)[at] = (y / step[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["store_scales"][at] = scales
        answer["scales"] = s["store_scales"][:-1]
    else:
        s["store"][at] = y.bfloat16()
    answer["out"] = s["store"][:-1]
    if case["tokens"]:
        s["q_wide"][..., -rot:] = _turned(s["q"].float(), angles[:, None], case["interleaved"], False).bfloat16()
        answer["q"] = s["q_wide"]
    return answer


def _rotate_plain(s):
    case = s["case"]
    angles = s["rotation"][s["positions"].long()]
    return _turned(s["x"][..., -case["rotary"]:].float(), angles[:, None], case["interleaved"], case["inverse"]).bfloat16()


def _rows_of(s, ids):
    if s["scales"] is None:
        return s["cache"][ids].float().flatten(-3, -2)
    rows = s["cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
    return (rows * s["scales"][ids][..., None]).flatten(-3, -2)


def _shared_plain(s):
    """The prefix's logits for all of a group's queries in one product, each request's own rows in a padded batch, and one softmax
    over the two."""
    case = s["case"]
    h, d, ratio, page, vdim, longest = case["heads"], case["dim"], case["ratio"], case["page"], case["vdim"], s["longest"]
    scale = 1 / math.sqrt(d)
    table = s["table"].long().clamp(min=0)
    begin, count = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    i = torch.arange(longest, device="cuda")
    outs, lses = [], []
    for k, shared in enumerate(s["shared"]):
        r0, r1 = s["cuts"][k], s["cuts"][k + 1]
        n = r1 - r0
        q = s["q"][(begin[r0:r1, None] + i).clamp(max=s["q"].shape[0] - 1)].float().view(n, longest * h, d)
        pages = shared // page
        prefix = _rows_of(s, table[r0, :pages])
        one = torch.matmul(q.view(-1, d), prefix.T).mul_(scale).view(n, longest, h, -1)
        rows = _rows_of(s, table[r0:r1, pages:pages + -(-s["widest"] // page)])
        seen = torch.div((s["lens"][r0:r1].long() - count[r0:r1])[:, None] + i + 1, ratio, rounding_mode="floor") - shared
        hidden = torch.arange(rows.shape[1], device="cuda")[None, None] >= seen[..., None]
        two = torch.matmul(q, rows.transpose(1, 2)).mul_(scale).view(n, longest, h, -1)
        two.masked_fill_(hidden[:, :, None], -math.inf)
        sink = s["sink"][None, None] if s["sink"] is not None else torch.full((1, 1, 1), -math.inf, device="cuda")
        top = torch.maximum(sink, one.amax(3)) if pages else sink.expand(n, longest, h)
        top = torch.maximum(top, two.amax(3)) if two.shape[3] else top
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        one, two = one.sub_(top[..., None]).exp_(), two.sub_(top[..., None]).exp_()
        total = one.sum(3) + two.sum(3) + torch.exp(sink - top)
        o = torch.matmul(one.view(n * longest * h, -1), prefix[:, :vdim]).view(n, longest, h, vdim)
        o = o + torch.matmul(two.view(n, longest * h, -1), rows[..., :vdim]).view(n, longest, h, vdim)
        o = o / torch.where(total > 0, total, torch.ones_like(total))[..., None]
        token = torch.arange(s["q"].shape[0], device="cuda")
        r = torch.searchsorted(s["cu_q"].long(), token, right=True) - 1
        take = (r >= r0) & (r < r1)
        outs.append(o[r[take] - r0, token[take] - begin[r[take]]])
        lses.append((top + torch.log(total))[r[take] - r0, token[take] - begin[r[take]]])
    return {"out": torch.cat(outs).bfloat16(), "lse": torch.cat(lses)}


def _run_own(s):
    import sparse_attention_kv_csa_gb300 as csa
    case = s["case"]
    if case["kind"] == "norm":
        out, stream, mean, rstd = csa.layer_norm_forward(s["x"], s["weight"], s["bias"], s["eps"], residual=s["residual"])
        answer = {"out": out, "mean": mean, "rstd": rstd}
        if stream is not None:
            answer["stream"] = stream
        return answer
    if case["kind"] == "grad":
        dx, dweight, dbias = csa.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], grad_residual=s["dh"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    rot = case["rotary"] if "rotary" in case else 0
    if case["kind"] == "append":
        kw = {}
        if case["bits8"]:
            kw["scales"] = s["store_scales"][:-1]
        if case["tokens"]:
            kw["queries"], kw["query_out"] = s["q"], s["q_wide"][..., -rot:]
        csa.append_rows(s["rows"], s["positions"], s["rotation"], s["slots"], s["store"][:-1], rotary=s["part"],
                        interleaved=case["interleaved"], **kw)
        answer = {"out": s["store"][:-1]}
        if case["bits8"]:
            answer["scales"] = s["store_scales"][:-1]
        if case["tokens"]:
            answer["q"] = s["q_wide"]
        return answer
    if case["kind"] == "rotate":
        return csa.rotate(s["x"][..., -rot:], s["positions"], s["rotation"], interleaved=case["interleaved"], inverse=case["inverse"])
    out, lse = csa.shared_attention(s["q"], s["cache"], s["table"], s["cu_q"], s["lens"], s["cu_groups"], s["shared_rows"],
                                    case["ratio"], 1 / math.sqrt(case["dim"]), v_dim=case["vdim"], row_scales=s["scales"],
                                    sink=s["sink"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "grad": _grad_plain, "append": _append_plain, "rotate": _rotate_plain,
            "shared": _shared_plain}[state["case"]["kind"]](state)


# ---------------------------------------------------------------- floors

def work(case):
    if case["kind"] in ("norm", "grad"):
        n, d, b = case["rows"], case["dim"], 4 if case["type"] == "f32" else 2
        if case["kind"] == "norm":
            return {"bytes": n * d * b * (4 if case["residual"] else 2) + 8 * d + 8 * n, "flops": 9 * n * d}
        return {"bytes": n * d * b * (4 if case["residual"] else 3) + 12 * d + 8 * n, "flops": 14 * n * d}
    if case["kind"] == "append":
        n, rot = case["rows"], case["rotary"]
        width = case["dim"] + (0 if case["inside"] else rot)
        each = width * (3 if case["bits8"] else 4) + 12 + (4 if case["bits8"] else 0) + 4 * rot
        return {"bytes": n * each + case["tokens"] * case["heads"] * rot * 4, "flops": 3 * rot * (n + case["tokens"] * case["heads"])}
    if case["kind"] == "rotate":
        n, rot = case["tokens"], case["rotary"]
        return {"bytes": n * (4 * case["heads"] * rot + 4 + 4 * rot), "flops": 3 * n * case["heads"] * rot}
    cuts, prefix, behind, news = _lengths(case, 0)
    ratio, page, h, d, v = case["ratio"], case["page"], case["heads"], case["dim"], case["vdim"]
    rows = pairs = 0
    for k, p in enumerate(prefix):
        shared = p // ratio // page * page
        rows += shared
        for r in range(cuts[k], cuts[k + 1]):
            a, b = p + behind[r], news[r]
            pairs += sum((a - b + i + 1) // ratio for i in range(b))
            rows += a // ratio - shared
    row = d + 4 if case["bits8"] else 2 * d
    return {"bytes": rows * row + sum(news) * h * (2 * d + 2 * v + 4) + 4 * rows // page, "flops": 2 * pairs * h * (d + v)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _rotated64(x, positions, rotation, interleaved, inverse):
    """x [n, heads, rot] in 64 bits as complex numbers times e^(i angle), the angles as the table holds them."""
    half = x.shape[-1] // 2
    turn = torch.complex(rotation[positions.long(), :half].double(), rotation[positions.long(), half:].double())[:, None]
    if inverse:
        turn = turn.conj()
    z = torch.view_as_complex((x.unflatten(-1, (half, 2)) if interleaved else x.unflatten(-1, (2, half)).transpose(-1, -2)).contiguous())
    z = torch.view_as_real(z * turn)
    return z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm":
        x = s["x"].double()
        answer = {}
        if s["residual"] is not None:
            # the stream is what later layers read: its rounding is part of the definition
            answer["stream"] = None
            x = (s["x"].float() + s["residual"].float()).to(s["x"].dtype).double()
        answer["mean"] = torch.einsum("nd->n", x) / case["dim"]
        x = x - answer["mean"][:, None]
        answer["rstd"] = (torch.einsum("nd,nd->n", x, x) / case["dim"] + s["eps"]) ** -0.5
        answer["out"] = torch.einsum("nd,n,d->nd", x, answer["rstd"], s["weight"].double()) + s["bias"].double()
        return answer
    if case["kind"] == "grad":
        dy, w, r = s["dy"].double(), s["weight"].double(), s["rstd"].double()
        unit = torch.einsum("nd,n->nd", s["x"].double() - s["mean"].double()[:, None], r)
        through = torch.einsum("nd,nd,d->n", dy, unit, w) / case["dim"]
        level = torch.einsum("nd,d->n", dy, w) / case["dim"]
        dx = torch.einsum("nd,d,n->nd", dy, w, r) - (r * level)[:, None] - torch.einsum("nd,n->nd", unit, r * through)
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("nd,nd->d", dy, unit), "dbias": torch.einsum("nd->d", dy)}
    if case["kind"] == "append":
        rot, rows = case["rotary"], s["rows"].double()
        plain, part = (rows[:, :-rot], rows[:, -rot:]) if s["part"] is None else (rows, s["part"].double())
        y = torch.cat([plain, _rotated64(part[:, None], s["positions"], s["rotation"], case["interleaved"], False)[:, 0]], 1)
        keep = s["slots"] >= 0
        out = torch.zeros(s["store"][:-1].shape, dtype=torch.float64, device="cuda")
        answer = {"out": None}
        if case["bits8"]:
            scales = torch.zeros(out.shape[0], dtype=torch.float64, device="cuda")
            answer["scales"] = scales.index_copy_(0, s["slots"][keep], y[keep].abs().max(1).values / E4M3_MAX)
        else:
            answer["out"] = out.index_copy_(0, s["slots"][keep], y[keep])
        if case["tokens"]:
            q = torch.zeros(s["q_wide"].shape, dtype=torch.float64, device="cuda")
            q[..., -rot:] = _rotated64(s["q"].double(), s["positions"], s["rotation"], case["interleaved"], False)
            answer["q"] = q
        return answer
    if case["kind"] == "rotate":
        return _rotated64(s["x"][..., -case["rotary"]:].double(), s["positions"], s["rotation"], case["interleaved"], case["inverse"])
    if work(case)["flops"] > 4e12:
        return None
    q, h, d, v = s["q"], case["heads"], case["dim"], case["vdim"]
    out = torch.zeros((q.shape[0], h, v), dtype=torch.float64, device="cuda")
    lse = torch.full((q.shape[0], h), -math.inf, dtype=torch.float64, device="cuda")
    cuts, prefix, behind, news = _lengths(case, seed)
    group = [k for k in range(case["groups"]) for _ in range(cuts[k], cuts[k + 1])]
    begin = 0
    for r, b in enumerate(news):
        a = prefix[group[r]] + behind[r]
        ids = s["table"][r, : -(-(a // case["ratio"]) // case["page"])].long()
        k = s["cache"][ids] if s["scales"] is None else s["cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
        k = k.double()
        if s["scales"] is not None:
            k = k * s["scales"][ids].double()[..., None]
        k = k.reshape(-1, d)
        see = torch.tensor([(a - b + i + 1) // case["ratio"] for i in range(b)], device="cuda")
        x = torch.einsum("thd,kd->thk", q[begin:begin + b].double(), k) / math.sqrt(d)
        x = x.masked_fill(torch.arange(k.shape[0], device="cuda")[None, None] >= see[:, None, None], -math.inf)
        if s["sink"] is not None:
            x = torch.cat([x, s["sink"].double()[None, :, None].expand(b, h, 1)], 2)
        if x.shape[2]:
            z = torch.logsumexp(x, 2)
            p = torch.exp(x - torch.where(torch.isfinite(z), z, torch.zeros_like(z))[..., None])[..., : k.shape[0]]
            out[begin:begin + b] = torch.einsum("thk,kd->thd", p, k[:, :v])
            lse[begin:begin + b] = z
        begin += b
    return {"out": out, "lse": lse}
