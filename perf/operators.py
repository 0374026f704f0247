"""The serving operators' cases: what is measured, in plain torch operations and through the package.

The operators are what follows the Compressor when its rows are served: the norm that writes rows (in 8 bits with
scales) into a paged cache, the tables that say where rows lie, and the attention whose keys and values are those rows.

Kinds of cases:
  norm     rms_norm_forward: residual addition, norm, bf16 or 8-bit output, optionally to cache slots
  grad     rms_norm_backward
  pages    page_tables: block tables, row offsets and slots from request lengths
  attend   latent_attention over the paged cache, bf16 or 8-bit rows
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # one token's residual stream in a decode step: latency
        dict(name="norm_token", kind="norm", rows=1, dim=4096, residual=True, bits8=False, group=0, slots=False),
        # a prompt's compressed rows (8 x 4096 tokens at ratio 4, 64 padding rows) normed into an 8-bit cache
        dict(name="norm_rows_to_cache", kind="norm", rows=8256, dim=512, residual=False, bits8=True, group=0,
             slots=True),
        # a prompt's residual stream, 8-bit output with a scale every 128 columns for the next projection
        dict(name="norm_stream8", kind="norm", rows=16411, dim=4096, residual=True, bits8=True, group=128,
             slots=False),
        # training: the norm's gradient over a batch's residual stream
        dict(name="grad_stream", kind="grad", rows=16384, dim=4096, residual=True),
        # training: the gradient of the norm over few rows of an odd width
        dict(name="grad_rows_odd", kind="grad", rows=1031, dim=1001, residual=False),
        # a decode step of 64 requests: at most one new row each
        dict(name="pages_decode", kind="pages", requests=64, most=65536, new=1, ratio=4, page=64),
        # a large batch, prompts among the single tokens
        dict(name="pages_mixed", kind="pages", requests=2053, most=131072, new=2048, ratio=4, page=64),
        # one short request's decode step: latency
        dict(name="attend_one", kind="attend", requests=1, most=2048, even=True, new=1, heads=64, dim=512, vdim=512,
             ratio=4, page=64, bits8=False, sink=True),
        # a decode step of a ragged batch over bf16 rows
        dict(name="attend_decode", kind="attend", requests=64, most=32768, even=False, new=1, heads=64, dim=512,
             vdim=512, ratio=4, page=64, bits8=False, sink=True),
        # a decode step of a large batch with 128 heads over 8-bit rows
        dict(name="attend_decode8", kind="attend", requests=129, most=16384, even=False, new=1, heads=128, dim=512,
             vdim=512, ratio=4, page=64, bits8=True, sink=False),
        # a few tokens a request (a speculative step), 16 heads, a row of 576 whose first 512 are the values, every
        # token a row, small pages
        dict(name="attend_few", kind="attend", requests=33, most=6000, even=False, new=3, heads=16, dim=576,
             vdim=512, ratio=1, page=16, bits8=False, sink=False),
        # a prompt's last chunk of 4096 tokens: matrix products
        dict(name="attend_prompt", kind="attend", requests=1, most=16384, even=True, new=4096, heads=64, dim=512,
             vdim=512, ratio=4, page=64, bits8=False, sink=True),
    ]


def _between(rng, low, high):
    """A whole number of [low, high], spread over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "grad", "pages", "attend", "attend", "attend"])
    if kind == "norm":
        dim = rng.choice([128, 512, 576, 1000, 2048, 4096, 4100, _between(rng, 64, 8192)])
        rows = _between(rng, 1, max(1, 16411 * 4096 // max(dim, 4096)))
        group = rng.choice([0, 128]) if dim % 128 == 0 else 0
        return dict(kind="norm", rows=rows, dim=dim, residual=rng.random() < 0.5, bits8=rng.random() < 0.6, group=group,
                    slots=rng.random() < 0.4)
    if kind == "grad":
        dim = rng.choice([512, 1000, 2048, 4096, _between(rng, 64, 8192)])
        return dict(kind="grad", rows=_between(rng, 1, 16384 * 4096 // max(dim, 4096)), dim=dim,
                    residual=rng.random() < 0.5)
    if kind == "pages":
        ratio, page = rng.choice([1, 4, 16, 128]), rng.choice([1, 16, 64, 100])
        return dict(kind="pages", requests=_between(rng, 1, 2053), most=min(_between(rng, 64, 131072), 512 * ratio * page),
                    new=rng.choice([1, 1, 4, _between(rng, 1, 2048)]), ratio=ratio, page=page)
    heads = rng.choice([1, 8, 16, 24, 64, 128])
    dim, vdim = rng.choice([(512, 512), (512, 512), (576, 512), (256, 256), (128, 128), (192, 128)])
    ratio = rng.choice([1, 4, 4, 16])
    if rng.random() < 0.7:
        new = rng.choice([1, 1, 2, 5])
        requests = _between(rng, 1, 129)
        rows = _between(rng, 16, min(16384, 400000 // requests))
    else:
        new = _between(rng, 64, 2048)
        requests = _between(rng, 1, 4)
        rows = _between(rng, 64, 4096)
    case = dict(kind="attend", requests=requests, most=max(rows * ratio, new), even=rng.random() < 0.3, new=new,
                heads=heads, dim=dim, vdim=vdim, ratio=ratio, page=rng.choice([16, 64, 64, 128, 50]),
                bits8=rng.random() < 0.4, sink=rng.random() < 0.5)
    while work(case)["flops"] > 1.5e12:
        case["new"] //= 2
    return case


# ---------------------------------------------------------------- inputs

def _lengths(case, seed):
    """(tokens of each request, new tokens of each request).  The new tokens go by the case alone, so that the shapes
    of the outputs do, the whole lengths by the seed too."""
    n, most, new = case["requests"], case["most"], case["new"]
    rng = random.Random(n * 31 + new)
    if case["kind"] == "pages":
        # a prompt among every ten requests, the rest decode
        news = [rng.randint(1, new) if i % 10 == 0 else 1 for i in range(n)]
    else:
        news = [new if case["even"] else rng.randint(max(1, new // 2), new) for _ in range(n)]
    news = [min(b, most) for b in news]
    rng = random.Random(seed * 7919 + 17)
    return [most if case.get("even") else rng.randint(max(1, b, most // 8), most) for b in news], news


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g):
    return torch.randn(shape, device="cuda", generator=g)


def prepare(case, seed):
    g = _generator(seed)
    state = {"case": case}
    if case["kind"] in ("norm", "grad"):
        n, d = case["rows"], case["dim"]
        # a residual stream has a few columns far larger than the rest
        x = _randn((n, d), g) * torch.exp(0.5 * _randn((d,), g))
        state["x"] = x.bfloat16()
        state["weight"] = 1 + 0.2 * _randn((d,), g)
        state["eps"] = 1e-6
        if case["kind"] == "grad":
            state["rstd"] = torch.rsqrt(state["x"].float().square().mean(1) + 1e-6)
            state["dy"] = (0.01 * _randn((n, d), g)).bfloat16()
            state["dh"] = (0.01 * _randn((n, d), g)).bfloat16() if case["residual"] else None
            return state
        state["residual"] = _randn((n, d), g).bfloat16() if case["residual"] else None
        if case["slots"]:
            total = n + n // 2 + 64
            slots = torch.randperm(total, device="cuda", generator=g)[:n]
            state["slots"] = torch.where(torch.rand(n, device="cuda", generator=g) < 0.01, -1, slots)
            # one row past the cache, where the plain form puts rows that have no slot
            state["store"] = torch.zeros((total + 1, d), dtype=torch.uint8 if case["bits8"] else torch.bfloat16, device="cuda")
            if case["bits8"]:
                state["store"] = state["store"].view(torch.float8_e4m3fn)
                state["store_scales"] = torch.zeros((total + 1, d // case["group"] if case["group"] else 1), device="cuda")
        return state
    lens, news = _lengths(case, seed)
    page, ratio = case["page"], case["ratio"]
    pages_of = lambda tokens: -(-(tokens // ratio) // page)  # noqa: E731
    width = max(1, -(-(case["most"] // ratio) // page))
    if case["kind"] == "pages":
        before = [a - b for a, b in zip(lens, news)]
        held = sum(map(pages_of, before))
        need = sum(map(pages_of, lens))
        ids = torch.randperm(need + 64, device="cuda", generator=g).int()
        at, table = 0, torch.full((case["requests"], width), -1, dtype=torch.int32, device="cuda")
        count = torch.tensor([pages_of(b) for b in before], device="cuda")
        cols = torch.arange(width, device="cuda")
        start = torch.cumsum(count, 0) - count
        source = (start[:, None] + cols[None]).clamp(max=need + 63)
        state["table"] = torch.where(cols[None] < count[:, None], ids[source], table)
        state["free"] = ids[held:].contiguous()
        state["before"], state["after"] = _int32(before), _int32(lens)
        state["capacity"] = sum(b // ratio + 1 for b in news)
        return state
    d, h = case["dim"], case["heads"]
    used = [pages_of(a) for a in lens]
    n_pages = sum(used) + 3
    ids = torch.randperm(n_pages, device="cuda", generator=g).int()
    count = torch.tensor(used, device="cuda")
    cols = torch.arange(width, device="cuda")
    source = (torch.cumsum(count, 0) - count)[:, None] + cols[None]
    state["table"] = torch.where(cols[None] < count[:, None], ids[source.clamp(max=n_pages - 1)], -1).int().contiguous()
    rows = _randn((n_pages, page, d), g)
    if case["bits8"]:
        scales = rows.abs().amax(2) / E4M3_MAX
        state["cache"] = (rows / scales[..., None]).to(torch.float8_e4m3fn)
        state["scales"] = scales.contiguous()
    else:
        state["cache"], state["scales"] = rows.bfloat16(), None
    state["q"] = (1.5 * _randn((sum(news), h, d), g)).bfloat16()
    cu = [0]
    for b in news:
        cu.append(cu[-1] + b)
    state["cu_q"], state["lens"] = _int32(cu), _int32(lens)
    state["sink"] = _randn((h,), g) if case["sink"] else None
    state["longest"] = max(news)
    return state


# ---------------------------------------------------------------- plain forms

def _norm_plain(s):
    case = s["case"]
    x = s["x"].float()
    if s["residual"] is not None:
        stream = (x + s["residual"].float()).bfloat16()
        x = stream.float()
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"])
    y = x * rstd * s["weight"]
    scales = None
    if case["bits8"]:
        groups = y.view(y.shape[0], -1, case["group"] or y.shape[1])
        scales = groups.abs().amax(2) / E4M3_MAX
        step = torch.where(scales > 0, scales, torch.ones_like(scales))
        out = (groups / step[..., None]).view_as(y).to(torch.float8_e4m3fn)
    else:
        out = y.bfloat16()
    if case["slots"]:
        at = torch.where(s["slots"] < 0, s["store"].shape[0] - 1, s["slots"])
        if case["bits8"]:
            s["store"].view(torch.uint8)[at] = out.view(torch.uint8)
            s["store_scales"][at] = scales
            scales = s["store_scales"][:-1]
        else:
            s["store"][at] = out
        out = s["store"][:-1]
    answer = {"out": out, "rstd": rstd[:, 0]}
    if case["bits8"]:
        answer["scales"] = scales
    if s["residual"] is not None:
        answer["stream"] = stream
    return answer


def _grad_plain(s):
    h, dy = s["x"].float(), s["dy"].float()
    unit = h * s["rstd"][:, None]
    wdy = dy * s["weight"]
    dx = s["rstd"][:, None] * (wdy - unit * (wdy * unit).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.bfloat16(), "dweight": (dy * unit).sum(0)}


def _pages_plain(s):
    case = s["case"]
    page, ratio, free, cap = case["page"], case["ratio"], s["free"], s["capacity"]
    old = (s["before"] // ratio).long()
    new = torch.maximum((s["after"] // ratio).long(), old)
    held, need = (old + page - 1) // page, (new + page - 1) // page
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    cu_rows = torch.cat([zero, torch.cumsum(new - old, 0)])
    cu_pages = torch.cat([zero, torch.cumsum(need - held, 0)])
    cols = torch.arange(s["table"].shape[1], device="cuda")[None]
    source = cu_pages[:-1, None] + cols - held[:, None]
    fresh = torch.where(source < free.numel(), free[source.clamp(0, free.numel() - 1)], -1)
    table = torch.where(cols < held[:, None], s["table"], torch.where(cols < need[:, None], fresh, -1))
    i = torch.arange(cap, device="cuda")
    r = torch.searchsorted(cu_rows, i, right=True).sub(1).clamp(max=old.numel() - 1)
    row = old[r] + i - cu_rows[r]
    at = (row // page).clamp(max=table.shape[1] - 1)
    ids = table[r, at].long()
    slots = torch.where((i < cu_rows[-1]) & (row // page < table.shape[1]) & (ids >= 0), ids * page + row % page, -1)
    taken = cu_pages[-1].clamp(max=free.numel())
    counts = torch.stack([cu_rows[-1], taken, cu_pages[-1] - taken, need.max()]).int()
    return {"table": table.int(), "cu_rows": cu_rows.int(), "slots": slots, "counts": counts}


def _attend_plain(s):
    case = s["case"]
    n, h, d, ratio, page = case["requests"], case["heads"], case["dim"], case["ratio"], case["page"]
    vdim, longest = case["vdim"], s["longest"]
    scale = 1 / math.sqrt(d)
    table = s["table"].long()
    if s["scales"] is None:
        rows = s["cache"][table.clamp(min=0)].float()
    else:
        rows = s["cache"].view(torch.uint8)[table.clamp(min=0)].view(torch.float8_e4m3fn).float()
        rows = rows * s["scales"][table.clamp(min=0)][..., None]
    rows = rows.view(n, -1, d)
    begin = s["cu_q"][:-1].long()
    count = s["cu_q"][1:].long() - begin
    i = torch.arange(longest, device="cuda")
    q = s["q"][(begin[:, None] + i).clamp(max=s["q"].shape[0] - 1)].float().view(n, longest * h, d)
    seen = (s["lens"].long() - count)[:, None] + i + 1
    seen = torch.div(seen, ratio, rounding_mode="floor").clamp(max=rows.shape[1])
    hidden = torch.arange(rows.shape[1], device="cuda")[None, None] >= seen[..., None]
    x = torch.matmul(q, rows.transpose(1, 2)).mul_(scale).view(n, longest, h, -1)
    x.masked_fill_(hidden[:, :, None], -math.inf)
    sink = s["sink"][None, None] if s["sink"] is not None else torch.full((1, 1, 1), -math.inf, device="cuda")
    top = torch.maximum(x.amax(3), sink)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    x = x.sub_(top[..., None]).exp_()
    total = x.sum(3) + torch.exp(sink - top)
    o = torch.matmul(x.view(n, longest * h, -1), rows[..., :vdim]).view(n, longest, h, vdim)
    o = o / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    lse = top + torch.log(total)
    token = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(s["cu_q"].long(), token, right=True) - 1
    return {"out": o[r, token - begin[r]].bfloat16(), "lse": lse[r, token - begin[r]]}


def _run_own(s):
    import sparse_attention_kv_csa_gb300 as csa
    case = s["case"]
    if case["kind"] == "norm":
        kw = {}
        if case["bits8"]:
            kw = {"out_dtype": torch.float8_e4m3fn, "scale_group": case["group"]}
        if case["slots"]:
            kw["slots"], kw["out"] = s["slots"], s["store"][:-1]
            if case["bits8"]:
                kw["scales"] = s["store_scales"][:-1]
        out, scales, stream, rstd = csa.rms_norm_forward(s["x"], s["weight"], s["eps"], residual=s["residual"], **kw)
        answer = {"out": out, "rstd": rstd}
        if case["bits8"]:
            answer["scales"] = scales
        if stream is not None:
            answer["stream"] = stream
        return answer
    if case["kind"] == "grad":
        dx, dweight = csa.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], grad_residual=s["dh"])
        return {"dx": dx, "dweight": dweight}
    if case["kind"] == "pages":
        table, cu_rows, slots, counts = csa.page_tables(s["before"], s["after"], case["ratio"], case["page"], s["free"],
                                                        s["table"], s["capacity"])
        return {"table": table, "cu_rows": cu_rows, "slots": slots, "counts": counts}
    out, lse = csa.latent_attention(s["q"], s["cache"], s["table"], s["cu_q"], s["lens"], case["ratio"],
                                    1 / math.sqrt(case["dim"]), v_dim=case["vdim"], row_scales=s["scales"],
                                    sink=s["sink"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "grad": _grad_plain, "pages": _pages_plain, "attend": _attend_plain}[state["case"]["kind"]](state)


# ---------------------------------------------------------------- floors

def _seen_rows(case, seed=0):
    """(sum over new tokens of the rows that each sees, sum over requests of the rows that any token sees)."""
    pairs = rows = 0
    for a, b in zip(*_lengths(case, seed)):
        pairs += sum((a - b + i + 1) // case["ratio"] for i in range(b))
        rows += a // case["ratio"]
    return pairs, rows


def work(case):
    if case["kind"] == "norm":
        n, d = case["rows"], case["dim"]
        each = 2 + (1 if case["bits8"] else 2) + (4 if case["residual"] else 0)
        scales = (d // case["group"] if case["group"] else 1) if case["bits8"] else 0
        return {"bytes": n * d * each + 4 * d + n * (4 + 4 * scales + (8 if case["slots"] else 0)), "flops": 6 * n * d}
    if case["kind"] == "grad":
        n, d = case["rows"], case["dim"]
        return {"bytes": n * d * (6 + (2 if case["residual"] else 0)) + 8 * d + 4 * n, "flops": 10 * n * d}
    lens, news = _lengths(case, 0)
    if case["kind"] == "pages":
        ratio, page = case["ratio"], case["page"]
        width = max(1, -(-(case["most"] // ratio) // page))
        fresh = sum(a // ratio - (a - b) // ratio for a, b in zip(lens, news))
        held = sum(-(-((a - b) // ratio) // page) for a, b in zip(lens, news))
        return {"bytes": case["requests"] * (12 + 4 * width) + 4 * held + 8 * fresh, "flops": 0}
    pairs, rows = _seen_rows(case)
    h, d, v = case["heads"], case["dim"], case["vdim"]
    row = d + 4 if case["bits8"] else 2 * d
    return {"bytes": rows * row + sum(news) * h * (2 * d + 2 * v + 4) + 4 * rows // case["page"], "flops": 2 * pairs * h * (d + v)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm":
        x = s["x"].double()
        answer = {}
        if s["residual"] is not None:
            # the stream is what later layers read: its rounding is part of the definition
            answer["stream"] = None
            x = (s["x"].float() + s["residual"].float()).bfloat16().double()
        mean = torch.einsum("nd,nd->n", x, x) / case["dim"]
        answer["rstd"] = (mean + s["eps"]) ** -0.5
        y = torch.einsum("nd,n,d->nd", x, answer["rstd"], s["weight"].double())
        answer["out"] = None if case["bits8"] or case["slots"] else y
        if case["bits8"]:
            answer["scales"] = None if case["slots"] else y.reshape(case["rows"], -1, case["group"] or case["dim"]).abs().max(2).values / E4M3_MAX
        elif case["slots"]:
            out = torch.zeros((s["store"].shape[0] - 1, case["dim"]), dtype=torch.float64, device="cuda")
            keep = s["slots"] >= 0
            out.index_copy_(0, s["slots"][keep], y[keep])
            answer["out"] = out
        return answer
    if case["kind"] == "grad":
        h, dy, w, r = s["x"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()
        through = torch.einsum("nd,nd,d,n->n", dy, h, w, r) / case["dim"]
        dx = torch.einsum("nd,d,n->nd", dy, w, r) - torch.einsum("nd,n->nd", h, r * r * through)
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("nd,nd,n->d", dy, h, r)}
    if case["kind"] == "pages":
        return None
    if work(case)["flops"] > 4e12:
        return None
    q, h, d, v = s["q"], case["heads"], case["dim"], case["vdim"]
    out = torch.zeros((q.shape[0], h, v), dtype=torch.float64, device="cuda")
    lse = torch.full((q.shape[0], h), -math.inf, dtype=torch.float64, device="cuda")
    lens, news = _lengths(case, seed)
    begin = 0
    for r, (a, b) in enumerate(zip(lens, news)):
        ids = s["table"][r, : -(-(a // case["ratio"]) // case["page"])].long()
        k = s["cache"][ids] if s["scales"] is None else s["cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
        k = k.double()
        if s["scales"] is not None:
            k = k * s["scales"][ids].double()[..., None]
        k = k.reshape(-1, d)
        for first in range(0, b, 512):
            last = min(b, first + 512)
            see = torch.tensor([(a - b + i + 1) // case["ratio"] for i in range(first, last)], device="cuda")
            x = torch.einsum("thd,kd->thk", q[begin + first:begin + last].double(), k) / math.sqrt(d)
            x = x.masked_fill(torch.arange(k.shape[0], device="cuda")[None, None] >= see[:, None, None], -math.inf)
            if s["sink"] is not None:
                x = torch.cat([x, s["sink"].double()[None, :, None].expand(last - first, h, 1)], 2)
            if x.shape[2] == 0:
                continue
            z = torch.logsumexp(x, 2)
            p = torch.exp(x - torch.where(torch.isfinite(z), z, torch.zeros_like(z))[..., None])[..., : k.shape[0]]
            out[begin + first:begin + last] = torch.einsum("thk,kd->thd", p, k[:, :v])
            lse[begin + first:begin + last] = z
        begin += b
    return {"out": out, "lse": lse}
