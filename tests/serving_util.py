"""Plain 64-bit forms of the serving operators, and the error bounds that the kernels are held to.

A rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by 2^-24 (half a step)."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}


def attention64(q, cache, table, cu_q, seq_lens, ratio, scale, v_dim, row_scales=None, sink=None):
    """(out, lse, bound on out's error, bound on lse's) in 64 bits.

    eps, the error of one logit: a product of head_dim terms summed in fp32, head_dim 2^-24 of sum |q k| scale, and
    2^-22 of the logit and of 1 for the exponential's argument and value.  The weights are off by twice that and, where
    they are rounded to bf16 for the second product, 2^-8; the weighted sum and the total by (rows + head_dim) 2^-24;
    the result is rounded to bf16."""
    n, heads, dim = q.shape
    pages, page = cache.shape[:2]
    out = torch.zeros((n, heads, v_dim), dtype=torch.float64)
    lse = torch.full((n, heads), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    q64, cu = q.detach().cpu().double(), cu_q.tolist()
    flat = cache.detach().cpu()
    for r, length in enumerate(seq_lens.tolist()):
        ids = table[r].cpu().long()
        for i in range(cu[r + 1] - cu[r]):
            t = cu[r] + i
            seen = max(0, length - (cu[r + 1] - cu[r]) + i + 1) // ratio
            seen = min(seen, ids.numel() * page)
            j = torch.arange(seen)
            id_ = ids[j // page]
            good = (id_ >= 0) & (id_ < pages)
            id_, off = id_[good], (j % page)[good]
            if cache.dtype == torch.float8_e4m3fn:
                k = flat.view(torch.uint8)[id_, off].view(torch.float8_e4m3fn).double()
                k = k * row_scales.cpu().double()[id_, off][:, None]
            else:
                k = flat[id_, off].double()
            s = (q64[t] @ k.T) * scale
            absolute = (q64[t].abs() @ k.abs().T) * scale
            full = s if sink is None else torch.cat([s, sink.cpu().double()[:, None]], 1)
            if full.shape[1] == 0:
                continue
            z = torch.logsumexp(full, 1)
            lse[t] = z
            zf = torch.where(torch.isfinite(z), z, torch.zeros_like(z))
            w = torch.exp(s - zf[:, None])
            out[t] = w @ k[:, :v_dim]
            if s.shape[1]:
                eps = dim * 2.0 ** -24 * absolute.amax(1) + 2.0 ** -22 * (1 + s.abs().amax(1))
            else:
                eps = torch.zeros(heads, dtype=torch.float64)
            sums = (s.shape[1] + dim) * 2.0 ** -24
            tol[t] = 2.0 ** -8 * out[t].abs() + (2.0 ** -8 + 2 * eps + 2 * sums)[:, None] * (w @ k[:, :v_dim].abs())
            tol_lse[t] = eps + sums + 2.0 ** -22 * (1 + zf.abs())
    return out, lse, tol + 1e-30, tol_lse


def norm64(x, weight, eps, residual=None):
    """(h in x's type, y in 64 bits, rstd in 64 bits)."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    hd = h.double()
    rstd = (hd.square().mean(1) + eps).rsqrt()
    return h, hd * rstd[:, None] * (1.0 if weight is None else weight.double()), rstd


def pages_plain(before, after, ratio, page, free, table, capacity, taken=0):
    """Lists in, lists out: the tables by hand, one request after another."""
    out = [list(row) for row in table]
    cu, slots, at, need_all, widest = [0], [], taken, 0, 0
    for r, (a, b) in enumerate(zip(before, after)):
        old = max(a, 0) // ratio
        new = max(max(b, 0) // ratio, old)
        held, need = -(-old // page), -(-new // page)
        widest = max(widest, need)
        pages = list(table[r][:held])
        pages += [-1] * max(0, held - len(pages))
        for _ in range(need - held):
            pages.append(free[at] if at < len(free) else -1)
            at += 1
            need_all += 1
        out[r] = [pages[c] if c < min(need, len(pages)) else -1 for c in range(len(table[r]))]
        for row in range(old, new):
            c = row // page
            ok = c < len(table[r]) and pages[c] >= 0
            slots.append(pages[c] * page + row % page if ok else -1)
        cu.append(len(slots))
    total = len(slots)
    slots = (slots + [-1] * max(0, capacity - total))[:capacity]
    got = min(need_all, max(0, len(free) - taken))
    return out, cu, slots, [total, got, need_all - got, widest]
