"""Serving the Compressor's rows, from prompts to single tokens, with the package's operators:

    compress_forward    tokens' kv and score -> rows (ratio 4, overlapping windows)
    page_tables         which slots of the paged cache the new rows get
    rms_norm_forward    rows -> normed rows in 8 bits with a scale each, written to their slots
    latent_attention    queries of all heads over each request's rows, and afterwards
    rms_norm_forward    a residual stream's next norm

Inputs are random.  `python examples/serve_rows.py` prints the time of a prompt and of a decode step on the GPU;
`Server` is the loop that a serving program would have around its projections.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_kv_csa_gb300 as csa  # noqa: E402

RATIO, COFF = 4, 2


class Server:
    """A batch of requests whose compressed rows live in a paged 8-bit cache."""

    def __init__(self, requests, heads, dim, page_size, pages, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
        self.heads, self.dim, self.page_size = heads, dim, page_size
        self.ape = 0.25 * randn(RATIO, COFF * dim)
        self.norm, self.sink = 1 + 0.1 * randn(dim), randn(heads)
        self.cache = torch.zeros((pages, page_size, dim), dtype=torch.float8_e4m3fn, device="cuda")
        self.scales = torch.zeros((pages, page_size), device="cuda")
        self.free = torch.randperm(pages, device="cuda", generator=g).int()
        self.taken = torch.zeros(1, dtype=torch.int32, device="cuda")
        # (as wide as the pool, so no request needs more columns)
        self.table = torch.full((requests, pages), -1, dtype=torch.int32, device="cuda")
        self.lens = [0] * requests  # tokens so far
        self.tail = [None] * requests  # kv and score from the block before the open one on

    def _compress(self, kv, score, new):
        """Rows of the blocks that the new tokens complete, in request order.  A window reaches into the block before,
        so a request's pack starts there and that block's own row, already stored, is left out."""
        packs, lengths, keep, at = [], [], [], 0
        first = 0
        for r, n in enumerate(new):
            block = torch.stack([kv[first:first + n], score[first:first + n]])
            pack = block if self.tail[r] is None else torch.cat([self.tail[r], block], 1)
            first += n
            done = self.lens[r] // RATIO  # blocks stored
            held = min(done, 1)           # of them, in the pack
            rows = pack.shape[1] // RATIO
            keep += range(at + held, at + rows)
            packs.append(pack)
            lengths.append(pack.shape[1])
            at += rows
            self.tail[r] = pack[:, max(0, rows - 1) * RATIO:]
        cu = torch.tensor([0] + lengths).cumsum(0).int().cuda()
        cc = torch.tensor([0] + [n // RATIO for n in lengths]).cumsum(0).int().cuda()
        pack = torch.cat(packs, 1)
        if at == 0:
            return kv.new_empty((0, self.dim))
        rows = csa.compress_forward(pack[0].contiguous(), pack[1].contiguous(), self.ape, cu, cc, RATIO, COFF, self.dim, at)
        return rows[torch.tensor(keep, device="cuda", dtype=torch.long)]

    def step(self, kv, score, q, new):
        """kv, score bf16 [tokens, 2 dim] and q bf16 [tokens, heads, dim] of the new tokens (new[r] of request r, in
        order); returns the attention's output [tokens, heads, dim]."""
        before = torch.tensor(self.lens, dtype=torch.int32).cuda()
        rows = self._compress(kv, score, new)
        self.lens = [a + b for a, b in zip(self.lens, new)]
        after = torch.tensor(self.lens, dtype=torch.int32).cuda()
        _, _, slots, counts = csa.page_tables(before, after, RATIO, self.page_size, self.free, self.table, rows.shape[0],
                                              taken=self.taken, out=self.table)
        self.taken += counts[1:2]
        csa.rms_norm_forward(rows, self.norm, slots=slots, out=self.cache.view(-1, self.dim), scales=self.scales.view(-1))
        cu_q = torch.tensor([0] + list(new)).cumsum(0).int().cuda()
        out, _ = csa.latent_attention(q, self.cache, self.table, cu_q, after, RATIO, 1 / math.sqrt(self.dim),
                                      row_scales=self.scales, sink=self.sink)
        return out


def inputs(tokens, heads, dim, g):
    kv = torch.randn((tokens, COFF * dim), device="cuda", generator=g).bfloat16()
    score = (1.5 * torch.randn((tokens, COFF * dim), device="cuda", generator=g)).bfloat16()
    return kv, score, torch.randn((tokens, heads, dim), device="cuda", generator=g).bfloat16()


def main():
    heads, dim, prompts = 64, 512, [4096, 1000, 37, 8191]
    server = Server(len(prompts), heads, dim, 64, 256)
    g = torch.Generator(device="cuda").manual_seed(1)
    for name, new in [("prompts", prompts)] + [("decode", [1] * len(prompts))] * 6:
        kv, score, q = inputs(sum(new), heads, dim, g)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        out = server.step(kv, score, q, new)
        # what follows in a model: the output (its projection left out) joins the residual stream, whose norm feeds the
        # next products in 8 bits
        stream = out.view(out.shape[0], -1)
        csa.rms_norm_forward(stream[:, :4096], None, residual=stream[:, 4096:8192], out_dtype=torch.float8_e4m3fn, scale_group=128)
        end.record()
        torch.cuda.synchronize()
        print("%-8s %6d tokens  %8.3f ms  |out| %.4f" % (name, sum(new), start.elapsed_time(end), out.float().abs().mean().item()))


if __name__ == "__main__":
    main()
