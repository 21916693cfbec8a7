"""One attention layer in service on an 8-bit key/value cache, and a sequence that leaves the device and comes back.

Prompts of uneven length are admitted (their keys and values written, their queries attended to the cache), then every
sequence is decoded a token at a time. Half way one sequence is parked: its blocks, which are bytes, are compressed
without loss into page-locked host memory (format v3) and its blocks are taken by others; later it is restored into
other blocks and goes on. The outputs equal those of a run in which it never left.

    python examples/serve_cache.py [--steps 8] [--heads 32] [--kv-heads 8] [--dim 128]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import entropy_coding_gb300 as zc  # noqa: E402


class Server:
    """Sequences over one cache; blocks are handed out from a free list."""

    def __init__(self, n_blocks, kv_heads, dim, block, device="cuda"):
        self.cache = zc.KVCache.empty(n_blocks, kv_heads, dim, block, device)
        self.free = list(range(n_blocks))[::-1]
        self.blocks: dict[int, list[int]] = {}
        self.length: dict[int, int] = {}
        self.device = device

    def batch(self, news: dict[int, int]) -> zc.KVBatch:
        """Makes room for the sequences' new tokens and describes the step."""
        for s, n in news.items():
            have = self.blocks.setdefault(s, [])
            self.length[s] = self.length.get(s, 0) + n
            while len(have) * self.cache.block_tokens < self.length[s]:
                have.append(self.free.pop())
        width = max(len(self.blocks[s]) for s in news)
        table = [self.blocks[s] + [0] * (width - len(self.blocks[s])) for s in news]
        cu = [0]
        for n in news.values():
            cu.append(cu[-1] + n)
        i32 = dict(dtype=torch.int32, device=self.device)
        return zc.KVBatch(torch.tensor(table, **i32), torch.tensor(cu, **i32),
                          torch.tensor([self.length[s] for s in news], **i32), cu[-1], max(news.values()))

    def step(self, news: dict[int, int], qkv: dict[int, torch.Tensor], heads: int) -> dict[int, torch.Tensor]:
        """New tokens of some sequences through the layer: qkv[s] is [tokens, heads + 2 kv_heads, dim], a fused
        projection's output; returns each sequence's [tokens, heads, dim]."""
        batch = self.batch(news)
        x = torch.cat([qkv[s] for s in news])
        h = self.cache.kv_heads
        zc.kv_write(self.cache, batch, x[:, heads: heads + h], x[:, heads + h:])
        out, _ = zc.kv_attend(self.cache, batch, x[:, :heads])
        return dict(zip(news, out.split(list(news.values()))))

    def _parts(self, s):
        """The bytes that hold a sequence: codes and scales of its blocks."""
        at = torch.tensor(self.blocks[s], device=self.device)
        c = self.cache
        return [t.view(torch.uint8)[at].contiguous() for t in (c.k, c.v)] + [t[at].contiguous() for t in (c.k_scale, c.v_scale)]

    def park(self, s) -> tuple[list[torch.Tensor], int]:
        """Moves a sequence to host memory, losslessly compressed; its blocks are free."""
        blobs = [zc.compress(t, lane_words=True, host_blob=True) for t in self._parts(s)]
        self.free += self.blocks.pop(s)
        return blobs, self.length.pop(s)

    def restore(self, s, parked) -> None:
        blobs, n = parked
        k, v, ks, vs = (zc.decompress(b, device=self.device) for b in blobs)
        self.blocks[s] = [self.free.pop() for _ in range(len(k))]
        self.length[s] = n
        at = torch.tensor(self.blocks[s], device=self.device)
        c = self.cache
        c.k.view(torch.uint8)[at], c.v.view(torch.uint8)[at] = k, v
        c.k_scale[at], c.v_scale[at] = ks, vs


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    a = ap.parse_args(argv)
    prompts = {0: 700, 1: 130, 2: 1500, 3: 64}
    g = torch.Generator(device="cuda").manual_seed(0)

    def tokens(n):
        return torch.randn(n, a.heads + 2 * a.kv_heads, a.dim, generator=g, device="cuda").bfloat16()

    x0 = {s: tokens(n) for s, n in prompts.items()}
    xs = [{s: tokens(1) for s in prompts} for _ in range(a.steps)]

    def serve(leaves: bool):
        srv = Server(64, a.kv_heads, a.dim, 64)
        outs = [srv.step(prompts, x0, a.heads)]
        ratio = None
        for i, x in enumerate(xs):
            if leaves and i == a.steps // 2:
                size = sum(t.numel() * t.element_size() for t in srv._parts(2))
                parked = srv.park(2)
                ratio = sum(b.numel() for b in parked[0]) / size
                outs.append(srv.step({0: 1, 1: 1, 3: 1}, x, a.heads))  # the others go on, in its blocks if they need them
                srv.restore(2, parked)
                outs[-1].update(srv.step({2: 1}, x, a.heads))
            else:
                outs.append(srv.step(dict.fromkeys(prompts, 1), x, a.heads))
        srv.cache.check()
        return outs, ratio, srv

    plain, _, _ = serve(False)
    moved, ratio, srv = serve(True)
    # Steps of the same sequences give the same bits wherever their blocks are; in the step that was split in two the
    # keys are shared out differently over the GPU, and the float32 sums may round to another bfloat16.
    def alike(i, p, m):
        return torch.equal(p, m) if i != a.steps // 2 + 1 else torch.allclose(p.float(), m.float(), atol=2 ** -8, rtol=2 ** -7)

    same = all(alike(i, p[s], m[s]) for i, (p, m) in enumerate(zip(plain, moved)) for s in prompts)
    # against attention in float32 over the numbers that the cache holds
    q = xs[-1][2][:, :a.heads].float()
    one = zc.KVBatch(torch.tensor([srv.blocks[2]], dtype=torch.int32, device="cuda"),
                     torch.tensor([0, srv.length[2]], dtype=torch.int32, device="cuda"),
                     torch.tensor([srv.length[2]], dtype=torch.int32, device="cuda"), srv.length[2], srv.length[2])
    k, v = (t.repeat_interleave(a.heads // a.kv_heads, 1).float() for t in zc.kv_read(srv.cache, one))
    p = torch.softmax(torch.einsum("qhd,khd->hqk", q, k) * a.dim ** -0.5, -1)
    want = torch.einsum("hqk,khd->qhd", p, v)
    err = float((moved[-1][2].float() - want).abs().max() / want.abs().max())
    print(f"{sum(prompts.values())} prompt tokens, {a.steps} steps of {len(prompts)} sequences; parked sequence "
          f"{100 * ratio:.1f} % of its 8-bit blocks; same outputs: {same}; error against float32 {err:.2g}")
    return dict(same=same, ratio=ratio, error=err)


if __name__ == "__main__":
    main()
