"""One attention layer that serves a batch from a paged FP4 key/value cache.

    python examples/fp4_attention_layer.py

Prompts go in by chunks, then every sequence decodes token by token.  Each
step is the same five calls: the fused projection, ``qk_norm_rope``,
``fp4_kv_write``, ``fp4_kv_attention`` and the output projection.  The last
tokens are compared with the same layer over a bf16 cache, in float32."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_reduce_amd as fp4  # noqa: E402


class Layer:
    """Random weights, one page table row for each sequence."""

    def __init__(self, seqs, context, hidden=1024, q_heads=8, kv_heads=2, dim=128, page=64,
                 fmt=fp4.FORMAT_NVFP4, flags=fp4.FOUR_OVER_SIX, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.q_heads, self.kv_heads, self.dim, self.page = q_heads, kv_heads, dim, page
        width = (q_heads + 2 * kv_heads) * dim
        self.wqkv = (new(hidden, width) * hidden ** -0.5).bfloat16()
        self.wo = (new(q_heads * dim, hidden) * (q_heads * dim) ** -0.5).bfloat16()
        self.q_norm, self.k_norm = (1 + 0.1 * new(2, dim)).bfloat16().unbind(0)
        self.table = fp4.rope_table(context, dim)
        per = -(-context // page)
        self.pages = torch.randperm(seqs * per, generator=g, device="cuda").view(seqs, per).int()
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.cache, self.fmt, self.flags = None, fmt, flags
        self.kept = [[] for _ in range(seqs)]        # bf16 keys and values, for the comparison

    def calibrate(self, k, v):
        """The heads' largest magnitudes from the first keys and values, with room to spare."""
        if self.cache is None:
            am = [1.25 * t.float().abs().amax((0, 2)) for t in (k, v)]
            nv = self.fmt == fp4.FORMAT_NVFP4
            self.cache = fp4.KvCache.alloc(self.pages.numel(), self.page, self.kv_heads, self.dim,
                                           self.fmt, self.flags, am[0] if nv else None,
                                           am[1] if nv else None)

    def step(self, x, news, keep=False):
        """x [sum(news)][hidden]: each sequence's new tokens.  Returns the layer's output."""
        cut = torch.tensor([0] + news, device="cuda").cumsum(0)
        seq = torch.repeat_interleave(torch.arange(len(news), device="cuda"), cut[1:] - cut[:-1])
        pos = self.lens[seq] + torch.arange(len(x), device="cuda") - cut[seq]
        qkv = (x @ self.wqkv).view(len(x), -1, self.dim)
        q, k, v = qkv.split((self.q_heads, self.kv_heads, self.kv_heads), 1)
        q, k = fp4.qk_norm_rope(q, k, self.q_norm, self.k_norm, pos, self.table)
        self.calibrate(k, v)
        slots = self.pages[seq, pos // self.page].long() * self.page + pos % self.page
        fp4.fp4_kv_write(self.cache, k, v, slots)
        self.lens += (cut[1:] - cut[:-1]).int()
        if keep:
            for b in range(len(news)):
                self.kept[b].append((k[cut[b]:cut[b + 1]], v[cut[b]:cut[b + 1]]))
        out = fp4.fp4_kv_attention(self.cache, q, self.pages, self.lens, cut.int(), max_q=max(news))
        self.q = q
        return out.flatten(1) @ self.wo

    def dense(self, b, q):
        """The last token of sequence b attending over its bf16 keys and values."""
        k, v = (torch.cat(t).float() for t in zip(*self.kept[b]))
        group = self.q_heads // self.kv_heads
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        s = (q.float()[None] * k).sum(-1) * self.dim ** -0.5        # [kv][q_heads]
        o = (s.softmax(0)[..., None] * v).sum(0)
        return o.flatten().bfloat16()[None] @ self.wo


def run(lens=(1500, 700, 40), chunk=256, decode=16, **kw):
    """Serve prompts of these lengths; the relative error of every sequence's last output."""
    layer = Layer(len(lens), max(lens) + decode, **kw)
    hidden = layer.wqkv.shape[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    done = [0] * len(lens)
    while any(d < n for d, n in zip(done, lens)):
        news = [min(chunk, n - d) for d, n in zip(done, lens)]
        x = torch.randn(sum(news), hidden, generator=g, device="cuda").bfloat16()
        layer.step(x, news, keep=True)
        done = [d + n for d, n in zip(done, news)]
    ones = [1] * len(lens)
    for _ in range(decode):
        x = torch.randn(len(lens), hidden, generator=g, device="cuda").bfloat16()
        out = layer.step(x, ones, keep=True)
    errors = []
    for b in range(len(lens)):
        want = layer.dense(b, layer.q[b]).float()
        errors.append(float((out[b].float() - want).norm() / want.norm()))
    return errors


if __name__ == "__main__":
    for name, kw in (("NVFP4 4/6", {}), ("MXFP4", dict(fmt=fp4.FORMAT_MXFP4, flags=0))):
        print("%-10s last outputs off by %s of the bf16 cache's" % (
            name, ", ".join("%.3f" % e for e in run(**kw))), flush=True)
