"""Paged compressed KV cache: store, load, attention of new tokens and eviction, in
float64 numpy, one sequence, head and slot after the other.

Sources: the quantiser and the cache's grouping are ``oracle.codec`` (the walkthrough page
«FlexGen 单 GPU 高吞吐大模型推理引擎：论文解读与源码实战指南», section 6.3); the order load_cache, compute_layer,
store_cache and attention to the cached tokens plus the fresh ones come from the
source-notes page «FlexGen» (PtirisNote), "Flex Opt". Pages, ragged batches, shared key heads
and eviction have no counterpart there: their definitions are this module's.
"""
import numpy as np

from . import codec


class PagedCache:
    """Pools [pages][heads][page]..., a page table and the slots each sequence holds."""

    def __init__(self, table, ctx, pages, page, heads, dim, bits=4, group=64):
        self.table, self.ctx = np.asarray(table), np.asarray(ctx).copy()
        self.page, self.heads, self.dim, self.bits, self.group = page, heads, dim, bits, group
        shape = (pages, heads, page)
        self.codes = {n: np.zeros(shape + (dim * bits // 8,), np.uint8) for n in "kv"}
        self.meta = {n: np.zeros(shape + (dim // group, 2), np.float16) for n in "kv"}
        self.weight = np.zeros(shape, np.float64)
        self.pos = np.zeros(shape, np.int32)

    def at(self, b, slot):
        return int(self.table[b, slot // self.page]), slot % self.page

    def store(self, b, k16, v16, pos0=None):
        """New rows [n][heads][dim] of sequence b behind its slots (ctx is not changed)."""
        start = int(self.ctx[b]) if pos0 is None else pos0
        for n, x in (("k", k16), ("v", v16)):
            codes, meta = codec.compress(np.ascontiguousarray(x), self.bits, self.group, 2)
            for i in range(len(x)):
                p, s = self.at(b, int(self.ctx[b]) + i)
                self.codes[n][p, :, s] = codes[i]
                self.meta[n][p, :, s] = meta[i]
                self.pos[p, :, s] = start + i

    def load(self, b, start, count):
        """The codec's fp16 values of slots [start, start + count), [count][heads][dim] each."""
        out = []
        for n in "kv":
            x = np.zeros((count, self.heads, self.dim), np.float16)
            for i in range(count):
                p, s = self.at(b, start + i)
                x[i] = codec.decompress(self.codes[n][p, :, s], self.meta[n][p, :, s], (self.heads, self.dim),
                                        self.bits, self.group, 1)
            out.append(x)
        return out

    def values(self, n, b, head):
        """What attention takes the slots for: fp16(c * fp16(1/scale) + min), rounded once."""
        rows = np.zeros((int(self.ctx[b]), self.dim))
        for j in range(int(self.ctx[b])):
            p, s = self.at(b, j)
            c = codec.unpack(self.codes[n][p, head, s].reshape(self.dim // self.group, -1), self.bits).astype(np.float64)
            lo, scale = (self.meta[n][p, head, s, :, i].astype(np.float64)[:, None] for i in (0, 1))
            step = np.where(scale > 0, np.float16(1.0 / np.where(scale > 0, scale, 1.0)), 0.0).astype(np.float64)
            rows[j] = np.float16(c * step + lo).astype(np.float64).reshape(-1)
        return rows

    def attend(self, b, q, k_new=None, v_new=None):
        """q [n][heads * share][dim]; k_new, v_new [n][heads][dim] or None (cross attention).
        Returns o, lse, the probabilities' sums [heads][slots + fresh], and for error bounds the
        largest sum of |q_i k_i| of each row."""
        n, nq, _ = q.shape
        share, ctx = nq // self.heads, int(self.ctx[b])
        o, lse = np.zeros((n, nq, self.dim)), np.full((n, nq), -np.inf)
        size = np.zeros((n, nq))
        sums = np.zeros((self.heads, ctx + (0 if k_new is None else n)))
        for g in range(self.heads):
            k, v = self.values("k", b, g), self.values("v", b, g)
            if k_new is not None:
                k, v = (np.concatenate([x, y[:, g].astype(np.float64)]) for x, y in ((k, k_new), (v, v_new)))
            for h in range(g * share, (g + 1) * share):
                for i in range(n):
                    m = ctx + (0 if k_new is None else i + 1)
                    if m == 0:
                        continue
                    qi = q[i, h].astype(np.float64)
                    sc = k[:m] @ qi
                    size[i, h] = (np.abs(k[:m]) @ np.abs(qi)).max()
                    lse[i, h] = sc.max() + np.log(np.exp(sc - sc.max()).sum())
                    p = np.exp(sc - lse[i, h])
                    o[i, h] = p @ v[:m]
                    sums[g, :m] += p
        return o, lse, sums, size

    def accumulate(self, b, sums):
        for j in range(sums.shape[1]):
            p, s = self.at(b, j)
            self.weight[p, :, s] = (self.weight[p, :, s] if j < self.ctx[b] else 0.0) + sums[:, j]

    def evict(self, budget, recent):
        """Keeps `budget` slots per head; returns the new lengths (ctx is not changed)."""
        for b, n in enumerate(self.ctx):
            n = int(n)
            if n <= budget:
                continue
            for h in range(self.heads):
                where = [self.at(b, j) for j in range(n)]
                pos = [int(self.pos[p, h, s]) for p, s in where]
                w = [float(self.weight[p, h, s]) for p, s in where]
                w = [-np.inf if np.isnan(x) else x for x in w]
                first = [x > max(pos) - recent for x in pos]
                order = sorted(range(n), key=lambda j: (not first[j], 0.0 if first[j] else -w[j], j))
                kept = set(order[:budget])
                holes = [j for j in range(budget) if j not in kept]
                movers = [j for j in range(budget, n) if j in kept]
                for to, come in zip(holes, movers):
                    (dp, ds), (sp, ss) = where[to], where[come]
                    for pool in (*self.codes.values(), *self.meta.values(), self.weight, self.pos):
                        pool[dp, h, ds] = pool[sp, h, ss]
        return np.minimum(self.ctx, budget)
