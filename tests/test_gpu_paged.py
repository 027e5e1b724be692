"""Parity of the paged KV cache's store, load, attention and eviction with the float64
oracle, at the sizes and masks where they can go wrong, one after the other as a serving
step uses them, captured and replayed, and with what only the device can refuse.

Tolerances, with u = 2^-11 (half a step of fp16) and e = 2^-24 (of fp32):
  a score is a sum of head_dim exact products in fp32: at most (head_dim + 4) e times the sum
  of their magnitudes `size`, the factor log2 e and the subtraction of the maximum among
  them; one exponential is within 2^-21 of its value. So a probability is off by
      ep = 2 (head_dim + 4) e size + 2^-21, relative,
  the log-sum-exp by ep + keys e + 2 e |lse|, an accumulated weight by (2 ep + rows e) of what
  was added and e of the whole (both statistics and score enter).
  The output: probabilities rounded to fp16 (u, and 2^-25 where they underflow, against a
  largest one of 1), sums of `keys` terms, and one rounding: u |o| + (u + 2 ep + keys e)
  max|v| + keys 2^-25 max|v|."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import group_wise_int4_b200 as fq
from oracle.paged import PagedCache
from _helpers import sync_status, to_np

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U, E = 2.0 ** -11, 2.0 ** -24
TAIL = 2


class Case:
    """A cache on the device and the oracle's, filled through the device's own store."""

    def __init__(self, seed, ctx, heads=2, dim=64, bits=4, group=32, page=16, room=0, weights=True, spare=2):
        r = self.r = np.random.default_rng(seed)
        self.heads, self.dim, self.bits, self.group, self.page = heads, dim, bits, group, page
        per = [max(1, -(-(n + room) // page)) for n in ctx]
        pages = sum(per) + spare
        ids = r.permutation(pages)
        table = np.full((len(ctx), max(per)), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = ids[at:at + n]
            at += n
        self.ref = PagedCache(table, np.zeros(len(ctx), np.int32), pages, page, heads, dim, bits, group)
        self.ctx = torch.zeros(len(ctx), dtype=torch.int32, device="cuda")
        self.cache = fq.FlexPagedCache(torch.from_numpy(table).cuda(), self.ctx, pages, page, heads, dim, bits, group,
                                       weight=weights or None, slot_pos=weights or None)
        for t in (self.cache.k_codes, self.cache.v_codes):
            t.fill_(0xA5)                                  # what no call writes is not zero
        for t in (self.cache.k_meta, self.cache.v_meta):
            t.fill_(float("nan"))
        self.level = r.standard_normal((heads, dim))
        if sum(ctx):
            self.store([self.rows(n) for n in ctx], [self.rows(n) for n in ctx], advance=True)

    def rows(self, n, heads=None):
        h = heads or self.heads
        return (self.r.standard_normal((n, h, self.dim)) + self.level[np.arange(h) % self.heads]).astype(np.float16)

    def ragged(self, parts):
        """Rows of every sequence -> a strided device tensor with rows behind the last one, and offsets."""
        width = int(np.prod(parts[0].shape[1:]))
        flat = np.concatenate([x.reshape(len(x), width) for x in parts] + [np.full((TAIL, width), 7.5, np.float16)])
        wide = torch.full((len(flat), flat.shape[1] + 24), 9.0, dtype=torch.float16, device="cuda")
        wide[:, 8:8 + flat.shape[1]] = torch.from_numpy(flat).cuda()
        cu = np.concatenate([[0], np.cumsum([len(x) for x in parts])]).astype(np.int32)
        return wide[:, 8:], torch.from_numpy(cu).cuda(), int(cu[-1]), max(len(x) for x in parts)

    def set_ctx(self, lens):
        self.ref.ctx = np.asarray(lens).copy()
        self.ctx.copy_(torch.as_tensor(np.asarray(lens), dtype=torch.int32))

    def store(self, k, v, advance=False, pos0=None):
        kd, cu, total, most = self.ragged(k)
        vd = self.ragged(v)[0]
        p = None if pos0 is None else torch.as_tensor(pos0, dtype=torch.int32, device="cuda")
        fq.flex_paged_store_kv(self.cache, kd, vd, kd.stride(0), cu, most, pos0=p, total=total)
        for b in range(len(k)):
            self.ref.store(b, k[b], v[b], None if pos0 is None else int(pos0[b]))
        if advance:
            self.set_ctx([n + len(x) for n, x in zip(self.ref.ctx, k)])

    def slots(self, pool, b, n):
        """[heads][n]... of the device's pool."""
        t = to_np(pool)
        return np.stack([t[self.ref.at(b, j)[0], :, self.ref.at(b, j)[1]] for j in range(n)], 1) if n else None

    def check_slots(self, what="", weights=False, tol=None):
        for b, n in enumerate(self.ref.ctx):
            for name in "kv":
                for i in range(int(n)):
                    p, s = self.ref.at(b, i)
                    got = to_np(getattr(self.cache, name + "_codes")[p, :, s])
                    assert np.array_equal(got, self.ref.codes[name][p, :, s]), (what, name, b, i)
                    got = to_np(getattr(self.cache, name + "_meta")[p, :, s]).view(np.uint16)
                    assert np.array_equal(got, self.ref.meta[name][p, :, s].view(np.uint16)), (what, name, b, i)
            if self.cache.slot_pos is not None:
                for i in range(int(n)):
                    p, s = self.ref.at(b, i)
                    assert np.array_equal(to_np(self.cache.slot_pos[p, :, s]), self.ref.pos[p, :, s]), (what, b, i)

    def attend(self, q, k=None, v=None, accumulate=False, lse=True, check=True, ws=None, stream=None):
        nq = q[0].shape[1]
        qd, cu, total, most = self.ragged(q)
        o = torch.full((total + TAIL, nq * self.dim), 3.25, dtype=torch.float16, device="cuda")
        ls = torch.full((total + TAIL, nq), 3.25, device="cuda") if lse else None
        kd, vd, ks = None, None, 0
        if k is not None:
            kd, vd = self.ragged(k)[0], self.ragged(v)[0]
            ks = kd.stride(0)
        if ws is None:
            ws = torch.full((fq.flex_paged_attention_ws_bytes(self.cache, nq, total, most, accumulate, batch=len(q)),), 0xFF,
                            dtype=torch.uint8, device="cuda")
        before = self.cache.weight.clone() if accumulate else None
        fq.flex_paged_attention(self.cache, qd, qd.stride(0), nq, kd, vd, ks, o, ls, cu, most, ws, accumulate=accumulate,
                                total=total, stream=stream)
        sync_status()
        assert bool((o[total:] == 3.25).all()) and (ls is None or bool((ls[total:] == 3.25).all())), "rows behind the last"
        if check:
            self.check_attention(q, k, v, o, ls, before)
        return o, ls

    def check_attention(self, q, k, v, o, ls, before=None):
        o, ls = to_np(o).astype(np.float64), None if ls is None else to_np(ls).astype(np.float64)
        at = 0
        for b in range(len(q)):
            n, nq = q[b].shape[:2]
            ro, rl, sums, size = self.ref.attend(b, q[b], None if k is None else k[b], None if v is None else v[b])
            got = o[at:at + n].reshape(n, nq, self.dim)
            keys = sums.shape[1]
            ep = 2 * (self.dim + 4) * E * size + 2.0 ** -21
            vmax = max([np.abs(self.ref.values("v", b, g)).max(initial=0) for g in range(self.heads)] +
                       ([] if v is None else [np.abs(v[b].astype(np.float64)).max(initial=0)]))
            tol = U * np.abs(ro) + (U + 2 * ep + keys * (E + 2.0 ** -25))[..., None] * vmax
            err = np.abs(got - ro)
            assert np.all(err <= tol), (b, np.unravel_index(np.argmax(err - tol), err.shape), (err - tol).max())
            if ls is not None:
                lt = ls[at:at + n]
                some = np.isfinite(rl)
                assert np.array_equal(np.isfinite(lt), some) and np.all(lt[~some] == -np.inf)
                bound = ep + keys * E + 2 * E * np.abs(np.where(some, rl, 0))
                assert np.all(np.abs(lt[some] - rl[some]) <= bound[some]), b
            if before is not None and n:
                grown = int(self.ref.ctx[b]) + (0 if k is None else n)
                old = self.slots(before, b, grown)
                new = self.slots(self.cache.weight, b, grown)
                if old is not None:
                    old = old.astype(np.float64)
                    old[:, int(self.ref.ctx[b]):] = 0
                    want = old + sums
                    rows = n * nq // self.heads
                    bound = (2 * ep.max(initial=0) + keys * E + rows * E + 4 * E) * sums + 2 * E * np.abs(want) + 1e-30
                    assert np.all(np.abs(new - want) <= bound), (b, np.abs(new - want).max())
            at += n


def _scaled(c, n, heads):
    return [(x * c.dim ** -0.5).astype(np.float16) for x in (c.rows(m, heads) for m in n)]


SHAPES = [(64, 4, 32, 16), (64, 4, 64, 32), (64, 8, 32, 64), (64, 8, 64, 16), (128, 4, 32, 128), (128, 4, 64, 16),
          (128, 8, 32, 32), (128, 8, 64, 1024)]


@pytest.mark.parametrize("dim,bits,group,page", SHAPES)
def test_store_and_load(dim, bits, group, page):
    c = Case(1, [0, 17, 33, 1], heads=3, dim=dim, bits=bits, group=group, page=page, room=40)
    c.check_slots("filled")
    n = [5, 0, 1, 39]
    k, v = [c.rows(m) for m in n], [c.rows(m) for m in n]
    k[0][1, 0, :group] = 0.5                       # a constant group
    k[3][2, 1, :group] = -0.0
    v[0][3] *= np.float16(300)
    c.store(k, v, advance=True, pos0=[100, 7, 2 ** 20, 0])
    sync_status()
    c.check_slots("added")
    # every slot's value, as the codec gives it; rows behind the last one stay
    start, count = [0, 3, 16, 39], [5, 14, 18, 1]
    outs = [torch.full((sum(count) + TAIL, 3 * dim + 8), 5.0, dtype=torch.float16, device="cuda") for _ in "kv"]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(count)]), dtype=torch.int32, device="cuda")
    fq.flex_paged_load_kv(c.cache, outs[0], outs[1], 3 * dim + 8, cu, max(count), total=sum(count),
                          start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    sync_status()
    at = 0
    for b in range(4):
        for x, ref in zip(outs, c.ref.load(b, start[b], count[b])):
            got = to_np(x[at:at + count[b], :3 * dim]).reshape(count[b], 3, dim)
            assert np.array_equal(got.view(np.uint16), ref.view(np.uint16)), b
        at += count[b]
    for x in outs:
        assert bool((x[at:] == 5).all()) and bool((x[:, 3 * dim:] == 5).all())


def test_store_equal_counts_without_offsets():
    c = Case(2, [3, 20], room=8)
    k, v = [c.rows(4), c.rows(4)], [c.rows(4), c.rows(4)]
    kd, vd = (torch.from_numpy(np.concatenate(x).reshape(8, -1)).cuda() for x in (k, v))
    fq.flex_paged_store_kv(c.cache, kd, vd, kd.stride(0), None, 4)
    for b in range(2):
        c.ref.store(b, k[b], v[b])
    c.set_ctx([7, 24])
    sync_status()
    c.check_slots()


@pytest.mark.parametrize("dim,bits,group,page", SHAPES)
@pytest.mark.parametrize("share", [1, 4])
def test_one_token(dim, bits, group, page, share):
    ctx = [0, 1, 15, 16, 127, 128, 129, 300]
    c = Case(3, ctx, heads=3, dim=dim, bits=bits, group=group, page=page, room=1)
    n = [1] * len(ctx)
    c.attend(_scaled(c, n, 3 * share), [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True)


@pytest.mark.parametrize("dim,bits,group,page", SHAPES)
@pytest.mark.parametrize("share", [1, 3])
def test_chunks(dim, bits, group, page, share):
    ctx, n = [0, 5, 64, 200, 131, 17], [40, 1, 0, 19, 130, 7]
    c = Case(4, ctx, heads=2, dim=dim, bits=bits, group=group, page=page, room=130)
    c.attend(_scaled(c, n, 2 * share), [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True)


@pytest.mark.parametrize("dim,bits,group,page", SHAPES)
@pytest.mark.parametrize("n", [[1, 1, 1, 1], [3, 129, 0, 64]])
def test_cross(dim, bits, group, page, n):
    c = Case(5, [0, 130, 33, 64], heads=2, dim=dim, bits=bits, group=group, page=page)
    c.attend(_scaled(c, n, 4), accumulate=True)


def test_one_long_sequence_is_split():
    """Few rows over long histories: parts of one sequence's keys are joined."""
    c = Case(6, [5000, 3, 2100], heads=1, dim=64, bits=4, group=64, page=64, room=4)
    for n in ([1, 1, 1], [4, 2, 3]):
        c.attend(_scaled(c, n, 2), [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True)


def test_many_sequences():
    ctx = [(7 * i) % 61 for i in range(70)]
    c = Case(7, ctx, heads=1, page=16, room=3)
    n = [i % 4 for i in range(70)]
    c.attend(_scaled(c, n, 2), [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True)


def test_without_lse_and_weights():
    c = Case(8, [30, 200], weights=False)
    q, k, v = _scaled(c, [1, 1], 2), [c.rows(1), c.rows(1)], [c.rows(1), c.rows(1)]
    o, _ = c.attend(q, k, v, lse=False)
    o2, _ = c.attend(q, k, v)
    assert torch.equal(o, o2)


def test_weights_without_lse_output():
    c = Case(9, [30, 200], room=9)
    n = [9, 2]
    c.attend(_scaled(c, n, 2), [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True, lse=False)


def test_large_scores():
    """Scores of several thousand, of both signs: the running maximum moves, nothing overflows."""
    c = Case(10, [100, 40, 3], dim=64, room=20)
    for n in ([1, 1, 1], [20, 3, 1]):
        q = [(x * np.float16(60)) for x in (c.rows(m, 2) for m in n)]
        c.attend(q, [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True)


@pytest.mark.parametrize("bits,dim", [(4, 64), (4, 128), (8, 64), (8, 128)])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_hidden_tokens_do_not_reach_earlier_rows(bits, dim, bad):
    """A later token's key and value are not seen by earlier rows, whatever they hold."""
    c = Case(11, [20, 0], dim=dim, bits=bits, room=40)
    n = [40, 21]
    q, k, v = _scaled(c, n, 4), [c.rows(m) for m in n], [c.rows(m) for m in n]
    o, ls = c.attend(q, k, v)
    k2, v2 = [x.copy() for x in k], [x.copy() for x in v]
    k2[0][33, 1, 5], v2[0][33, 0, 7] = bad, bad
    v2[1][20] = bad
    o2, ls2 = c.attend(q, k2, v2, check=False)
    assert torch.equal(o[:33], o2[:33]) and torch.equal(ls[:33], ls2[:33])
    assert torch.equal(o[40:60], o2[40:60])
    got = to_np(o2).reshape(-1, 4, dim)
    # head pair 0 sees the bad value in dim 7 only, head pair 1 the bad key everywhere
    assert not np.isfinite(got[33:40, :2, 7].astype(np.float64)).any()
    keep = np.delete(np.arange(dim), 7)
    assert np.isfinite(got[33:40, :2][..., keep].astype(np.float64)).all()
    assert not np.isfinite(got[60].astype(np.float64)).any()


@pytest.mark.parametrize("one", [True, False])
def test_slots_behind_the_last_are_not_read(one):
    """The page a sequence ends in holds NaN metadata behind its last slot (Case fills it)."""
    c = Case(12, [1, 18, 129], dim=128, bits=8, page=64)
    n = [1, 1, 1] if one else [30, 2, 17]
    o, ls = c.attend(_scaled(c, n, 2))
    assert bool(torch.isfinite(o.float()).all()) and bool(torch.isfinite(ls).all())


def test_results_repeat():
    """The same call gives the same bits, weights too: no sum's order depends on timing."""
    c = Case(13, [900, 40, 0], heads=2, dim=64, room=33)
    n = [33, 1, 9]
    q, k, v = _scaled(c, n, 4), [c.rows(m) for m in n], [c.rows(m) for m in n]
    c.cache.weight.zero_()
    first = c.attend(q, k, v, accumulate=True, check=False)
    w = c.cache.weight.clone()
    for _ in range(3):
        c.cache.weight.zero_()
        again = c.attend(q, k, v, accumulate=True, check=False)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]) and torch.equal(w, c.cache.weight)


def test_two_streams_with_their_own_workspaces():
    c = Case(14, [1500, 3, 700], heads=2, room=40)
    calls = []
    for n in ([1, 1, 1], [40, 5, 17]):
        q, k, v = _scaled(c, n, 4), [c.rows(m) for m in n], [c.rows(m) for m in n]
        calls.append((n, q, k, v, c.attend(q, k, v)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    torch.cuda.synchronize()
    args = []
    for n, q, k, v, _ in calls:
        qd, cu, total, most = c.ragged(q)
        kd, vd = c.ragged(k)[0], c.ragged(v)[0]
        ws = torch.empty(fq.flex_paged_attention_ws_bytes(c.cache, 4, total, most), dtype=torch.uint8, device="cuda")
        o = torch.empty((total, 4 * c.dim), dtype=torch.float16, device="cuda")
        ls = torch.empty((total, 4), device="cuda")
        args.append((qd, qd.stride(0), 4, kd, vd, kd.stride(0), o, ls, cu, most, ws, False, total))
    torch.cuda.synchronize()
    for _ in range(5):
        for st, a in zip(streams, args):
            fq.flex_paged_attention(c.cache, *a[:11], accumulate=a[11], total=a[12], stream=st)
    torch.cuda.synchronize()
    sync_status()
    for a, (_, _, _, _, (o, ls)) in zip(args, calls):
        total = a[12]
        assert torch.equal(a[6], o[:total]) and torch.equal(a[7], ls[:total])


@pytest.mark.parametrize("bits,dim,group,page", [(4, 64, 32, 16), (4, 128, 64, 64), (8, 64, 64, 16), (8, 128, 32, 128)])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (16, 3), (40, 40), (64, 0), (100, 20)])
def test_evict(bits, dim, group, page, budget, recent):
    ctx = [0, 1, 63, 64, 65, 200, 101]
    c = Case(15, ctx, heads=3, dim=dim, bits=bits, group=group, page=page)
    _evict(c, budget, recent)


def _evict(c, budget, recent, fill=True):
    if fill:
        w = c.r.standard_normal(tuple(c.cache.weight.shape)).astype(np.float32)
        w[c.r.random(w.shape) < 0.4] = 0.25                # many equal ones
        w[c.r.random(w.shape) < 0.05] = np.nan
        w[c.r.random(w.shape) < 0.05] = np.inf
        w[c.r.random(w.shape) < 0.05] = -0.0
        w[c.r.random(w.shape) < 0.05] = -np.inf
        c.cache.weight.copy_(torch.from_numpy(w))
        c.ref.weight = w.astype(np.float64)
        pos = c.r.permutation(w.size).astype(np.int32).reshape(w.shape)
        c.cache.slot_pos.copy_(torch.from_numpy(pos))
        c.ref.pos = pos.copy()
    new = torch.zeros(c.cache.batch, dtype=torch.int32, device="cuda")
    ws = torch.full((fq.flex_paged_evict_ws_bytes(c.cache, budget),), 0xFF, dtype=torch.uint8, device="cuda")
    fq.flex_paged_evict(c.cache, budget, recent, new, ws)
    sync_status()
    lens = c.ref.evict(budget, recent)
    assert np.array_equal(to_np(new), lens)
    c.set_ctx(lens)
    c.check_slots("evicted")
    for b, n in enumerate(lens):
        if n:
            ref = np.stack([c.ref.weight[c.ref.at(b, j)[0], :, c.ref.at(b, j)[1]] for j in range(int(n))], 1)
            assert np.array_equal(c.slots(c.cache.weight, b, int(n)).astype(np.float64), ref, equal_nan=True), b


def test_evict_many_slots():
    """More slots than the selection keeps in shared memory at once."""
    n = 40000
    c = Case(16, [0, 0], heads=2, dim=64, bits=4, group=64, page=1024, room=n)
    w = torch.rand(tuple(c.cache.weight.shape), device="cuda").mul_(64).round_()
    pos = torch.randperm(w.numel(), device="cuda").to(torch.int32).view(w.shape)
    for t in (c.cache.k_codes, c.cache.v_codes):
        t.random_(0, 256)
    c.cache.weight.copy_(w)
    c.cache.slot_pos.copy_(pos)
    c.ctx.copy_(torch.tensor([n, 33000], dtype=torch.int32))
    codes = c.cache.k_codes.clone()
    budget, recent = 9000, 500
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(fq.flex_paged_evict_ws_bytes(c.cache, budget), dtype=torch.uint8, device="cuda")
    fq.flex_paged_evict(c.cache, budget, recent, new, ws)
    sync_status()
    assert new.tolist() == [budget, budget]
    for b, m in enumerate((n, 33000)):
        ids = to_np(c.cache.page_table[b]).astype(np.int64)
        for h in range(2):
            ww, pp = (to_np(t[ids, h]).reshape(-1)[:m] for t in (w, pos))
            first = pp > pp.max() - recent
            order = np.lexsort((np.arange(m), -np.where(first, 0, ww), ~first))
            kept = np.zeros(m, bool)
            kept[order[:budget]] = True
            src = np.arange(budget)
            src[~kept[:budget]] = np.nonzero(kept)[0][kept[:budget].sum():]
            got = to_np(c.cache.slot_pos[ids, h]).reshape(-1)[:budget]
            assert np.array_equal(got, pp[src])
            old, now = (to_np(t[ids, h]).reshape(-1, codes.shape[-1])[:m] for t in (codes, c.cache.k_codes))
            assert np.array_equal(now[:budget], old[src]) and np.array_equal(now[budget:], old[budget:])


def test_a_bounded_cache_step_by_step():
    """Chunks, single tokens and evictions in turn, as a serving loop uses the operators; the
    oracle follows with the device's own weights, so that equal choices are compared."""
    c = Case(17, [0, 0, 0], heads=2, dim=64, bits=4, group=64, page=16, room=96)
    pos = np.zeros(3, np.int64)
    budget, recent = 48, 12
    for n in ([40, 7, 1], [1, 30, 1], [20, 1, 33], [1, 1, 1], [1, 1, 1], [30, 2, 0], [1, 1, 1]):
        q, k, v = _scaled(c, n, 4), [c.rows(m) for m in n], [c.rows(m) for m in n]
        c.attend(q, k, v, accumulate=True)
        c.store(k, v, advance=True, pos0=pos.astype(np.int32))
        pos += n
        c.check_slots("stored")
        c.ref.weight = to_np(c.cache.weight).astype(np.float64)
        _evict(c, budget, recent, fill=False)


def test_captured_calls_follow_their_inputs():
    """A captured step replayed with other lengths, tables and rows."""
    c = Case(18, [700, 30, 0], heads=2, dim=64, room=64)
    n0 = [1, 40, 9]
    q, k, v = _scaled(c, n0, 4), [c.rows(m) for m in n0], [c.rows(m) for m in n0]
    qd, cu, total, most = c.ragged(q)
    kd, vd = c.ragged(k)[0], c.ragged(v)[0]
    o = torch.empty((total, 4 * c.dim), dtype=torch.float16, device="cuda")
    ls = torch.empty((total, 4), device="cuda")
    ws = torch.empty(fq.flex_paged_attention_ws_bytes(c.cache, 4, total, most, True), dtype=torch.uint8, device="cuda")
    ew = torch.empty(fq.flex_paged_evict_ws_bytes(c.cache, 600), dtype=torch.uint8, device="cuda")
    new = torch.zeros(3, dtype=torch.int32, device="cuda")

    def step():
        fq.flex_paged_attention(c.cache, qd, qd.stride(0), 4, kd, vd, kd.stride(0), o, ls, cu, most, ws, accumulate=True,
                                total=total)
        fq.flex_paged_store_kv(c.cache, kd, vd, kd.stride(0), cu, most, total=total)
        fq.flex_paged_evict(c.cache, 600, 50, new, ew)

    weight, pools = c.cache.weight.clone(), [t.clone() for t in (c.cache.k_codes, c.cache.k_meta, c.cache.v_codes,
                                                                  c.cache.v_meta, c.cache.slot_pos)]

    def restore():
        for t, x in zip((c.cache.k_codes, c.cache.k_meta, c.cache.v_codes, c.cache.v_meta, c.cache.slot_pos), pools):
            t.copy_(x)
        c.cache.weight.copy_(weight)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()                                             # kernels are loaded outside the capture
    torch.cuda.synchronize()
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n, ctx in ((n0, [700, 30, 0]), ([40, 1, 9], [650, 30, 0]), ([0, 0, 50 - 12], [700, 30, 0])):
        restore()
        cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32))
        c.set_ctx(ctx)
        graph.replay()
        sync_status()
        qh, kh, vh = (to_np(x[:, :w]) for x, w in ((qd, 4 * c.dim), (kd, 2 * c.dim), (vd, 2 * c.dim)))
        ends = np.concatenate([[0], np.cumsum(n)])
        parts = [[x[a:b].reshape(b - a, x.shape[1] // c.dim, c.dim) for a, b in zip(ends[:-1], ends[1:])] for x in (qh, kh, vh)]
        m = int(ends[-1])
        c.check_attention(*parts, torch.cat([o[:m]]), ls[:m])
        assert new.tolist() == [min(x, 600) for x in ctx]


def test_two_captured_steps_with_their_own_workspaces():
    c = Case(19, [2500, 900], heads=1, dim=64, page=64, room=2)
    graphs = []
    for n in ([1, 1], [2, 1]):
        q, k, v = _scaled(c, n, 2), [c.rows(m) for m in n], [c.rows(m) for m in n]
        want = c.attend(q, k, v)
        qd, cu, total, most = c.ragged(q)
        kd, vd = c.ragged(k)[0], c.ragged(v)[0]
        ws = torch.empty(fq.flex_paged_attention_ws_bytes(c.cache, 2, total, most), dtype=torch.uint8, device="cuda")
        o = torch.empty((total, 2 * c.dim), dtype=torch.float16, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fq.flex_paged_attention(c.cache, qd, qd.stride(0), 2, kd, vd, kd.stride(0), o, None, cu, most, ws, total=total)
        graphs.append((g, o, want[0][:total], (qd, kd, vd, cu, ws)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (g, _, _, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    sync_status()
    for _, o, want, _ in graphs:
        assert torch.equal(o, want)


def _status():
    rc = fq.flex_get_status()
    assert fq.flex_get_status() == fq.FLEX_OK              # it is cleared
    return rc


def test_bad_pages_and_lengths_are_reported():
    """Page ids outside the pool, lengths outside the table and offsets that do not fit are
    reported; nothing is touched through them and the other sequences are right."""
    c = Case(20, [40, 30, 25], heads=2, dim=64, room=16)
    n = [1, 2, 1]
    q, k, v = _scaled(c, n, 2), [c.rows(m) for m in n], [c.rows(m) for m in n]
    qd, cu, total, most = c.ragged(q)
    kd, vd = c.ragged(k)[0], c.ragged(v)[0]
    good, _ = c.attend(q, k, v)
    ws = torch.empty(fq.flex_paged_attention_ws_bytes(c.cache, 2, total, most, True), dtype=torch.uint8, device="cuda")
    o = torch.empty((total, 2 * c.dim), dtype=torch.float16, device="cuda")
    table, ctx, offs = c.cache.page_table.clone(), c.ctx.clone(), cu.clone()

    def attend(acc=False):
        fq.flex_paged_attention(c.cache, qd, qd.stride(0), 2, kd, vd, kd.stride(0), o, None, cu, most, ws, total=total,
                                accumulate=acc)
        return _status()

    def bad(what, where, value, rows):
        what[where] = value
        for acc in (False, True):
            assert attend(acc) == fq.FLEX_ERR_INVALID_ARG
            assert all(torch.equal(o[r], good[r]) for r in rows)
        c.cache.page_table.copy_(table)
        c.ctx.copy_(ctx)
        cu.copy_(offs)

    bad(c.cache.page_table, (1, 0), c.cache.num_pages, [0, 3])
    bad(c.cache.page_table, (1, 1), -1, [0, 3])
    bad(c.ctx, 0, -5, [1, 2, 3])
    bad(c.ctx, 2, 1 << 29, [0, 1, 2])
    bad(cu, 2, 0, [0])                                     # decreasing
    bad(cu, 3, total + 7, [0, 1, 2])                       # behind the rows
    bad(cu, 1, -3, [3])
    before = [t.clone() for t in (c.cache.k_codes, c.cache.v_meta, c.cache.slot_pos)]
    c.ctx[1] = table.shape[1] * c.page                     # no slot left in the table
    fq.flex_paged_store_kv(c.cache, kd, vd, kd.stride(0), cu, most, total=total)
    assert _status() == fq.FLEX_ERR_INVALID_ARG
    p0 = int(table[1, -1])
    if p0 >= 0:
        assert torch.equal(c.cache.k_codes[p0], before[0][p0])
    c.ctx.copy_(ctx)
    out = torch.full((total, 2 * c.dim), 5.0, dtype=torch.float16, device="cuda")
    for start in (-1, 1 << 29):
        s = torch.tensor([0, start, 0], dtype=torch.int32, device="cuda")
        fq.flex_paged_load_kv(c.cache, out, out.clone(), 2 * c.dim, cu, most, total=total, start=s)
        assert _status() == fq.FLEX_ERR_INVALID_ARG
        assert bool((out[1] == 5).all()) and not bool((out[0] == 5).all())
    c.cache.page_table[0, 0] = 1 << 30
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    ew = torch.empty(fq.flex_paged_evict_ws_bytes(c.cache, 8), dtype=torch.uint8, device="cuda")
    fq.flex_paged_evict(c.cache, 8, 2, new, ew)
    assert _status() == fq.FLEX_ERR_INVALID_ARG and new.tolist() == [8, 8, 8]


def test_overlapping_offsets_are_survived():
    """Offsets that repeat rows ask for more tiles than `total` allows: reported or not, no
    call reads or writes outside its tensors, and the next call is right."""
    c = Case(21, [3000] * 6, heads=1, dim=64, page=64, room=2)
    n = [1] * 6
    q, k, v = _scaled(c, n, 1), [c.rows(m) for m in n], [c.rows(m) for m in n]
    good, _ = c.attend(q, k, v)
    qd, cu, total, most = c.ragged(q)
    kd, vd = c.ragged(k)[0], c.ragged(v)[0]
    ws = torch.full((fq.flex_paged_attention_ws_bytes(c.cache, 1, total, 6),), 0x7F, dtype=torch.uint8, device="cuda")
    o = torch.empty((total, c.dim), dtype=torch.float16, device="cuda")
    cu.copy_(torch.tensor([0, 6, 0, 6, 0, 6, 0], dtype=torch.int32))
    fq.flex_paged_attention(c.cache, qd, qd.stride(0), 1, kd, vd, kd.stride(0), o, None, cu, 6, ws, total=total)
    assert _status() == fq.FLEX_ERR_INVALID_ARG
    again, _ = c.attend(q, k, v)
    assert torch.equal(good, again)


def test_pool_larger_than_32_bit_offsets():
    """Slots whose byte offsets pass 2^32, at the end of the pool."""
    pages, heads, page, dim = 1 << 13, 40, 128, 128        # 41.9 M slots of 128 bytes: 5.4 GB a pool
    table = torch.tensor([[pages - 1, pages - 3], [pages - 2, 0]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    shape = (pages, heads, page)
    pools = tuple(torch.empty(shape + s, dtype=t, device="cuda") for s, t in
                  (((dim,), torch.uint8), ((2, 2), torch.float16)) * 2)
    cache = fq.FlexPagedCache(table, ctx, pools=pools, weight=True, slot_pos=True, num_bits=8, group_size=64)
    assert cache.k_codes.numel() > 1 << 32
    r = np.random.default_rng(22)
    rows = [r.standard_normal((140, heads, dim)).astype(np.float16) for _ in range(4)]
    ref = PagedCache([[0, 1], [2, 3]], [0, 0], 4, page, heads, dim, 8, 64)
    kd, vd = (torch.from_numpy(np.concatenate(x).reshape(280, -1)).cuda() for x in (rows[:2], rows[2:]))
    fq.flex_paged_store_kv(cache, kd, vd, heads * dim, None, 140)
    for b in range(2):
        ref.store(b, rows[b], rows[2 + b])
    out = [torch.empty_like(kd), torch.empty_like(vd)]
    fq.flex_paged_load_kv(cache, *out, heads * dim, None, 140)
    ctx.fill_(140)
    ref.ctx[:] = 140
    sync_status()
    for b in range(2):
        for x, want in zip(out, ref.load(b, 0, 140)):
            assert np.array_equal(to_np(x[b * 140:b * 140 + 140]).reshape(140, heads, dim), want)
    for n in (1, 33):
        q = (r.standard_normal((2 * n, heads, dim)) * 0.09).astype(np.float16)
        o = torch.empty((2 * n, heads * dim), dtype=torch.float16, device="cuda")
        ws = torch.empty(fq.flex_paged_attention_ws_bytes(cache, heads, 2 * n, n, True), dtype=torch.uint8, device="cuda")
        fq.flex_paged_attention(cache, torch.from_numpy(q).cuda().view(2 * n, -1), heads * dim, heads, None, None, 0, o, None,
                                None, n, ws, accumulate=True)
        sync_status()
        for b in range(2):
            small = PagedCache([[0, 1], [2, 3]], [140, 140], 4, page, 1, dim, 8, 64)
            for h in (0, heads - 1):
                for name in "kv":
                    small.codes[name][:, 0], small.meta[name][:, 0] = ref.codes[name][:, h], ref.meta[name][:, h]
                want = small.attend(b, q[b * n:b * n + n, h:h + 1])[0][:, 0]
                got = to_np(o[b * n:b * n + n, h * dim:(h + 1) * dim]).astype(np.float64)
                assert np.all(np.abs(got - want) <= U * np.abs(want) + 2 * U * 5.0)
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    ew = torch.empty(fq.flex_paged_evict_ws_bytes(cache, 100), dtype=torch.uint8, device="cuda")
    fq.flex_paged_evict(cache, 100, 10, new, ew)
    sync_status()
    assert new.tolist() == [100, 100]


def test_the_whole_batch_is_empty():
    c = Case(23, [0, 0], heads=2, room=16)
    c.attend([c.rows(0, 2), c.rows(0, 2)], [c.rows(0), c.rows(0)], [c.rows(0), c.rows(0)])
    o, ls = c.attend(_scaled(c, [2, 1], 2))
    assert not bool(o[:3].any()) and bool((ls[:3] == float("-inf")).all())


@pytest.mark.parametrize("dim,bits,group,page", SHAPES)
@pytest.mark.parametrize("most", [12, 20, 64, 200])
def test_every_row_tile(dim, bits, group, page, most):
    """8 and 16 rows of the rows kernel, one and two of the latter's tiles, and 128 and 256 rows."""
    ctx = [0, 63, 64, 65, 300]
    n = [most, 1, most // 2, 0, most - 3]
    c = Case(30 + most, ctx, heads=2, dim=dim, bits=bits, group=group, page=page, room=most)
    c.attend(_scaled(c, n, 2), [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True)
    c.attend(_scaled(c, n, 2))


@pytest.mark.parametrize("most", [30, 100, 290])
def test_long_histories_are_split(most):
    """Few sequences: the tiles' keys are cut into parts and joined."""
    c = Case(31, [4000, 10, 2300], heads=1, dim=64, bits=4, group=64, page=64, room=most)
    n = [most, 2, most // 3]
    c.attend(_scaled(c, n, 1), [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True)
    c.attend(_scaled(c, n, 1))


def test_many_ragged_sequences():
    """More sequences than a warp has lanes, with tiles of 128 rows and with splits."""
    ctx = [(37 * i) % 260 for i in range(45)] + [3100]
    c = Case(32, ctx, heads=1, dim=128, bits=8, group=64, page=32, room=41)
    n = [(5 * i) % 41 for i in range(45)] + [40]
    c.attend(_scaled(c, n, 1), [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True)


@pytest.mark.parametrize("dim", [64, 128])
def test_evict_tables_of_several_kinds(dim):
    """Up to 2048 slots a table, few and many moves, and more slots."""
    for seed, ctx, page, room, budget, recent in ((33, [2048, 2000, 9], 1024, 0, 2040, 100), (34, [2048, 1100], 128, 0, 700, 650),
                                                  (35, [2100, 3000, 50], 64, 200, 1000, 30), (36, [1500], 16, 0, 1499, 0)):
        _evict(Case(seed, ctx, heads=2, dim=dim, bits=4, group=32, page=page, room=room), budget, recent)


def test_one_sequence_of_the_table():
    """batch smaller than the table's: the first sequences alone."""
    c = Case(37, [70, 30, 5], heads=2, room=3)
    q, k, v = _scaled(c, [2], 2), [c.rows(2)], [c.rows(2)]
    qd, cu, total, most = c.ragged(q)
    kd, vd = c.ragged(k)[0], c.ragged(v)[0]
    o = torch.empty((total, 2 * c.dim), dtype=torch.float16, device="cuda")
    ls = torch.empty((total, 2), device="cuda")
    for b, rows in ((None, cu), (1, None)):
        ws = torch.empty(fq.flex_paged_attention_ws_bytes(c.cache, 2, total, most, batch=1), dtype=torch.uint8, device="cuda")
        fq.flex_paged_attention(c.cache, qd, qd.stride(0), 2, kd, vd, kd.stride(0), o, ls, rows, most, ws, total=total, batch=b)
        sync_status()
        c.check_attention(q, k, v, o, ls)


def test_masks_of_the_lowest_value():
    """Scores that overflow to -infinity (a key of the lowest values) weigh nothing; a row whose
    only key is one attends to it all the same or to nothing, but is never NaN by accident."""
    c = Case(38, [5, 0], heads=1, dim=64, room=40)
    q = [np.full((2, 1, 64), 60000, np.float16), np.full((40, 1, 64), 60000, np.float16)]
    k = [np.full((2, 1, 64), -60000, np.float16), np.full((40, 1, 64), -60000, np.float16)]
    v = [c.rows(2), c.rows(40)]
    c.attend(q, k, v, accumulate=True)


def test_workspace_contents_do_not_matter():
    c = Case(39, [2600, 700], heads=1, dim=64, page=64, room=60)
    for n in ([1, 1], [60, 3]):
        q, k, v = _scaled(c, n, 1), [c.rows(m) for m in n], [c.rows(m) for m in n]
        outs = []
        for fill in (0, 0x7F, 0xFF):
            size = fq.flex_paged_attention_ws_bytes(c.cache, 1, sum(n), max(n), True)
            c.cache.weight.zero_()
            o, ls = c.attend(q, k, v, accumulate=True, check=False,
                             ws=torch.full((size,), fill, dtype=torch.uint8, device="cuda"))
            outs.append((o, ls, c.cache.weight.clone()))
        for x in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(outs[0], x))


@pytest.mark.parametrize("most", [1, 5])
def test_tables_far_longer_than_the_sequences(most):
    """The weights' pass over a table of a million slots a sequence, of which few are held."""
    c = Case(40, [300, 20, 130], heads=6, dim=64, page=1024, room=most)
    wide = torch.full((3, 1 << 10), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.cache.page_table.shape[1]] = c.cache.page_table
    c.cache.page_table, c.cache.max_pages = wide, 1 << 10
    n = [most, 1, most]
    for _ in range(2):
        c.attend(_scaled(c, n, 12), [c.rows(m) for m in n], [c.rows(m) for m in n], accumulate=True)
    one = [1, 1, 1]
    c.attend(_scaled(c, one, 6), [c.rows(1)] * 3, [c.rows(1)] * 3, accumulate=True)


@pytest.mark.parametrize("bits,dim", [(4, 64), (8, 128)])
def test_one_long_prompt_among_single_tokens(bits, dim):
    """Store and load of a batch of 50 sequences of which one has nearly all rows."""
    n = [1 if i % 7 else 0 for i in range(50)]
    n[41] = 333
    c = Case(41, [(3 * i) % 20 for i in range(50)], heads=2, dim=dim, bits=bits, room=333)
    k, v = [c.rows(m) for m in n], [c.rows(m) for m in n]
    start = c.ref.ctx.copy()
    c.store(k, v, advance=True)
    sync_status()
    c.check_slots("added")
    outs = [torch.full((sum(n) + TAIL, 2 * dim), 5.0, dtype=torch.float16, device="cuda") for _ in "kv"]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    fq.flex_paged_load_kv(c.cache, outs[0], outs[1], 2 * dim, cu, max(n), total=sum(n),
                          start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    sync_status()
    at = 0
    for b in range(50):
        for x, ref in zip(outs, c.ref.load(b, int(start[b]), n[b])):
            assert np.array_equal(to_np(x[at:at + n[b]]).reshape(n[b], 2, dim).view(np.uint16), ref.view(np.uint16)), b
        at += n[b]
    assert all(bool((x[at:] == 5).all()) for x in outs)


@pytest.mark.parametrize("most", [60, 200])
def test_a_gemm_right_behind_the_tiles(most):
    """The output projection after a chunk's attention, launch after launch without a pause: the
    GEMM's early blocks and the tiles share the multiprocessors' tensor memory."""
    c = Case(42, [700, 0, 90], heads=4, dim=64, page=64, room=most)
    n = [most, 3, most // 2]
    q, k, v = _scaled(c, n, 8), [c.rows(m) for m in n], [c.rows(m) for m in n]
    want = c.attend(q, k, v)[0]
    qd, cu, total, _ = c.ragged(q)
    kd, vd = c.ragged(k)[0], c.ragged(v)[0]
    W = fq.CompressedWeight(torch.from_numpy((c.r.standard_normal((768, 512)) * 0.05).astype(np.float16)).cuda())
    ws = torch.empty(fq.flex_paged_attention_ws_bytes(c.cache, 8, total, most, True), dtype=torch.uint8, device="cuda")
    gws = torch.zeros(max(16, fq.flex_gemm_ws_bytes(total, 768, 512)), dtype=torch.uint8, device="cuda")
    o = torch.empty((total, 512), dtype=torch.float16, device="cuda")
    ys = [torch.empty((total, 768), dtype=torch.float16, device="cuda") for _ in range(12)]
    fq.flex_dequant_gemm(want[:total].contiguous(), W, None, None, ys[0], total, fq.FLEX_EPI_NONE, gws)
    first = ys[0].clone()
    for i, y in enumerate(ys):
        fq.flex_paged_attention(c.cache, qd, qd.stride(0), 8, kd, vd, kd.stride(0), o, None, cu, most, ws, total=total,
                                accumulate=i % 2 == 1)
        fq.flex_dequant_gemm(o, W, None, None, y, total, fq.FLEX_EPI_NONE, gws)
    sync_status()
    assert torch.equal(o, want[:total]) and all(torch.equal(y, first) for y in ys)


@pytest.mark.parametrize("dim,bits", [(64, 4), (128, 4), (128, 8)])
@pytest.mark.parametrize("share,n", [(1, [1, 1]), (4, [1, 1]), (1, [12, 3]), (2, [40, 5]), (1, [200, 40])])
@pytest.mark.parametrize("size", [40.0, 3000.0, 20000.0])
def test_weights_of_large_scores_are_probabilities(dim, bits, share, n, size):
    """Scores of 1e4 to 1e10, whose fp32 sums are off by up to whole units: the pass that adds the
    weights sums them in another order than the attention did, but what a row adds to a slot is
    a probability all the same."""
    c = Case(43, [150, 70], heads=2, dim=dim, bits=bits, room=max(n))
    k, v = [(c.rows(m) * np.float16(size / 8)) for m in n], [c.rows(m) for m in n]
    q = [c.rows(m, 2 * share) * np.float16(size / 4) for m in n]
    c.cache.weight.zero_()
    c.attend(q, k, v, accumulate=True, check=False)
    for b, m in enumerate(n):
        w = c.slots(c.cache.weight, b, int(c.ref.ctx[b]) + m).astype(np.float64)
        assert np.isfinite(w).all()
        assert w.min() >= 0 and w.max() <= m * share
        assert (w.sum(1) > 0).all()


def _exact_rows(c, n, factors, fine):
    """Key rows of exact integers: 30 dims of the first half are 8 f 2^p (f: 0 or 1 a key), one of the
    second half is the key's fine value, two more are 15 and 8. Each group spans 15 or 255
    steps of a power of two, so the codes are exact."""
    p, top = (12, 15) if c.bits == 4 else (8, 255)
    x = np.zeros((n, c.heads, c.dim), np.float64)
    x[:, :, :30] = 8 * np.asarray(factors)[:, None, None]
    half = c.dim // 2
    x[:, :, half] = np.asarray(fine)[:, None]
    x[:, :, half + 1], x[:, :, half + 2] = 15, 8
    x[:, :, c.group - 1::c.group] = top                      # and 0 is among the rest of every group
    x[:, :, :half] *= 2.0 ** p
    y = x.astype(np.float16)
    assert np.array_equal(y, x)
    return y


# {of the 30 large dims, of the fine value, of 15, of 8}: scores of -2^30 to 2^30, below, across and
# above 2^23, where the sums are exact and fine values differ by whole steps of fp32
EXACT_QUERIES = [(8, 1, 34944, 15), (8, 1, 35968, 0), (0, 1, 0, 0), (4, 1, 0, 0), (-8, 1, 0, 0), (1024, 64, 0, 0), (16, 1, 0, 0),
                 (0, 0.25, 2, 3), (32, 2, 0, 0), (-1024, 64, 0, 0), (-8, 1, -34944, -15), (8, 1, 34944, 14)]


def _exact_queries(c, n, share, first=0):
    x = np.zeros((n, c.heads * share, c.dim), np.float64)
    half = c.dim // 2
    for r in range(n * c.heads * share):
        base, fine, a, b = EXACT_QUERIES[(r + r // 12 + first) % 12]
        row = x.reshape(-1, c.dim)[r]
        row[:30] = base * (1 if c.bits == 4 else 16)
        row[half:half + 3] = fine, a, b
    y = x.astype(np.float16)
    assert np.array_equal(y, x)
    return y


def _check_exact(c, q, k, v, o, ls, before):
    """The ordinary tolerances without the scores' own error, which is none here: an exponential's
    argument is off by 4 e of the distance to the maximum (difference exact, factor and
    product rounded), and the exponential by 2^-21."""
    o, ls = to_np(o).astype(np.float64), to_np(ls).astype(np.float64)
    at = 0
    for b in range(len(q)):
        n, nq = q[b].shape[:2]
        share, ctx = nq // c.heads, int(c.ref.ctx[b])
        ro, rl, sums, _ = c.ref.attend(b, q[b], None if k is None else k[b], None if v is None else v[b])
        got = o[at:at + n].reshape(n, nq, c.dim)
        keys = sums.shape[1]
        ep = np.zeros((n, nq))
        for g in range(c.heads):
            kk = c.ref.values("k", b, g)
            if k is not None:
                kk = np.concatenate([kk, k[b][:, g].astype(np.float64)])
            for h in range(g * share, (g + 1) * share):
                for i in range(n):
                    s = kk[:ctx + (0 if k is None else i + 1)] @ q[b][i, h].astype(np.float64)
                    assert np.array_equal(s, s.astype(np.float32))
                    far = s.max(initial=-np.inf) - s
                    ep[i, h] = 8 * E * far[far < 100].max(initial=0) + 2.0 ** -21      # beyond: below every bound
        vmax = max([np.abs(c.ref.values("v", b, g)).max(initial=0) for g in range(c.heads)] +
                   ([] if v is None else [np.abs(v[b].astype(np.float64)).max(initial=0)]))
        tol = U * np.abs(ro) + (U + 2 * ep + keys * (E + 2.0 ** -25))[..., None] * vmax
        assert np.all(np.abs(got - ro) <= tol), (b, (np.abs(got - ro) - tol).max())
        some = np.isfinite(rl)
        assert np.array_equal(np.isfinite(ls[at:at + n]), some)
        bound = ep + keys * E + 2 * E * np.abs(np.where(some, rl, 0))
        assert np.all(np.abs(np.where(some, ls[at:at + n] - rl, 0)) <= bound), b
        if before is not None:
            grown = ctx + (0 if k is None else n)
            old, new = (c.slots(t, b, grown).astype(np.float64) for t in (before, c.cache.weight))
            old[:, ctx:] = 0
            bound = (2 * ep.max() + (keys + n * share + 4) * E) * sums + 2 * E * np.abs(old + sums) + 1e-30
            assert np.all(np.abs(new - old - sums) <= bound), (b, np.abs(new - old - sums).max())
        at += n


@pytest.mark.parametrize("dim,bits,group", [(64, 4, 32), (128, 4, 64), (64, 8, 32), (128, 8, 64)])
@pytest.mark.parametrize("share,n", [(1, [1, 1]), (4, [1, 1]), (1, [6, 2]), (2, [6, 1]), (1, [24, 3]), (1, [40, 30]), (3, [20, 9]),
                                     (1, [140, 70])])
@pytest.mark.parametrize("cross", [False, True])
def test_scores_around_two_to_the_23rd(dim, bits, group, share, n, cross):
    """Rows whose scores are below, across and above 2^23, up to 2^30 and of both signs, side by side
    in one tile, and in one row keys of which some score near 0: the maximum moves between
    the ranges, and every difference of a few units counts in full."""
    ctx = [300, 90]
    c = Case(44, ctx, heads=2, dim=dim, bits=bits, group=group, page=16, room=max(n))
    r = c.r

    def keys(m, start):
        at = np.arange(start, start + m)
        # 64 keys near 0, 64 far, then in runs of 5; fine values that rise, fall and scatter
        far = np.where(at < 128, at >= 64, at // 5 % 3 > 0)
        return _exact_rows(c, m, far, np.where(at % 7 < 3, at // 24 % 16, r.integers(0, 16, m)))
    for b, m in enumerate(ctx):
        ids = range(m)
        x = keys(m, 0)
        c.ref.ctx[b] = 0
        c.ref.store(b, x, c.rows(m))
        c.ref.ctx[b] = m
        for j in ids:
            p, s = c.ref.at(b, j)
            for name in "kv":
                getattr(c.cache, name + "_codes")[p, :, s] = torch.from_numpy(c.ref.codes[name][p, :, s]).cuda()
                getattr(c.cache, name + "_meta")[p, :, s] = torch.from_numpy(c.ref.meta[name][p, :, s]).cuda()
        assert all(np.array_equal(c.ref.values("k", b, g), x[:, g].astype(np.float64)) for g in range(2))
    q = [_exact_queries(c, m, share, first=i) for i, m in enumerate(n)]
    k, v = (None, None) if cross else ([keys(m, 40 + 9 * i) for i, m in enumerate(n)], [c.rows(m) for m in n])
    for acc in (False, True):
        c.cache.weight.zero_()
        before = c.cache.weight.clone() if acc else None
        o, ls = c.attend(q, k, v, accumulate=acc, check=False)
        _check_exact(c, q, k, v, o, ls, before)


@pytest.mark.parametrize("dim,bits", [(64, 4), (128, 8)])
@pytest.mark.parametrize("n", [[1, 1], [3, 2], [12, 5], [40, 33], [150, 40]])
def test_keys_of_minus_infinity_weigh_nothing(dim, bits, n):
    """A fresh key whose score is -infinity adds nothing; a row with no other key gets zeros and a
    log-sum-exp of -infinity, as one without any key."""
    c = Case(45, [0, 20], heads=2, dim=dim, bits=bits, room=max(n))
    q, k, v = [np.abs(x) for x in _scaled(c, n, 4)], [c.rows(m) for m in n], [c.rows(m) for m in n]
    for x in q:
        x[:] = np.maximum(x, np.float16(0.01))
    k[0][0, :, 3] = -np.inf                                  # the first sequence's first key
    k[1][-1, 1, 0] = -np.inf                                 # the other's last one, one key head
    c.cache.weight.zero_()
    o, ls = c.attend(q, k, v, accumulate=True, check=False)
    got, ls = to_np(o).astype(np.float64), to_np(ls).astype(np.float64)
    assert not got[0].any() and np.all(ls[0] == -np.inf)
    assert np.isfinite(got).all() and np.isfinite(ls[1:]).all()
    far = [x.copy() for x in k]
    far[0][0, :, 3], far[1][-1, 1, 0] = 0, 0
    for b, m in enumerate(n):
        first = n[0] * b
        for i in (range(1, m) if b == 0 else [m - 1]):
            hide = 0 if b == 0 else m - 1
            keep = [j for j in range(i + 1) if j != hide]
            for h in (range(4) if b == 0 else (2, 3)):
                g = h // 2
                kk = np.concatenate([c.ref.values("k", b, g), far[b][keep, g].astype(np.float64)])
                vv = np.concatenate([c.ref.values("v", b, g), v[b][keep, g].astype(np.float64)])
                qi = q[b][i, h].astype(np.float64)
                s = kk @ qi
                p = np.exp(s - s.max())
                want = p @ vv / p.sum()
                size = (np.abs(kk) @ qi).max()
                ep = 2 * (dim + 4) * E * size + 2.0 ** -21
                tol = U * np.abs(want) + (U + 2 * ep + len(kk) * (E + 2.0 ** -25)) * np.abs(vv).max()
                assert np.all(np.abs(got[first + i, h * dim:(h + 1) * dim] - want) <= tol), (b, i, h)
                assert abs(ls[first + i, h] - s.max() - np.log(p.sum())) <= ep + len(kk) * E + 2 * E * abs(s.max())
    w = c.slots(c.cache.weight, 0, n[0])
    assert np.isfinite(w).all() and not w[:, 0].any()


@pytest.mark.parametrize("dim,bits", [(64, 4), (128, 4), (64, 8), (128, 8)])
@pytest.mark.parametrize("ctx,n", [([30, 0], [1, 2]), ([30, 0], [4, 3]), ([30, 0], [12, 9]), ([30, 0], [40, 20]), ([30, 0], [150, 40]),
                                   ([5000, 700], [1, 2]), ([5000, 700], [12, 3]), ([5000, 700], [60, 3]), ([9000, 700], [150, 3])])
def test_infinite_values_of_any_weight(dim, bits, ctx, n):
    """An infinite fresh value makes its dim infinite in every row that sees it, however small its
    weight (it underflows fp16 and, where the parts of a long history are joined, fp32), in every
    kernel alike; the other dims have the bits that a value of 0 gives."""
    c = Case(46, ctx, heads=1, dim=dim, bits=bits, page=64, room=max(n))
    q, k, v = [np.abs(x) for x in _scaled(c, n, 2)], [c.rows(m) for m in n], [c.rows(m) for m in n]
    at = [n[0] // 2, 0]
    zero = [x.copy() for x in v]
    for b, j in enumerate(at):
        k[b][j] = -300 if ctx[b] < 1000 else -3000           # about 50 dims' worth below the other scores
        q[b][:] = np.maximum(q[b], np.float16(0.05))
        v[b][j, 0, 5], v[b][j, 0, dim - 1] = np.inf, -np.inf
        zero[b][j, 0, 5] = zero[b][j, 0, dim - 1] = 0
    want, wl = c.attend(q, k, zero)
    o, ls = c.attend(q, k, v, check=False)
    assert torch.equal(ls, wl)
    got, want = (to_np(x).reshape(-1, 2, dim) for x in (o, want))
    seen = np.zeros(len(got), bool)
    seen[at[0]:n[0]] = seen[n[0] + at[1]:n[0] + n[1]] = True
    rest = [d for d in range(dim) if d not in (5, dim - 1)]
    assert np.array_equal(got[..., rest].view(np.uint16), want[..., rest].view(np.uint16))
    assert np.array_equal(got[~seen].view(np.uint16), want[~seen].view(np.uint16))
    if ctx[1] == 0:                                          # its first row sees nothing else
        seen[n[0]] = False
    assert np.all(got[seen][..., 5] == np.inf) and np.all(got[seen][..., dim - 1] == -np.inf)


@pytest.mark.parametrize("n", [1, 3, 12, 60, 150])
def test_infinite_values_in_a_part_of_no_weight(n):
    """The last part of a long history, the fresh keys' own, has scores some hundreds below the first
    part's: joined, its factor underflows."""
    c = Case(47, [0], heads=1, dim=64, page=64, room=6000 + n)
    low = np.abs(c.rows(6000)) + np.float16(1)
    low[3000:] *= -20
    low[:3000] *= 20
    c.store([low], [c.rows(6000)], advance=True)
    q, k, v = [np.abs(_scaled(c, [n], 1)[0]) + np.float16(0.1)], [-20 * (np.abs(c.rows(n)) + np.float16(1))], [c.rows(n)]
    want, wl = c.attend(q, k, v)
    v[0][0, 0, 5], v[0][0, 0, 40] = np.inf, np.nan
    o, ls = c.attend(q, k, v, check=False)
    assert torch.equal(ls, wl)
    rest = [d for d in range(64) if d not in (5, 40)]
    assert torch.equal(o[:n, rest], want[:n, rest])
    assert bool((o[:n, 5] == float("inf")).all()) and bool(o[:n, 40].isnan().all())


@pytest.mark.parametrize("bad", [-1, -(1 << 31), 1 << 20, (1 << 31) - 1, "one too many"])
@pytest.mark.parametrize("n", [[1, 1, 1], [3, 40, 2]])
@pytest.mark.parametrize("wide", [False, True])
def test_a_sequence_of_impossible_length_keeps_its_cache(bad, n, wide):
    """A ctx_len outside the table is reported and nothing of its sequence changes: no slot, position
    or weight, in the store, the running weights and the eviction (of both kinds of table);
    its new length stays what it was, so that it is reported again. The others are right."""
    c = Case(48, [40, 90, 25], heads=2, dim=64, page=64, room=2300 if wide else 45)
    cap = c.cache.page_table.shape[1] * c.page
    c.cache.weight.copy_(torch.from_numpy(np.abs(c.r.standard_normal(tuple(c.cache.weight.shape))).astype(np.float32)))
    c.ref.weight = to_np(c.cache.weight).astype(np.float64)
    q, k, v = _scaled(c, n, 4), [c.rows(m) for m in n], [c.rows(m) for m in n]
    qd, cu, total, most = c.ragged(q)
    kd, vd = c.ragged(k)[0], c.ragged(v)[0]
    o = torch.empty((total, 4 * c.dim), dtype=torch.float16, device="cuda")
    ws = torch.empty(fq.flex_paged_attention_ws_bytes(c.cache, 4, total, most, True), dtype=torch.uint8, device="cuda")
    pools = lambda: [getattr(c.cache, x) for x in ("k_codes", "k_meta", "v_codes", "v_meta", "weight", "slot_pos")]
    mine = torch.as_tensor([x for x in to_np(c.cache.page_table[1]) if x >= 0], dtype=torch.int64, device="cuda")
    before = [x[mine].clone() for x in pools()]

    def same():
        return all(torch.equal(x[mine].view(torch.uint8), y.view(torch.uint8)) for x, y in zip(pools(), before))
    value = cap + 1 if bad == "one too many" else bad
    c.ctx[1] = value
    fq.flex_paged_attention(c.cache, qd, qd.stride(0), 4, kd, vd, kd.stride(0), o, None, cu, most, ws, total=total, accumulate=True)
    assert _status() == fq.FLEX_ERR_INVALID_ARG and same()
    fq.flex_paged_store_kv(c.cache, kd, vd, kd.stride(0), cu, most, total=total)
    assert _status() == fq.FLEX_ERR_INVALID_ARG and same()
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    ew = torch.empty(fq.flex_paged_evict_ws_bytes(c.cache, 20), dtype=torch.uint8, device="cuda")
    fq.flex_paged_evict(c.cache, 20, 5, new, ew)
    assert _status() == fq.FLEX_ERR_INVALID_ARG and same()
    assert new.tolist() == [20, value, 20]


@pytest.mark.parametrize("bits,group", [(4, 32), (8, 64)])
@pytest.mark.parametrize("n", [1, 5, 9, 40])
def test_steps_of_every_scale(bits, group, n):
    """The step that attention takes for a scale is the correctly rounded fp16(1 / scale), for every
    positive fp16 scale whose reciprocal is finite there: one slot a head, code 1, minimum 0, so
    that the output is the step itself; 1, 5 and 9 rows of the rows kernel, 40 of the tiles."""
    scales = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16)
    with np.errstate(over="ignore"):
        want = (1.0 / scales.astype(np.float64)).astype(np.float16)
    scales, want = scales[np.isfinite(want)], want[np.isfinite(want)]
    assert scales[0] < 1.6e-5 and scales[-1] == 65504 and len(scales) > 30000
    heads, dim = 64, 64
    pages = -(-len(scales) // heads)
    table, ctx = torch.arange(pages, dtype=torch.int32, device="cuda").view(-1, 1), torch.ones(pages, dtype=torch.int32, device="cuda")
    cache = fq.FlexPagedCache(table, ctx, pages, 16, heads, dim, bits, group)
    padded = np.resize(scales, (pages, heads))
    for codes, meta in ((cache.k_codes, cache.k_meta), (cache.v_codes, cache.v_meta)):
        codes.fill_(0x11 if bits == 4 else 1)
        meta[:, :, 0, :, 1] = torch.from_numpy(padded).cuda()[:, :, None]
    # keys: the same values; a query of zeros, so that only the value's step is in the output
    total = pages * n
    q = torch.zeros((total, heads * dim), dtype=torch.float16, device="cuda")
    o = torch.empty_like(q)
    ws = torch.empty(fq.flex_paged_attention_ws_bytes(cache, heads, total, n), dtype=torch.uint8, device="cuda")
    fq.flex_paged_attention(cache, q, heads * dim, heads, None, None, 0, o, None, None, n, ws)
    sync_status()
    got = to_np(o).reshape(pages, n, heads, dim).transpose(0, 2, 1, 3).reshape(pages * heads, n, dim)[:len(scales)]
    assert np.array_equal(got.view(np.uint16), np.broadcast_to(want[:, None, None], got.shape).view(np.uint16))
    # and the keys': a query of one 1 in a dim, against the log-sum-exp of the one score
    q.view(total, heads, dim)[:, :, 17] = 1
    ls = torch.empty((total, heads), device="cuda")
    fq.flex_paged_attention(cache, q, heads * dim, heads, None, None, 0, o, ls, None, n, ws)
    sync_status()
    got = to_np(ls).reshape(pages, n, heads).transpose(0, 2, 1).reshape(pages * heads, n)[:len(scales)]
    assert np.all(np.abs(got - want.astype(np.float64)[:, None]) <= 2 * E * want.astype(np.float64)[:, None] + 2.0 ** -21)


@pytest.mark.parametrize("per", [2, 20])
def test_moves_and_weights_behind_32_bit_offsets(per):
    """The last pages of a pool of 5.4 GB: accumulated weights, and what eviction moves (codes,
    metadata, weights, positions) in tables of up to 2048 slots and of more."""
    pages, heads, page, dim = 1 << 13, 40, 128, 128
    ids = pages - 1 - np.random.default_rng(23).permutation(per)
    table = torch.from_numpy(ids.astype(np.int32)).cuda().view(1, per)
    held = per * page - 9
    ctx = torch.tensor([held], dtype=torch.int32, device="cuda")
    shape = (pages, heads, page)
    pools = tuple(torch.empty(shape + s, dtype=t, device="cuda") for s, t in
                  (((dim,), torch.uint8), ((2, 2), torch.float16)) * 2)
    cache = fq.FlexPagedCache(table, ctx, pools=pools, weight=True, slot_pos=True, num_bits=8, group_size=64)
    r = np.random.default_rng(24)
    ref = PagedCache([np.arange(per)], [held], per, page, 1, dim, 8, 64)
    used = torch.from_numpy(ids.copy()).cuda()
    for codes, meta in ((pools[0], pools[1]), (pools[2], pools[3])):
        codes[used] = torch.from_numpy(r.integers(0, 256, (per, heads, page, dim), dtype=np.uint8)).cuda()
        m = np.stack([r.standard_normal((per, heads, page, 2)) - 1, 60 + 50 * r.random((per, heads, page, 2))], -1)
        meta[used] = torch.from_numpy(m.astype(np.float16)).cuda()
    cache.weight[used] = torch.from_numpy(r.random((per, heads, page), dtype=np.float32)).cuda()
    pos = r.permutation(per * page * heads).astype(np.int32).reshape(per, heads, page)
    cache.slot_pos[used] = torch.from_numpy(pos).cuda()
    for n in (1, 3, 33):
        q = (r.standard_normal((n, heads, dim)) * 0.09).astype(np.float16)
        o = torch.empty((n, heads * dim), dtype=torch.float16, device="cuda")
        ws = torch.empty(fq.flex_paged_attention_ws_bytes(cache, heads, n, n, True), dtype=torch.uint8, device="cuda")
        old = to_np(cache.weight[used]).astype(np.float64)
        fq.flex_paged_attention(cache, torch.from_numpy(q).cuda().view(n, -1), heads * dim, heads, None, None, 0, o, None,
                                None, n, ws, accumulate=True)
        sync_status()
        new = to_np(cache.weight[used]).astype(np.float64)
        for h in (0, heads - 1):
            for name, codes, meta in (("k", pools[0], pools[1]), ("v", pools[2], pools[3])):
                ref.codes[name][:, 0], ref.meta[name][:, 0] = to_np(codes[used, h]), to_np(meta[used, h])
            ro, _, sums, size = ref.attend(0, q[:, h:h + 1])
            ep = 2 * (dim + 4) * E * size.max() + 2.0 ** -21
            vmax = np.abs(ref.values("v", 0, 0)).max()
            got = to_np(o).reshape(n, heads, dim)[:, h].astype(np.float64)
            assert np.all(np.abs(got - ro[:, 0]) <= U * np.abs(ro[:, 0]) + (U + 2 * ep + held * (E + 2.0 ** -25)) * vmax)
            was, now = (x[:, h].reshape(-1)[:held] for x in (old, new))
            bound = (2 * ep + (held + n + 4) * E) * sums[0] + 2 * E * np.abs(was + sums[0]) + 1e-30
            assert np.all(np.abs(now - was - sums[0]) <= bound), (n, h)
    budget, recent = per * page // 3, 17
    before = [to_np(x[used]) for x in (*pools, cache.weight, cache.slot_pos)]
    new_len = torch.zeros(1, dtype=torch.int32, device="cuda")
    ew = torch.empty(fq.flex_paged_evict_ws_bytes(cache, budget), dtype=torch.uint8, device="cuda")
    fq.flex_paged_evict(cache, budget, recent, new_len, ew)
    sync_status()
    assert new_len.tolist() == [budget]
    after = [to_np(x[used]) for x in (*pools, cache.weight, cache.slot_pos)]
    for h in range(heads):
        w, p = (x[:, h].reshape(-1)[:held] for x in before[4:])
        first = p > p.max() - recent
        order = np.lexsort((np.arange(held), -np.where(first, 0, w), ~first))
        kept = np.zeros(held, bool)
        kept[order[:budget]] = True
        src = np.arange(per * page)
        src[:budget][~kept[:budget]] = np.nonzero(kept)[0][kept[:budget].sum():]
        for x, y in zip(before, after):
            x, y = (t[:, h].reshape((per * page,) + t.shape[3:]) for t in (x, y))
            assert np.array_equal(y.view(np.uint8), x[src].view(np.uint8)), h


def test_replays_leave_the_same_cache_as_calls():
    """A captured attention, store and eviction, replayed with other lengths and offsets: outputs,
    slots, positions and weights have the bits that the same calls leave without a capture."""
    c = Case(49, [700, 30, 0], heads=2, dim=64, room=64)
    n0 = [1, 40, 9]
    q, k, v = _scaled(c, n0, 4), [c.rows(m) for m in n0], [c.rows(m) for m in n0]
    qd, cu, total, most = c.ragged(q)
    kd, vd = c.ragged(k)[0], c.ragged(v)[0]
    o = torch.empty((total, 4 * c.dim), dtype=torch.float16, device="cuda")
    ls = torch.empty((total, 4), device="cuda")
    ws = torch.empty(fq.flex_paged_attention_ws_bytes(c.cache, 4, total, most, True), dtype=torch.uint8, device="cuda")
    ew = torch.empty(fq.flex_paged_evict_ws_bytes(c.cache, 25), dtype=torch.uint8, device="cuda")
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    state = [getattr(c.cache, x) for x in ("k_codes", "k_meta", "v_codes", "v_meta", "slot_pos", "weight")] + [o, ls, new]
    start = [x.clone() for x in state]

    def step():
        fq.flex_paged_attention(c.cache, qd, qd.stride(0), 4, kd, vd, kd.stride(0), o, ls, cu, most, ws, accumulate=True,
                                total=total)
        fq.flex_paged_store_kv(c.cache, kd, vd, kd.stride(0), cu, most, total=total)
        fq.flex_paged_evict(c.cache, 25, 5, new, ew)

    def restore(n, ctx):
        for x, y in zip(state, start):
            x.copy_(y)
        cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32))
        c.set_ctx(ctx)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n, ctx in ((n0, [700, 30, 0]), ([40, 1, 9], [650, 30, 0]), ([0, 0, 38], [700, 30, 26]), ([1, 1, 1], [0, 25, 26])):
        restore(n, ctx)
        step()
        sync_status()
        want = [x.clone() for x in state]
        assert not torch.equal(want[5], start[5]) and want[8].tolist() == [min(x, 25) for x in ctx]
        restore(n, ctx)
        graph.replay()
        sync_status()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(state, want)), (n, ctx)


@pytest.mark.parametrize("share", [1, 5, 100])
def test_a_bound_far_above_the_rows(share):
    """`most` is a bound only: 2^24 with a few rows in the sequences, in every call."""
    most = 1 << 24
    c = Case(50, [300, 0, 65], heads=2, dim=64, page=64, room=5)
    n = [3, 5, 0]
    q, k, v = _scaled(c, n, 2 * share), [c.rows(m) for m in n], [c.rows(m) for m in n]
    qd, cu, total, _ = c.ragged(q)
    kd, vd = c.ragged(k)[0], c.ragged(v)[0]
    o = torch.full((total + TAIL, 2 * share * c.dim), 3.25, dtype=torch.float16, device="cuda")
    ls = torch.empty((total, 2 * share), device="cuda")
    ws = torch.empty(fq.flex_paged_attention_ws_bytes(c.cache, 2 * share, total, most, True), dtype=torch.uint8, device="cuda")
    before = c.cache.weight.clone()
    fq.flex_paged_attention(c.cache, qd, qd.stride(0), 2 * share, kd, vd, kd.stride(0), o, ls, cu, most, ws, accumulate=True, total=total)
    sync_status()
    c.check_attention(q, k, v, o[:total], ls, before)
    assert bool((o[total:] == 3.25).all())
    fq.flex_paged_store_kv(c.cache, kd, vd, kd.stride(0), cu, most, total=total)
    for b in range(3):
        c.ref.store(b, k[b], v[b])
    c.set_ctx([303, 5, 65])
    sync_status()
    c.check_slots("added")
    outs = [torch.full((total + TAIL, 2 * c.dim), 5.0, dtype=torch.float16, device="cuda") for _ in "kv"]
    fq.flex_paged_load_kv(c.cache, *outs, 2 * c.dim, cu, most, total=total, start=torch.tensor([300, 0, 65], dtype=torch.int32, device="cuda"))
    sync_status()
    for x, i in zip(outs, (0, 1)):
        ref = np.concatenate([c.ref.load(0, 300, 3)[i], c.ref.load(1, 0, 5)[i]]).reshape(total, -1)
        assert np.array_equal(to_np(x[:total]).view(np.uint16), ref.view(np.uint16)) and bool((x[total:] == 5).all())


FIRST_CALLS = r"""
import threading
import torch
import group_wise_int4_b200 as fq
calls = []
for most in (1, 40, 200):
    for _ in range(8):
        table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
        cache = fq.FlexPagedCache(table, torch.full((2,), 20, dtype=torch.int32, device="cuda"), 8, 64, 2, 64)
        x = torch.zeros((2 * most, 3 * 128), dtype=torch.float16, device="cuda")
        o = torch.empty((2 * most, 128), dtype=torch.float16, device="cuda")
        ws = torch.empty(fq.flex_paged_attention_ws_bytes(cache, 2, 2 * most, most), dtype=torch.uint8, device="cuda")
        calls.append((cache, x, o, ws, most, torch.cuda.Stream()))
torch.cuda.synchronize()
start, wrong = threading.Barrier(len(calls)), []
def run(cache, x, o, ws, most, stream):
    start.wait()
    try:
        fq.flex_paged_attention(cache, x, 384, 2, x[:, 128:], x[:, 256:], 384, o, None, None, most, ws, stream=stream)
    except Exception as e:
        wrong.append(repr(e))
threads = [threading.Thread(target=run, args=c) for c in calls]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not wrong, wrong
assert fq.flex_get_status() == fq.FLEX_OK
print("fine")
"""


def test_first_calls_of_several_threads():
    """A kernel's first launch sets its shared memory; another thread's must not come between."""
    for _ in range(3):
        p = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=240)
        assert p.returncode == 0 and "fine" in p.stdout, p.stdout + p.stderr
