"""Pins of the paged-cache oracle: against the contiguous cache's oracle, closed forms,
and its own invariants."""
import numpy as np

from oracle import layer as ol
from oracle.paged import PagedCache


def _rows(r, n, heads, dim):
    return r.standard_normal((n, heads, dim)).astype(np.float16)


def _cache(r, ctx, heads=2, dim=64, bits=4, group=32, page=16, room=16):
    per = -(-(max(ctx) + room) // page)
    table = r.permutation(per * len(ctx)).reshape(len(ctx), per)
    c = PagedCache(table, [0] * len(ctx), per * len(ctx), page, heads, dim, bits, group)
    hist = []
    for b, n in enumerate(ctx):
        hist.append((_rows(r, n, heads, dim), _rows(r, n, heads, dim)))
        c.store(b, *hist[-1])
        c.ctx[b] = n
    return c, hist


def test_slots_hold_what_the_contiguous_cache_holds():
    r = np.random.default_rng(1)
    for bits in (4, 8):
        c, hist = _cache(r, [21, 5], bits=bits)
        for b, (k, v) in enumerate(hist):
            ref = ol.KVCache(1, 2, len(k), 64, bits, 32)
            ref.store(k.transpose(1, 0, 2)[None], v.transpose(1, 0, 2)[None], 0)
            want = ref.load(len(k))
            got = c.load(b, 0, len(k))
            for x, y in zip(got, want):
                assert np.array_equal(x.astype(np.float64).transpose(1, 0, 2)[None], y)
            assert [int(c.pos[c.at(b, j)[0], 0, c.at(b, j)[1]]) for j in range(len(k))] == list(range(len(k)))


def test_attention_values_are_within_an_fp16_step_of_the_codec():
    """|fp16(c s16 + m) - fp16(c s + m)|: half a step of each rounding and c times the step's own."""
    r = np.random.default_rng(2)
    c, _ = _cache(r, [40])
    k, _ = c.load(0, 0, 40)
    v = c.values("k", 0, 1)
    bound = 2.0 ** -11 * (2 * np.abs(v) + 2 * np.abs(k[:, 1].astype(np.float64)) + 8) + 1e-12
    assert np.all(np.abs(v - k[:, 1].astype(np.float64)) <= bound)


def test_one_token_is_the_decode_attention():
    """With one new token and the same values it is the contiguous cache's decode step."""
    r = np.random.default_rng(3)
    c, hist = _cache(r, [33], heads=3)
    q, k, v = _rows(r, 1, 3, 64) * np.float16(0.125), _rows(r, 1, 3, 64), _rows(r, 1, 3, 64)
    ref = ol.KVCache(1, 3, 34, 64, 4, 32)
    ref.store(hist[0][0].transpose(1, 0, 2)[None], hist[0][1].transpose(1, 0, 2)[None], 0)
    want = ol.decode_attention(q, k, v, ref, 33)
    o, _, sums, _ = c.attend(0, q, k, v)
    assert np.max(np.abs(o.reshape(-1) - np.asarray(want).reshape(-1))) < 4e-3       # fp16 values of either form
    assert np.allclose(sums.sum(1), 1.0)


def test_chunks_and_shared_heads():
    r = np.random.default_rng(4)
    c, _ = _cache(r, [17])
    q, k, v = _rows(r, 6, 8, 64), _rows(r, 6, 2, 64), _rows(r, 6, 2, 64)
    o, lse, sums, _ = c.attend(0, q, k, v)
    # equal keys: the plain mean of what is seen
    o2, lse2, _, _ = c.attend(0, np.zeros_like(q), k, v)
    vals = np.concatenate([c.values("v", 0, 1), v[:3, 1].astype(np.float64)])
    assert np.allclose(o2[2, 5], vals.mean(0)) and np.allclose(lse2[2, 5], np.log(20))
    # a head of a shared group alone is the same head
    o3, _, _, _ = c.attend(0, q[:, [1, 6]], k, v)
    assert np.allclose(o3[:, 0], o[:, 1]) and np.allclose(o3[:, 1], o[:, 6])
    assert np.allclose(sums.sum(1), 6 * 4)
    # a later token does not change an earlier one
    k[4:], v[4:] = 9, 9
    assert np.allclose(c.attend(0, q, k, v)[0][:4], o[:4])


def test_cross_attention_without_states():
    r = np.random.default_rng(5)
    c, _ = _cache(r, [0, 9])
    o, lse, sums, _ = c.attend(0, _rows(r, 3, 2, 64))
    assert not o.any() and np.all(lse == -np.inf) and sums.shape == (2, 0)
    o, lse, sums, _ = c.attend(1, _rows(r, 3, 2, 64))
    assert np.all(np.isfinite(lse)) and np.allclose(sums.sum(1), 3)


def test_eviction_by_hand():
    c = PagedCache([[1, 0]], [20], 2, 16, 1, 64, 4, 64)
    for j in range(20):
        p, s = c.at(0, j)
        c.weight[p, 0, s], c.pos[p, 0, s], c.codes["k"][p, 0, s] = [5, 1, 7, 7][j % 4] + 0.0, j, j
    c.weight[1, 0, 3] = np.nan
    n = c.evict(8, 3)
    # recent: 17, 18, 19; then weight 7 in slot order: 2, 6, 7, 10, 11 (3 holds a NaN)
    # kept below the budget: 2, 6, 7; the others fill 0, 1, 3, 4, 5 in order
    want = [10, 11, 2, 17, 18, 19, 6, 7]
    assert list(n) == [8]
    assert [int(c.pos[1, 0, s]) for s in range(8)] == want
    assert [int(c.codes["k"][1, 0, s, 0]) for s in range(8)] == want
    assert int(c.pos[1, 0, 8]) == 8                       # behind the budget nothing changes


def test_eviction_keeps_short_sequences():
    r = np.random.default_rng(6)
    c, _ = _cache(r, [8, 3])
    before = c.codes["k"].copy(), c.pos.copy()
    assert list(c.evict(8, 8)) == [8, 3]
    assert np.array_equal(before[0], c.codes["k"]) and np.array_equal(before[1], c.pos)
