"""Host-side checks of the paged cache's C entry points and of its binding: every refusal
returns before any CUDA call, so they run without a GPU."""
import ctypes

import pytest
import torch

import group_wise_int4_b200 as fq

P = ctypes.c_void_p


def _cache(**kw):
    c = fq.flex_paged_cache(k_codes=1 << 20, k_meta=2 << 20, v_codes=3 << 20, v_meta=4 << 20, weight=5 << 20,
                            slot_pos=6 << 20, page_table=7 << 20, ctx_len=8 << 20, num_pages=8, page_size=16,
                            max_pages=4, batch=2, n_kv_heads=2, head_dim=64, cfg=fq.config(4, 64, 3))
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    (dict(k_codes=None), fq.FLEX_ERR_INVALID_ARG), (dict(v_meta=None), fq.FLEX_ERR_INVALID_ARG),
    (dict(page_table=None), fq.FLEX_ERR_INVALID_ARG), (dict(ctx_len=None), fq.FLEX_ERR_INVALID_ARG),
    (dict(num_pages=0), fq.FLEX_ERR_INVALID_ARG), (dict(max_pages=-1), fq.FLEX_ERR_INVALID_ARG),
    (dict(batch=0), fq.FLEX_ERR_INVALID_ARG), (dict(n_kv_heads=0), fq.FLEX_ERR_INVALID_ARG),
    (dict(head_dim=96), fq.FLEX_ERR_UNSUPPORTED), (dict(page_size=24), fq.FLEX_ERR_UNSUPPORTED),
    (dict(page_size=8), fq.FLEX_ERR_UNSUPPORTED), (dict(page_size=2048), fq.FLEX_ERR_UNSUPPORTED),
    (dict(cfg=fq.config(4, 64, 3, 1)), fq.FLEX_ERR_UNSUPPORTED), (dict(cfg=fq.config(3, 64, 3)), fq.FLEX_ERR_UNSUPPORTED),
    (dict(cfg=fq.config(4, 128, 3)), fq.FLEX_ERR_UNSUPPORTED), (dict(cfg=fq.config(4, 64, 1)), fq.FLEX_ERR_UNSUPPORTED),
    (dict(batch=70000), fq.FLEX_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 27, page_size=16), fq.FLEX_ERR_SHAPE),
    (dict(num_pages=1 << 27, n_kv_heads=2), fq.FLEX_ERR_SHAPE),
    (dict(k_codes=(1 << 20) + 8), fq.FLEX_ERR_ALIGN), (dict(weight=(5 << 20) + 4), fq.FLEX_ERR_ALIGN),
    (dict(page_table=(7 << 20) + 2), fq.FLEX_ERR_ALIGN),
]


def _calls(c):
    """Every entry point with arguments that are right but for the cache."""
    L, r = fq.lib(), ctypes.byref(c)
    return [
        L.flex_paged_store_kv(r, P(4096), P(8192), 128, None, 2, 6, 3, None, None),
        L.flex_paged_load_kv(r, P(4096), P(8192), 128, None, 2, 6, 3, None, None),
        L.flex_paged_attention_ws_bytes(r, 2, 2, 6, 3, 0),
        L.flex_paged_attention(r, P(4096), 128, 2, P(8192), P(12288), 128, P(16384), None, None, 2, 6, 3, 0, P(1 << 30),
                               1 << 30, None),
        L.flex_paged_evict_ws_bytes(r, 8),
        L.flex_paged_evict(r, 8, 4, P(4096), P(1 << 30), 1 << 30, None),
    ]


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_caches_refused_by_every_call(change, want):
    assert _calls(_cache(**change)) == [want] * 6


def test_null_cache():
    L = fq.lib()
    assert L.flex_paged_store_kv(None, P(4096), P(8192), 128, None, 2, 6, 3, None, None) == fq.FLEX_ERR_INVALID_ARG
    assert L.flex_paged_evict_ws_bytes(None, 8) == fq.FLEX_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["flex_paged_store_kv", "flex_paged_load_kv"])
def test_store_and_load_arguments(name):
    f, r = getattr(fq.lib(), name), ctypes.byref(_cache())
    assert f(r, None, P(8192), 128, None, 2, 6, 3, None, None) == fq.FLEX_ERR_INVALID_ARG
    assert f(r, P(4096), P(8192), 120, None, 2, 6, 3, None, None) == fq.FLEX_ERR_INVALID_ARG     # rows overlap
    assert f(r, P(4096), P(8192), 132, None, 2, 6, 3, None, None) == fq.FLEX_ERR_ALIGN
    assert f(r, P(4100), P(8192), 128, None, 2, 6, 3, None, None) == fq.FLEX_ERR_ALIGN
    assert f(r, P(4096), P(8192), 128, None, 2, 7, 3, None, None) == fq.FLEX_ERR_INVALID_ARG     # total != batch * most
    assert f(r, P(4096), P(8192), 128, None, 3, 9, 3, None, None) == fq.FLEX_ERR_INVALID_ARG     # more than the table has
    assert f(r, P(4096), P(8192), 128, P(16384), 2, -1, 3, None, None) == fq.FLEX_ERR_INVALID_ARG
    assert f(r, P(4096), P(8192), 128, P(16386), 2, 6, 3, None, None) == fq.FLEX_ERR_ALIGN
    assert f(r, P(4096), P(8192), 128, None, 2, 6, 3, P(2), None) == fq.FLEX_ERR_ALIGN
    assert f(r, P(4096), P(8192), 128, P(16384), 2, 1 << 30, 1 << 25, None, None) == fq.FLEX_ERR_UNSUPPORTED


def test_attention_arguments():
    L, r = fq.lib(), ctypes.byref(_cache())

    def call(cache=r, q=4096, qs=256, heads=4, k=8192, v=12288, ks=128, o=16384, lse=None, cu=None, batch=2, total=6,
             most=3, acc=0, ws=1 << 30, size=1 << 30):
        return L.flex_paged_attention(cache, P(q), qs, heads, P(k), P(v), ks, P(o), P(lse), P(cu), batch, total, most, acc,
                                      P(ws), size, None)
    inv, al = fq.FLEX_ERR_INVALID_ARG, fq.FLEX_ERR_ALIGN
    assert call(q=None) == inv and call(o=None) == inv and call(k=None) == inv and call(v=None) == inv
    assert call(heads=3) == inv and call(heads=0) == inv and call(heads=65538) == fq.FLEX_ERR_UNSUPPORTED
    assert call(qs=248) == inv and call(ks=120) == inv and call(total=5) == inv and call(batch=3, total=9) == inv
    assert call(qs=260) == al and call(ks=132) == al and call(q=4104) == al and call(o=16392) == al and call(k=8200) == al
    assert call(lse=16386) == al and call(cu=16386) == al and call(ws=(1 << 30) + 8) == al
    need = L.flex_paged_attention_ws_bytes(r, 4, 2, 6, 3, 0)
    assert need > 0 and call(size=need - 1) == fq.FLEX_ERR_WORKSPACE and call(ws=None) == fq.FLEX_ERR_WORKSPACE
    no_weight = ctypes.byref(_cache(weight=None))
    assert call(no_weight, acc=1) == inv
    assert L.flex_paged_attention_ws_bytes(no_weight, 4, 2, 6, 3, 1) == inv
    assert L.flex_paged_attention_ws_bytes(r, 4, 2, 6, 3, 1) >= need
    # nothing to do needs no device
    assert call(total=0, most=0) == fq.FLEX_OK


def test_evict_arguments():
    L, r = fq.lib(), ctypes.byref(_cache())

    def call(cache=r, budget=8, recent=4, out=4096, ws=1 << 30, size=1 << 30):
        return L.flex_paged_evict(cache, budget, recent, P(out), P(ws), size, None)
    inv = fq.FLEX_ERR_INVALID_ARG
    assert call(budget=0) == inv and call(recent=9) == inv and call(recent=-1) == inv and call(out=None) == inv
    assert call(out=8 << 20) == inv and call(out=(8 << 20) + 4) == inv           # over ctx_len
    assert call(ctypes.byref(_cache(weight=None))) == inv and call(ctypes.byref(_cache(slot_pos=None))) == inv
    assert call(out=4098) == fq.FLEX_ERR_ALIGN and call(ws=(1 << 30) + 8) == fq.FLEX_ERR_ALIGN
    need = L.flex_paged_evict_ws_bytes(r, 8)
    assert need > 0 and call(size=need - 1) == fq.FLEX_ERR_WORKSPACE and call(ws=None) == fq.FLEX_ERR_WORKSPACE
    assert L.flex_paged_evict_ws_bytes(r, 0) == inv


def test_struct_layout():
    assert int(fq.lib().flex_abi_layout(4, -1)) == ctypes.sizeof(fq.flex_paged_cache)


# ---- the binding ----------------------------------------------------------------------
def _py_cache(**kw):
    table, ctx = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    a = dict(num_pages=8, page_size=16, n_kv_heads=2, head_dim=64)
    a.update(kw)
    return fq.FlexPagedCache(table, ctx, **a)


def test_binding_checks_the_cache():
    c = _py_cache(weight=True, slot_pos=True)
    assert (c.num_pages, c.n_kv_heads, c.page_size, c.head_dim, c.batch, c.max_pages) == (8, 2, 16, 64, 2, 4)
    first = c.struct().weight
    c.weight = torch.zeros_like(c.weight)
    assert c.struct().weight == c.weight.data_ptr() != first            # another tensor: another struct
    c.ctx_len = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="ctx_len"):
        c.struct()
    with pytest.raises(ValueError, match="page_table"):
        fq.FlexPagedCache(torch.zeros((2, 4)), torch.zeros(2, dtype=torch.int32), 8, 16, 2, 64)
    with pytest.raises(ValueError, match="weight"):
        _py_cache(weight=torch.zeros(8, 2, 8))


def test_binding_checks_rows():
    c = _py_cache(weight=True, slot_pos=True)
    x = torch.zeros((6, 128), dtype=torch.float16)
    cu = torch.zeros(3, dtype=torch.int32)
    ws = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_new"):
        fq.flex_paged_store_kv(c, x[:5], x, 128, None, 4)
    with pytest.raises(ValueError, match="v_new"):
        fq.flex_paged_store_kv(c, x, x.float(), 128, None, 3)
    with pytest.raises(ValueError, match="total"):
        fq.flex_paged_store_kv(c, x, x, 128, cu, 3)
    with pytest.raises(ValueError, match="cu"):
        fq.flex_paged_store_kv(c, x, x, 128, cu[:2], 3, total=6, batch=2)
    with pytest.raises(ValueError, match="pos0"):
        fq.flex_paged_store_kv(c, x, x, 128, cu, 3, total=6, pos0=cu[:1])
    with pytest.raises(ValueError, match="k_out"):
        fq.flex_paged_load_kv(c, x, x, 128, cu, 3, total=7)
    with pytest.raises(ValueError, match="q:"):
        fq.flex_paged_attention(c, x, 128, 4, x, x, 128, x, None, cu, 3, ws, total=6)
    with pytest.raises(ValueError, match="lse"):
        fq.flex_paged_attention(c, x, 128, 2, x, x, 128, x, torch.zeros((5, 2)), cu, 3, ws, total=6)
    with pytest.raises(ValueError, match="new_len"):
        fq.flex_paged_evict(c, 8, 4, torch.zeros(1, dtype=torch.int32), ws)


def test_binding_refuses_outputs_with_a_stride_of_their_own():
    """o and lse have no stride argument: a view of wider rows would be written across its neighbours."""
    c = _py_cache(weight=True, slot_pos=True)
    x, cu, ws = torch.zeros((6, 128), dtype=torch.float16), torch.zeros(3, dtype=torch.int32), torch.zeros(16, dtype=torch.uint8)
    wide, wide_lse = torch.zeros((6, 160), dtype=torch.float16), torch.zeros((6, 4))

    def call(o, lse):
        fq.flex_paged_attention(c, x, 128, 2, x.clone(), x.clone(), 128, o, lse, cu, 3, ws, total=6)
    for o in (wide[:, :128], wide[:, 32:], torch.zeros((9, 128), dtype=torch.float16)[3:8], torch.zeros((128, 6), dtype=torch.float16).T, torch.zeros((12, 128), dtype=torch.float16)[::2]):
        with pytest.raises(ValueError, match="o: "):
            call(o, None)
    o = torch.zeros((7, 128), dtype=torch.float16)
    for lse in (wide_lse[:, :2], torch.zeros((2, 6)).T):
        with pytest.raises(ValueError, match="lse"):
            call(o[:6], lse)
    for good in (o, o[1:], o.view(-1), o.view(7, 2, 64)):                # any shape, as long as the rows follow each other
        with pytest.raises(ValueError, match="CUDA"):                    # (the caches of this file have no device)
            call(good, torch.zeros((6, 2)))


def test_binding_refuses_sizes_that_do_not_fit_the_call():
    """The C arguments are 32 bits wide and ctypes cuts what does not fit: a budget of 2^32 + 5 slots
    would keep 5."""
    c = _py_cache(weight=True, slot_pos=True)
    x, cu, ws = torch.zeros((6, 128), dtype=torch.float16), torch.zeros(3, dtype=torch.int32), torch.zeros(1 << 20, dtype=torch.uint8)
    new = torch.zeros(2, dtype=torch.int32)
    big = (1 << 32) + 5
    for budget, recent in ((big, 4), (1 << 31, 4), (8, 1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            fq.flex_paged_evict(c, budget, recent, new, ws)
        if recent == 4:
            with pytest.raises(ValueError, match="32 bits"):
                fq.flex_paged_evict_ws_bytes(c, budget)
    for call in (lambda **kw: fq.flex_paged_store_kv(c, x, x, 128, cu, **kw), lambda **kw: fq.flex_paged_load_kv(c, x, x, 128, cu, **kw),
                 lambda **kw: fq.flex_paged_attention(c, x, 128, 2, x, x, 128, x.clone(), None, cu, ws=ws, **kw)):
        with pytest.raises(ValueError, match="32 bits"):
            call(most=big, total=6)
        with pytest.raises(ValueError, match="32 bits"):
            call(most=3, total=big)
        with pytest.raises(ValueError, match="32 bits|offsets"):
            call(most=3, total=6, batch=big)
    with pytest.raises(ValueError, match="32 bits"):
        fq.flex_paged_store_kv(c, x, x, 128, None, big)
    for kw in (dict(n_heads=big, total=6, most=3), dict(n_heads=2, total=big, most=3), dict(n_heads=2, total=6, most=big)):
        with pytest.raises(ValueError, match="32 bits"):
            fq.flex_paged_attention_ws_bytes(c, **kw)
    with pytest.raises(ValueError, match="32 bits"):
        fq.flex_paged_attention(c, x, 128, big, x, x, 128, x.clone(), None, cu, 3, ws, total=6)


def test_a_cache_without_weights_may_say_so():
    c = _py_cache(weight=False, slot_pos=False)
    assert c.weight is None and c.slot_pos is None and not c.struct().weight and not c.struct().slot_pos
    with pytest.raises(ValueError, match="weight"):
        _py_cache(weight=1)
    with pytest.raises(ValueError, match="slot_pos"):
        _py_cache(slot_pos=1)
