"""A decoder layer over pages: the library's LayerNorm, dequantising GEMMs and paged attention and
store put together as a serving loop does, for a ragged batch, against the layer calls over a
contiguous cache, one sequence at a time. Both quantise the same keys and values; queries are
scaled by 1/8 (head_dim 64), which fp16 holds exactly. The bound is the layers' own
(_helpers.layer_tolerance). Slots are the same but for codes next to a border: the projections'
fp32 sums are split differently for other row counts, so a value may be off by its last fp16 place."""
import pytest
import torch

import group_wise_int4_b200 as fq
import synth
from _helpers import assert_layer_close, sync_status, to_np

pytestmark = pytest.mark.gpu

H, HEADS, DIM, FFN = 512, 8, 64, 1280


class PagedLayer:
    def __init__(self, layer, cache, rows):
        self.L, self.cache = layer, cache
        buf = lambda *s: torch.empty(s, dtype=torch.float16, device="cuda")
        self.n1, self.qkv, self.o, self.x1, self.n2, self.f = (buf(rows, w) for w in (H, 3 * H, H, H, H, FFN))
        shapes = ((3 * H, H), (H, H), (FFN, H), (H, FFN))
        self.gws = torch.zeros(max(16, *(fq.flex_gemm_ws_bytes(m, n, k) for n, k in shapes for m in range(1, rows + 1))),
                               dtype=torch.uint8, device="cuda")

    def step(self, x, y, cu, total, most, aws):
        L, w, v = self.L, self.L.w, self.L.vec
        n1, qkv, o, x1, n2, f = (t[:total] for t in (self.n1, self.qkv, self.o, self.x1, self.n2, self.f))
        fq.flex_layernorm(x, v["ln1_g"], v["ln1_b"], n1, total, H)
        fq.flex_dequant_gemm(n1, w["w_qkv"], v["b_qkv"], None, qkv, total, fq.FLEX_EPI_NONE, self.gws)
        qkv[:, :H] *= 0.125
        fq.flex_paged_attention(self.cache, qkv, 3 * H, HEADS, qkv[:, H:], qkv[:, 2 * H:], 3 * H, o, None, cu, most, aws, total=total)
        fq.flex_paged_store_kv(self.cache, qkv[:, H:], qkv[:, 2 * H:], 3 * H, cu, most, total=total)
        fq.flex_dequant_gemm(o, w["w_o"], v["b_o"], x, x1, total, fq.FLEX_EPI_RESIDUAL, self.gws)
        fq.flex_layernorm(x1, v["ln2_g"], v["ln2_b"], n2, total, H)
        fq.flex_dequant_gemm(n2, w["w_fc1"], v["b_fc1"], None, f, total, fq.FLEX_EPI_RELU, self.gws)
        fq.flex_dequant_gemm(f, w["w_fc2"], v["b_fc2"], x1, y, total, fq.FLEX_EPI_RESIDUAL, self.gws)


def test_a_ragged_batch_through_a_layer():
    lens, steps = [20, 7, 33], 4
    layer = fq.FlexLayer(synth.layer_params(H, FFN, 60), HEADS)
    table = torch.tensor([[5, 0, 9], [2, 7, 3], [8, 1, 4]], dtype=torch.int32, device="cuda")
    ctx = torch.zeros(3, dtype=torch.int32, device="cuda")
    cache = fq.FlexPagedCache(table, ctx, 10, 16, HEADS, DIM)
    mine = PagedLayer(layer, cache, sum(lens))
    aws = torch.empty(max(fq.flex_paged_attention_ws_bytes(cache, HEADS, sum(lens), max(lens)),
                          fq.flex_paged_attention_ws_bytes(cache, HEADS, 3, 1)), dtype=torch.uint8, device="cuda")
    prompts = [synth.activations((n, H), 61 + i, device="cuda") for i, n in enumerate(lens)]
    tokens = [[synth.activations((1, H), 70 + 3 * s + i, device="cuda") for i in range(3)] for s in range(steps)]

    # one sequence at a time, contiguous
    want = [[] for _ in lens]
    caches = []
    for i, n in enumerate(lens):
        kv = fq.FlexKVCache(1, HEADS, DIM, n + steps)
        ws = torch.zeros(max(fq.flex_workspace_bytes(layer, 1, n), fq.flex_workspace_bytes(layer, 1, 1)), dtype=torch.uint8, device="cuda")
        y = torch.empty_like(prompts[i])
        fq.flex_prefill_layer(layer, kv, prompts[i], y, 1, n, ws)
        want[i].append(y)
        for s in range(steps):
            y = torch.empty((1, H), dtype=torch.float16, device="cuda")
            fq.flex_decode_layer(layer, kv, tokens[s][i], y, 1, n + s, ws)
            want[i].append(y)
        caches.append(kv)
    sync_status()

    # all of them, ragged, over pages: the prompts, then a token each
    offsets = torch.tensor([0, 20, 27, 60], dtype=torch.int32, device="cuda")
    y = torch.empty((60, H), dtype=torch.float16, device="cuda")
    mine.step(torch.cat(prompts), y, offsets, 60, 33, aws)
    ctx += torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = [list(y.split(lens))]
    for s in range(steps):
        y = torch.empty((3, H), dtype=torch.float16, device="cuda")
        mine.step(torch.cat(tokens[s]), y, torch.arange(4, dtype=torch.int32, device="cuda"), 3, 1, aws)
        ctx += 1
        got.append(list(y.split(1)))
    sync_status()
    for i in range(3):
        for s in range(steps + 1):
            assert_layer_close(got[s][i], to_np(want[i][s]), f"sequence {i}, step {s}")
        # the slots: equal codes, or neighbours (a step is the group's span / 15)
        n = lens[i] + steps
        rows = [torch.empty((n, H), dtype=torch.float16, device="cuda") for _ in "kv"]
        one = fq.FlexPagedCache(table[i:i + 1].contiguous(), ctx[i:i + 1].contiguous(), pools=(cache.k_codes, cache.k_meta, cache.v_codes,
                                                                                             cache.v_meta))
        fq.flex_paged_load_kv(one, *rows, H, None, n)
        sync_status()
        kv = caches[i]
        for x, codes, meta in zip(rows, (kv.k_codes, kv.v_codes), (kv.k_meta, kv.v_meta)):
            ref = fq.flexq_decompress(codes, meta, (1, HEADS, n, DIM), kv.cfg)[0].transpose(0, 1).reshape(n, H)
            span = meta[0, ..., 0, :].float()
            step = (1 / span[..., 1]).transpose(0, 1).repeat_interleave(DIM, 1)
            assert bool(((x.float() - ref.float()).abs() <= 1.1 * step).all())
