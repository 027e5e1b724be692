"""Failure detection in the paged attention's tensor-core tiles, without a fault.

flex_set_gemm_gate holds back the values of every later tile (the keys flow, so scores are
computed and the warps that issue products, those that take exponentials and those that
load are all in the middle of their work); the test passes a zero that nothing changes and
a limit of 5 ms. Each block's wait runs out, its roles give up, what was issued ends (by
the fixed limit, not by the short one), tensor memory is freed and the call returns. The
status is FLEX_ERR_TIMEOUT once, and the same call right after gives the same bits as
before: no late arrival or product has reached another block."""
import re

import pytest
import torch

import group_wise_int4_b200 as fq
from test_gpu_paged import Case, _scaled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,bits,group", [(64, 4, 64), (128, 4, 64), (128, 8, 32)])
@pytest.mark.parametrize("ctx,n,cross", [([40, 0], [50, 33], True),              # one block of keys: all scores are issued at once
                                         ([0, 60], [40, 64], False),             # fresh keys first, and keys of both kinds
                                         ([900, 130, 64], [40, 1, 90], False),   # 128 rows; more blocks than stages
                                         ([700, 100], [290, 150], True),         # 256 rows
                                         ([6000], [100], False)])                # parts of one sequence, joined
def test_held_values_time_out_then_the_next_call_is_exact(dim, bits, group, ctx, n, cross):
    c = Case(70, ctx, heads=2, dim=dim, bits=bits, group=group, page=64, room=max(n))
    q = _scaled(c, n, 2)
    k, v = (None, None) if cross else ([c.rows(m) for m in n], [c.rows(m) for m in n])
    o, ls = c.attend(q, k, v)
    gate = torch.zeros(1, dtype=torch.int32, device="cuda")      # nothing ever sets it
    old = fq.flex_set_wait_limit_ns(5_000_000)
    fq.flex_set_gemm_gate(gate)
    try:
        with pytest.raises(AssertionError, match=re.escape(fq.flex_status_string(fq.FLEX_ERR_TIMEOUT))):   # attend checks it
            c.attend(q, k, v, check=False)
    finally:
        fq.flex_set_gemm_gate(None)
        fq.flex_set_wait_limit_ns(old)
    assert fq.flex_get_status() == fq.FLEX_OK                    # the status word was cleared
    again = c.attend(q, k, v, check=False)
    assert torch.equal(o, again[0]) and torch.equal(ls, again[1])


def test_an_open_gate_changes_nothing():
    c = Case(71, [300, 20], heads=2, room=60)
    n = [60, 5]
    q, k, v = _scaled(c, n, 2), [c.rows(m) for m in n], [c.rows(m) for m in n]
    o, ls = c.attend(q, k, v)
    gate = torch.ones(1, dtype=torch.int32, device="cuda")
    fq.flex_set_gemm_gate(gate)
    try:
        again = c.attend(q, k, v)
    finally:
        fq.flex_set_gemm_gate(None)
    assert torch.equal(o, again[0]) and torch.equal(ls, again[1])
