"""Calls of the MoE step with no tokens or no rows: nothing is refused that the
other calls of the step accept."""
import pytest
import torch

import grouped_fp8_weight_gb300 as dg
from grouped_fp8_weight_gb300 import binding as B
from grouped_fp8_weight_gb300 import build as build_mod

P = 0x10000                     # never read: nothing is launched


@pytest.mark.parametrize("T,topk,rows,pairs", [(4, 2, P, None), (4, 2, P, P), (0, 1, None, None),
                                               (0, 2, None, None), (0, 2, None, P)])
def test_a_cast_to_no_rows_is_ok_without_device(T, topk, rows, pairs):
    """Every slot unused or no tokens at all, and no padding."""
    build_mod.build()
    assert B.lib().dg_quant_rows_fp8(P, T, 64, topk, rows, pairs, 0, None, None, None) == B.DG_OK


def test_a_row_map_without_its_pairs_is_still_refused():
    build_mod.build()
    for rows, pairs in ((P, None), (None, P)):
        assert B.lib().dg_quant_rows_fp8(P, 4, 64, 2, rows, pairs, 8, P, P, None) == B.DG_ERR_INVALID_ARG
        assert "go together" in B.lib().dg_last_error().decode()


@pytest.mark.gpu
def test_a_cast_of_no_tokens_fills_the_padding_rows():
    idx = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    _, rows, pairs = dg.dg_moe_sort(idx, 3, 16)
    R = pairs.shape[0]
    assert R == 45
    x = torch.empty(0, 144, dtype=torch.bfloat16, device="cuda")
    q = torch.full((R, 144), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((R, 2), float("nan"), device="cuda")
    dg.dg_quant_rows_fp8(x, q, s, rows, pairs)
    dg.dg_sync_check()
    assert not q.any() and bool((s == 2.0 ** -100 * (1 / torch.tensor(448.0, device="cuda"))).all())


@pytest.mark.gpu
def test_a_cast_of_tokens_without_experts_to_no_rows():
    idx = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    _, rows, pairs = dg.dg_moe_sort(idx, 3, 16)
    x = torch.ones(5, 144, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(0, 144, dtype=torch.uint8, device="cuda")
    dg.dg_quant_rows_fp8(x, q, torch.empty(0, 2, device="cuda"), rows, pairs[:0])
    dg.dg_sync_check()
