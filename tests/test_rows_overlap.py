"""Outputs that would be written into a call's inputs are refused: what a CTA reads would depend on which has written first.

Rows of the two may lie between one another (columns of one tensor).  The refusals need no GPU; addresses are made up, and every
call with such addresses is one that is refused before anything is launched."""
import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw
from test_kv_host import edit


@pytest.mark.parametrize("rows_before", [1, 1 << 20, (1 << 20) + 5, (1 << 21) - 1])
@pytest.mark.parametrize("vocab,column", [(1, 0), (2, 0), (2, 1), (2, -1), (3, 2)])
def test_edits_far_apart(rows_before, vocab, column):
    """Rows of three logits, some of them edited, and an output that begins many rows in front, in the same columns or one on."""
    at = 1 << 40
    assert edit(rows=1 << 21, vocab=vocab, ld=3, ld_out=3, logits=at, out=at - 12 * rows_before + 4 * column) == uw.ERR_INVALID_ARG
    assert edit(rows=1 << 21, vocab=vocab, ld=3, ld_out=3, out=at, logits=at - 12 * rows_before + 4 * column) == uw.ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("before", [3, (1 << 20) + 5])
@pytest.mark.parametrize("column", [1, 2])
def test_edits_between_one_another(before, column):
    """One column of logits and another of outputs that begins many rows in front of it."""
    rows = (1 << 20) + 64
    big = torch.arange((rows + before) * 3, dtype=torch.float32, device="cuda").view(-1, 3) % 1000
    was = big.clone()
    bias_ids = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
    bias = torch.full((rows, 1), 0.5, device="cuda")
    uw.edit_logits(big[before:, :1], rows, 1, big[:rows, column:column + 1], bias_ids=bias_ids, bias=bias)
    torch.cuda.synchronize()
    was[:rows, column] = was[before:, 0] + 0.5
    assert torch.equal(big, was)
