"""Outputs that would be written into a call's inputs are refused: what a CTA reads would depend on which has written first.

Rows of the two may lie between one another (columns of one tensor).  The refusals need no GPU; addresses are made up, and every
call with such addresses is one that is refused before anything is launched."""
import ctypes

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


# ------------------------------------------------------------------------------------------------ append and attention
H, D = 2, 64


class Cache(ctypes.Structure):
    """A cache's handle as far as the checks of arguments read it, on no device: a call that passes them is refused for that."""
    _fields_ = [("d", uw.KVDesc), ("device", ctypes.c_int), ("rest", ctypes.c_byte * 4096)]


@pytest.fixture
def handle():
    return Cache(uw.KVDesc(4096, 8192, 4, 2048, 128, 64, 16, H, D), -1)


def batch_of(rows):
    return uw.KVBatchDesc(1, 4096, 4096, 4096, 4, 4)


def append(handle, rows, q, ldq, q_out, ldq_out, k=0, ldk=0, v=0, ldv=0, q_heads=4, dtype=1):
    s = uw.lib().uw_kv_append(ctypes.byref(handle), ctypes.byref(batch_of(rows)), None, rows, dtype, q, ldq, q_heads, k, ldk, v, ldv, None, q_out, ldq_out, None)
    return s, uw.lib().uw_last_error().decode()


def overlaps(got, words):
    s, m = got
    assert s == uw.ERR_INVALID_ARG and words in m, got


def passes(got):
    """The checks are behind it: no device, or not the cache's."""
    s, m = got
    assert s == uw.ERR_CUDA or (s == uw.ERR_INVALID_ARG and "the cache is on device -1" in m), got


A = 1 << 30
WQ, WK = 4 * D, H * D      # elements of a row


@pytest.mark.parametrize("rows", [1, 2, 77])
def test_append_queries(handle, rows):
    ld = WQ + 2 * WK
    overlaps(append(handle, rows, A, ld, A + 16, ld), "q_out")                       # shifted by eight elements
    overlaps(append(handle, rows, A, ld, A - 16, ld), "q_out")
    overlaps(append(handle, rows, A, ld, A + 2 * (WQ - 8), ld), "q_out")
    overlaps(append(handle, rows, A, ld, A, ld, dtype=0), "q_out")                   # another type
    overlaps(append(handle, rows, A, ld, A + 4 * (WQ - 8), 2 * ld, dtype=0), "q_out")
    passes(append(handle, rows, A, ld, A, ld))                                       # itself
    passes(append(handle, rows, A, ld, A + 2 * WQ, ld))                              # columns beside it
    passes(append(handle, rows, A, ld, A + 4 * WQ, 2 * ld, dtype=0))                 # behind fp32 rows, in their padding
    passes(append(handle, rows, A, 0, A + 2 * WQ * rows, 0))                         # behind it
    passes(append(handle, rows, A + 2 * WQ * rows, 0, A, 0))
    if rows > 1:
        overlaps(append(handle, rows, A, WQ, A, ld), "q_out")                        # itself with another stride
        overlaps(append(handle, rows, A, ld, A + 2 * (ld - 8), ld), "q_out")         # the next row
        overlaps(append(handle, rows, A, 0, A + 2 * WQ * (rows - 1), 0), "q_out")    # the last row
        overlaps(append(handle, rows, A + 2 * WQ * (rows - 1), 0, A, 0), "q_out")


@pytest.mark.parametrize("rows", [1, 2, 77])
@pytest.mark.parametrize("dtype", [0, 1])
def test_append_queries_into_keys_and_values(handle, rows, dtype):
    """q, k and v as columns of one product's output; turned queries over the keys or values would be read as those."""
    ld, es = WQ + 2 * WK, 4 if dtype == 0 else 2
    k, v, o = A + es * WQ, A + es * (WQ + WK), A + es * ld * rows + 64
    c = lambda q_out, ldo: append(handle, rows, A, ld, q_out, ldo, k, ld, v, ld, dtype=dtype)  # noqa: E731
    passes(c(o, 0))
    if dtype == 1:
        passes(c(A, ld))
    passes(append(handle, rows, 0, 0, 0, 0, k, ld, v, ld, dtype=dtype))
    passes(append(handle, rows, 0, 0, 0, 0, k, ld, k, ld, dtype=dtype))   # keys that are the values
    far = append(handle, rows, o + 4 * ld * rows, ld, k, ld * es // 2, k, ld, v, ld, dtype=dtype)
    overlaps(far, "q_out")
    overlaps(append(handle, rows, o + 4 * ld * rows, ld, v + es * (WK - 8), ld * es // 2, k, ld, v, ld, dtype=dtype), "q_out")


def attend(handle, rows, q, ldq, out, ldo):
    s = uw.lib().uw_kv_attend(ctypes.byref(handle), ctypes.byref(batch_of(rows)), rows, q, ldq, 4, 1.0, 1, 0, out, ldo, None, 4096, 1 << 40, None)
    return s, uw.lib().uw_last_error().decode()


@pytest.mark.parametrize("rows", [1, 2, 300])
def test_attend_out_over_q(handle, rows):
    ld = 3 * WQ
    overlaps(attend(handle, rows, A, ld, A, ld), "out")
    overlaps(attend(handle, rows, A, ld, A + 16, ld), "out")
    overlaps(attend(handle, rows, A, ld, A - 16, ld), "out")
    overlaps(attend(handle, rows, A, ld, A + 2 * (WQ - 8), ld), "out")
    passes(attend(handle, rows, A, ld, A + 2 * WQ, ld))
    passes(attend(handle, rows, A, ld, A + 4 * WQ, ld))
    passes(attend(handle, rows, A + 4 * WQ, ld, A, ld))
    passes(attend(handle, rows, A, 0, A + 2 * WQ * rows, 0))
    if rows > 1:
        overlaps(attend(handle, rows, A, ld, A + 2 * (ld - 8), ld), "out")
        overlaps(attend(handle, rows, A, ld, A, 2 * ld), "out")
        overlaps(attend(handle, rows, A, 0, A + 2 * WQ * (rows - 1), 0), "out")
        overlaps(attend(handle, rows, A + 2 * WQ * (rows - 1), 0, A, 0), "out")
