"""Attention by each form of the first kernel that cuts the work, and by each size of items: which one a call takes is derived from its
sizes and from its workspace's (two places of R rows for each SM's range), not assumed.

The small form holds up to 512 sequences and 4096 tiles of rows; the general one any number.  More tiles than that come with items of
256 rows alone: by items of 16 a call brings 16 rows a sequence at most on average, by 128 at most 128, so at most two tiles for each of
512 sequences.  Bounds as in the tests of attention."""
import math

import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw
from test_gpu_kv import BF16, F64, attend, batch_of, check_attend, plain_attend

pytestmark = pytest.mark.gpu


def item_rows(c, rows, Hq, D):
    need = c["cache"].workspace_size(c["batch"], rows, Hq)
    return need // (2 * torch.cuda.get_device_properties(0).multi_processor_count * (D + 2) * 4)


def small_form(S, rows, group, R):
    return S <= 512 and rows * group // R + S <= 4096


CASES = [
    # sequences, new tokens of each, the longest past, Hq, H, D, window, causal, R
    (520, 5, 40, 64, 1, 64, 0, True, 256),
    (520, 5, 40, 128, 2, 128, 0, True, 256),
    (600, 3, 700, 64, 1, 64, 50, True, 256),
    (530, 9, 90, 32, 1, 64, 0, False, 256),
    (2100, 3, 30, 64, 1, 64, 0, True, 256),     # the line does not fit in shared memory
    (2100, 1, 300, 64, 1, 64, 0, True, 128),
    (513, 4, 500, 16, 2, 64, 100, True, 128),
    (513, 1, 900, 16, 2, 128, 0, True, 16),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_general_form_by_sequences(case):
    S, few, most, Hq, H, D, window, causal, R = case
    new = [0 if i % 11 == 7 else few for i in range(S)]
    new[3] = few + 2 * R // (Hq // H)                 # several tiles of rows
    past = [(i * 7919) % most for i in range(S)]
    past[5] = 4000
    c = batch_of(new, past, 16, H=H, D=D)
    rows = sum(new)
    assert item_rows(c, rows, Hq, D) == R and not small_form(S, rows, Hq // H, R)
    q = torch.randn(rows, Hq, D, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, Hq, causal, window)
    check_attend(c, q, out, lse, new, causal, window)


@pytest.mark.parametrize("S,n,window", [(16, 1030, 0), (5, 3400, 200)])
def test_general_form_by_tiles(S, n, window):
    """Few sequences with more tiles of rows than the small form holds; some of the sequences are checked, their first, middle and last rows."""
    Hq, D, R = 64, 64, 256
    new, past = [n] * S, [(37 * i) % 300 for i in range(S)]
    c = batch_of(new, past, 32, H=1, D=D)
    rows = sum(new)
    assert item_rows(c, rows, Hq, D) == R and not small_form(S, rows, Hq, R) and S <= 512
    q = torch.randn(rows, Hq, D, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, Hq, window=window)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    for s in range(S):
        a = c["at"][s]
        k, v = c["seqs"][s]
        for lo, hi in ((0, 40), (n // 2, n // 2 + 40), (n - 40, n)):
            upto = past[s] + hi                       # the rows lo..hi are the last ones of this much of the sequence
            ref, rl, b, bl = plain_attend(q[a + lo:a + hi].cpu(), k[:upto], v[:upto], hi - lo, D ** -0.5, True, window)
            assert ((out[a + lo:a + hi].cpu().to(F64) - ref).abs() <= b).all()
            assert ((lse[a + lo:a + hi].cpu().to(F64) - rl).abs() <= bl).all()


@pytest.mark.parametrize("S,few,group,R", [(512, 1, 16, 16), (512, 9, 14, 128), (512, 8, 64, 256), (17, 16, 1, 16), (17, 17, 1, 128), (3, 128, 1, 128),
                                           (3, 129, 1, 256)])
def test_small_form_up_to_its_end(S, few, group, R):
    """The last sizes of the small form and of each size of items, and one more."""
    new, past = [few] * S, [(i * 31) % 70 for i in range(S)]
    c = batch_of(new, past, 8, H=1, D=64)
    rows = sum(new)
    assert item_rows(c, rows, group, 64) == R and small_form(S, rows, group, R)
    q = torch.randn(rows, group, 64, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, group)
    check_attend(c, q, out, lse, new)


def test_one_chunk_beside_many_single_tokens():
    """A batch whose average is below 16 rows: its one chunk goes by items of 16 rows, in many tiles."""
    new = [1] * 256
    new[100] = 512
    past = [(i * 37) % 200 for i in range(256)]
    c = batch_of(new, past, 16, H=1, D=64)
    rows = sum(new)
    assert item_rows(c, rows, 4, 64) == 16
    q = torch.randn(rows, 4, 64, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, 4)
    check_attend(c, q, out, lse, new)
    idle = [0] * 128                                  # a step of 128 places, one of them with a prompt
    idle[77] = 500
    c = batch_of(idle, [0] * 128, 16, H=1, D=64)
    assert item_rows(c, 500, 4, 64) == 16
    q = torch.randn(500, 4, 64, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, 4)
    check_attend(c, q, out, lse, idle)
    assert not math.isinf(float(lse.max()))
