"""Attention by items of 256 rows that hold few: single tokens beside chunks of prompts, whose keys and values go through the same ring as
long items' do, with values that are put right (in front of a window, behind a sequence) in many places of it.  Bounds as in the tests of
attention; and the same bits in every run."""
import pytest
import torch

from test_gpu_kv import BF16, attend, batch_of, check_attend
from test_gpu_kv_plans import item_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [8, 16, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 130, 1000])
def test_single_tokens_beside_a_chunk(D, window, page):
    new, past = [1] * 32 + [260] + [2] * 8, [(997 * i) % 2500 for i in range(41)]
    H, G = 4, 24
    c = batch_of(new, past, page, H=H, D=D)
    rows = sum(new)
    assert item_rows(c, rows, H * G, D) == 256
    q = (torch.randn(rows, H * G, D, generator=c["g"]) * 0.5).to(BF16).cuda()
    out, lse = attend(c, q, H * G, window=window)
    check_attend(c, q, out, lse, new, window=window)
    for _ in range(30):
        o, l = attend(c, q, H * G, window=window)
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("few,R", [(1, 128), (3, 256)])
def test_tokens_of_many_heads_behind_a_window(D, few, R):
    """64 query heads for each key head: one token is half a tile of rows, three a tile and a half."""
    S, H, G = 40, 4, 64
    new = [few if i % 9 else 1 for i in range(S)]
    past = [(613 * i) % 3000 for i in range(S)]
    c = batch_of(new, past, 16, H=H, D=D)
    rows = sum(new)
    assert item_rows(c, rows, H * G, D) == R
    q = torch.randn(rows, H * G, D, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, H * G, window=1000)
    check_attend(c, q, out, lse, new, window=1000)
    for _ in range(50):
        o, l = attend(c, q, H * G, window=1000)
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("D", [64, 128])
def test_short_items_one_after_another(D):
    """Many items of one or two tiles of keys in a range: every tile's values are put right."""
    new = [5 if i % 3 else 0 for i in range(300)]
    new[7] = 900
    past = [(31 * i) % 200 for i in range(300)]
    c = batch_of(new, past, 16, H=2, D=D)
    rows = sum(new)
    G = 40
    assert item_rows(c, rows, 2 * G, D) == 256
    q = torch.randn(rows, 2 * G, D, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, 2 * G)
    check_attend(c, q, out, lse, new)
    for _ in range(20):
        o, l = attend(c, q, 2 * G)
        assert torch.equal(o, out) and torch.equal(l, lse)
