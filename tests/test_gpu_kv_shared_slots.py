"""Appends where rows meet in one slot: padded places of a batch that share a page, or a table that names one twice."""
import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.mark.parametrize("S,H,D,dtype", [(2, 8, 128, torch.float32), (64, 2, 64, BF16), (300, 4, 128, BF16)])
def test_one_slot_of_many_rows(S, H, D, dtype):
    """Every eight elements of the slot are some row's at that place; the other slots are left as they were."""
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    k, v = (torch.full((3, 16, H, D), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    cache = uw.KVCache(k, v)
    batch = uw.KVBatch(i32(list(range(S + 1))), i32([6] * S), i32([[1]] * S))
    # a row's elements are its number, a whole one that bf16 holds
    row = torch.arange(S, dtype=torch.float32).view(S, 1, 1).expand(S, H, D) % 256
    kn, vn = row.to(dtype).cuda().contiguous(), (-row).to(dtype).cuda().contiguous()
    cache.append(batch, S, kn, vn, dtype=uw.OUT_F32 if dtype == torch.float32 else uw.OUT_BF16)
    cache.check()
    for c, sign in ((k, 1), (v, -1)):
        got = (sign * c[1, 5].float()).view(H, D // 8, 8).cpu()
        assert (got == got[..., :1]).all()                    # one row's each
        assert ((got >= 0) & (got < min(S, 256))).all() and (got == got.round()).all()
        other = torch.ones(3, 16, dtype=torch.bool)
        other[1, 5] = False
        assert (c.cpu()[other] == 7).all()
