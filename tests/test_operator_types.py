"""Tensors of another type than a call reads or writes are refused before anything runs."""
import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("w", [torch.zeros(2, 16, 64, dtype=F16), torch.zeros(2, 16, 64, dtype=BF16)])
def test_group_weights(w):
    # half-precision numbers would be read as bf16; weights in host memory would be read from the device
    with pytest.raises(ValueError):
        uw.Group(w)


def refused(call, *args, **kw):
    with pytest.raises(ValueError, match="the call's type is"):
        call(*args, **kw)


@pytest.mark.parametrize("held,asked", [(F32, uw.OUT_BF16), (BF16, uw.OUT_F32), (F16, uw.OUT_BF16)])
def test_calls(held, asked):
    t = torch.zeros(4, 64, dtype=held)
    g = uw.Group.__new__(uw.Group)
    g._h = None
    refused(g.matmul, 0, 0, 4, t, x_rows=4, out_dtype=asked)
    refused(uw.Router(64, 2).route, t, 4, 0, 0, 0, 0, 0, dtype=asked)
    refused(uw.token_logprobs, t, 4, 64, dtype=asked)
    n = uw.BlockNorm(64, res_dtype=asked, block_dtype=asked)
    refused(n.run, 4, t, 0)
    refused(n.run, 4, 0, t)
    refused(n.run, 4, 0, 0, y=t)
    if held != BF16:
        refused(n.run, 4, 0, 0, u=t)


def test_group_output_is_bf16_unless_asked():
    g = uw.Group.__new__(uw.Group)
    g._h = None
    refused(g.matmul, 0, 0, 4, torch.zeros(4, 64), x_rows=4)
