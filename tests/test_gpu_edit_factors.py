"""Penalties on repeated tokens over the whole range of fp32: a logit above 0 is divided, any other multiplied.

A product is rounded once, by 2^-24 of itself or half the smallest number, 2^-150.  A quotient is a product with the reciprocal of the
factor: the factor or its multiple by a power of 2 (exact), so that the reciprocal is an ordinary number, within 2^-24 of itself; the product,
2^-24 or 2^-150; the power of 2, exact or 2^-150 (a product that is below the ordinary numbers has no power of 2 to make it larger: those are
of factors above 2^126, by 2^-64).  In all (2^-23 + 2^-47) of the value and 2^-149.  A bias: one sum more, 2^-24 of it.  A bf16 output adds 2^-8 of the
value, or half of the smallest, 2^-134.  A value becomes infinite from the middle between the type's largest number and 2^128 on, 2^128 (1 - 2^-25)
or for bf16 2^128 (1 - 2^-9); nearer to it than the other bounds it may be either."""
import math

import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw

pytestmark = pytest.mark.gpu
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
DT = {F32: uw.OUT_F32, BF16: uw.OUT_BF16}
FACTORS = [2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 1.5 * 2.0 ** -127, 2.0 ** -126, 1e-30, 0.7, 1.0, 1.1, 1.3, 3.0, 1e30, 2.0 ** 126, 2.0 ** 127, 3e38]


def check(got, want, more):
    dtype, got = got.dtype, got.double()
    border = 2.0 ** 128 * (1 - 2.0 ** (-9 if dtype == BF16 else -25))
    over, under = want.abs() * (1 - 2.0 ** -22) >= border, want.abs() * (1 + 2.0 ** -22) < border
    assert torch.equal(got[over], want[over].sign() * math.inf)
    assert torch.isfinite(got[under]).all()
    odd = torch.isinf(got)
    assert torch.equal(got[odd].sign(), want[odd].sign())
    bound = (2.0 ** -23 + 2.0 ** -47) * want.abs() + more
    if dtype == BF16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -134
    assert ((got - want).abs()[~odd] <= bound[~odd]).all()


@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("pad", [0, 1])     # rows of 16-byte pieces and others
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quotients_and_products(dtype, pad, place):
    g = torch.Generator().manual_seed(3)
    R, V = len(FACTORS), 2000
    rep = torch.tensor(FACTORS, dtype=torch.float64).to(F32)
    x = (torch.randn(R, V + pad, generator=g) * 3).to(dtype)
    # logits beside the factors, whose quotients are ordinary numbers
    x[:, :200] = (torch.randn(R, 200, generator=g).abs() * rep[:, None].clamp(1e-38, 1e37)).to(dtype)
    x[:, 200:210] = torch.tensor([0.0, -0.0, 1e-38, -1e-38, 2.0 ** -149, 3e38, -3e38, math.inf, -math.inf, 1.0]).to(dtype)
    tokens = torch.arange(0, 1500, dtype=I32).repeat(R, 1)
    want = x[:, :V].double()
    z = want[:, :1500].clone()
    want[:, :1500] = torch.where(z > 0, z / rep.double()[:, None], z * rep.double()[:, None])
    d = x.cuda()
    out = d if place else torch.zeros(R, V + pad, dtype=dtype, device="cuda")
    uw.edit_logits(d, R, V, out, tokens=tokens.cuda(), lengths=torch.full((R,), 1500, dtype=I32, device="cuda"), repetition=rep.cuda(), dtype=DT[dtype])
    torch.cuda.synchronize()
    got = out[:, :V].cpu()
    assert torch.equal(got[:, 1500:], x[:, 1500:V])
    check(got, want, 2.0 ** -149)


def test_quotients_under_biases():
    """A token with a bias goes through the same penalty."""
    R, V = len(FACTORS), 300
    rep = torch.tensor(FACTORS, dtype=torch.float64).to(F32)
    x = (rep[:, None] * torch.linspace(0.01, 1.0, V)).contiguous()
    ids = torch.arange(0, 64, dtype=I32).repeat(R, 1)
    bias = torch.full((R, 64), 0.25)
    want = x.double() / rep.double()[:, None]
    want[:, :64] += 0.25
    out = torch.zeros(R, V, device="cuda")
    uw.edit_logits(x.cuda(), R, V, out, tokens=torch.arange(0, V, dtype=I32).repeat(R, 1).cuda(), lengths=torch.full((R,), V, dtype=I32, device="cuda"),
                   repetition=rep.cuda(), bias_ids=ids.cuda(), bias=bias.cuda())
    torch.cuda.synchronize()
    check(out.cpu(), want, 2.0 ** -24 * want.abs() + 2.0 ** -149)
