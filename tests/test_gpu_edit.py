"""Edits of logits against a plain form in 64 bits.

An edited logit takes a product or a quotient, two of the penalties' terms and a sum of its biases, each rounded to fp32: within
(6 + the biases of the token) 2^-24 of the magnitudes that meet in it.  A bf16 output adds 2^-8 of the value.  Logits without an
edit are the input's, rounded to the output's type."""
import math

import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw

pytestmark = pytest.mark.gpu
F32, BF16, I32, F64 = torch.float32, torch.bfloat16, torch.int32, torch.float64
DT = {F32: uw.OUT_F32, BF16: uw.OUT_BF16}


def make(R, V, n=0, bias=0, masks=None, dtype=F32, pad=0, seed=0, repeat=50):
    g = torch.Generator().manual_seed(seed + R + V)
    c = dict(R=R, V=V, logits=(torch.randn(R, V + pad, generator=g) * 3).to(dtype), tokens=None, g=g)
    for k in ("lengths", "prompt_lengths", "repetition", "frequency", "presence", "bias_ids", "bias", "bias_lengths", "allowed", "mask_rows"):
        c[k] = None
    if n:
        c["tokens"] = torch.randint(0, max(1, min(V, repeat)), (R, n), generator=g, dtype=I32) * 13 % V
        c["lengths"] = torch.randint(0, n + 1, (R,), generator=g, dtype=I32)
        c["lengths"][0] = n
        c["prompt_lengths"] = (c["lengths"] * torch.rand(R, generator=g)).to(I32)
        c["repetition"] = 0.7 + torch.rand(R, generator=g)
        c["frequency"], c["presence"] = torch.rand(R, generator=g) - 0.3, torch.rand(R, generator=g)
    if bias:
        c["bias_ids"] = torch.randint(0, V, (R, bias), generator=g, dtype=I32)
        c["bias"] = torch.randn(R, bias, generator=g) * 5
    if masks:
        c["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (masks, (V + 31) // 32), generator=g, dtype=I32)
        if masks != R:
            c["mask_rows"] = torch.randint(-1, masks, (R,), generator=g, dtype=I32)
    return c


EDITS = ("tokens", "lengths", "prompt_lengths", "repetition", "frequency", "presence", "bias_ids", "bias", "bias_lengths", "allowed", "mask_rows")


def plain(c):
    R, V = c["R"], c["V"]
    x = c["logits"][:, :V].to(F64).clone()
    mag, terms = x.abs().clone(), torch.full((R, V), 6.0, dtype=F64)
    touched = torch.zeros(R, V, dtype=torch.bool)
    for r in range(R):
        one = lambda k, d: float(c[k][r]) if c[k] is not None else d  # noqa: E731
        if c["tokens"] is not None:
            n = min(max(int(c["lengths"][r]), 0), c["tokens"].shape[1])
            p = int(c["prompt_lengths"][r]) if c["prompt_lengths"] is not None else 0
            t = c["tokens"][r, :n].long()
            made = t[max(p, 0):]
            t, made = t[(t >= 0) & (t < V)], made[(made >= 0) & (made < V)]
            seen, count = torch.zeros(V, dtype=torch.bool), torch.bincount(made, minlength=V).to(F64)
            seen[t] = True
            rep = one("repetition", 1.0)
            x[r] = torch.where(seen, torch.where(x[r] > 0, x[r] / rep, x[r] * rep), x[r])
            mag[r] = torch.maximum(mag[r], x[r].abs())
            d = one("frequency", 0.0) * count + one("presence", 0.0) * (count > 0)
            x[r] -= d
            mag[r] += abs(one("frequency", 0.0)) * count + abs(one("presence", 0.0)) * (count > 0)
            touched[r] |= seen
        if c["bias_ids"] is not None:
            n = c["bias_ids"].shape[1] if c["bias_lengths"] is None else min(max(int(c["bias_lengths"][r]), 0), c["bias_ids"].shape[1])
            for i, b in zip(c["bias_ids"][r, :n].tolist(), c["bias"][r, :n].tolist()):
                if 0 <= i < V:
                    x[r, i] += b
                    mag[r, i] += abs(b)
                    terms[r, i] += 1
                    touched[r, i] = True
        if c["allowed"] is not None:
            m = r if c["mask_rows"] is None else int(c["mask_rows"][r])
            if 0 <= m < c["allowed"].shape[0]:
                v = torch.arange(V)
                dead = ((c["allowed"][m].long()[v // 32] >> (v % 32)) & 1) == 0
                x[r, dead] = -math.inf
                touched[r] |= dead
    return x, terms * 2.0 ** -24 * mag, touched


def run(c, out_dtype=None, place=False, stream=None, **kw):
    dtype = c["logits"].dtype
    out_dtype = out_dtype or dtype
    x = c["logits"].cuda()
    big = x if place else torch.full((c["R"], c["V"] + 3), 7.0, dtype=out_dtype, device="cuda")
    e = {k: c[k].cuda() if c[k] is not None else None for k in EDITS}
    uw.edit_logits(x, c["R"], c["V"], big, dtype=DT[dtype], out_dtype=DT[out_dtype], stream=stream, **e)
    torch.cuda.synchronize()
    out = big.cpu()
    pad = out[:, c["V"]:]
    if place:
        assert torch.equal(pad.view(torch.int16 if dtype == BF16 else I32), c["logits"][:, c["V"]:].view(torch.int16 if dtype == BF16 else I32))
    else:
        assert (pad == 7).all()
    return out[:, :c["V"]]


def check(c, out):
    ref, b, touched = plain(c)
    plain_bits = c["logits"][:, :c["V"]].to(out.dtype)
    left = ~touched
    assert torch.equal(torch.nan_to_num(out[left], 1e30), torch.nan_to_num(plain_bits[left], 1e30))
    got = out.to(F64)
    odd = ~torch.isfinite(ref)
    assert torch.equal(torch.nan_to_num(got[odd], 1e30), torch.nan_to_num(ref[odd], 1e30))
    if out.dtype == BF16:
        b = b * (1 + 2.0 ** -7) + 2.0 ** -8 * ref.abs()
    assert ((got - ref).abs()[~odd] <= b[~odd] + 1e-38).all()


CASES = [
    # R, V, n, bias, masks, pad
    (1, 1, 3, 1, 1, 0),
    (1, 128256, 4000, 8, None, 0),
    (3, 31, 40, 3, 3, 1),
    (5, 1000, 100, 0, 2, 0),
    (4, 32003, 700, 300, 4, 61),
    (2, 50001, 1, 0, None, 7),
    (9, 20000, 0, 5, None, 0),
    (200, 8193, 33, 2, 50, 0),
    (3, 4097, 0, 0, 3, 7),
]


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_edits(case, dtype, out_dtype):
    R, V, n, bias, masks, pad = case
    c = make(R, V, n, bias, masks, dtype, pad)
    out = run(c, out_dtype)
    check(c, out)
    assert torch.equal(torch.nan_to_num(run(c, out_dtype).float(), 1e30), torch.nan_to_num(out.float(), 1e30))
    if dtype == out_dtype:
        assert torch.equal(run(c, place=True), out)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_not_finite(dtype):
    c = make(4, 4096, 500, 10, 4, dtype, repeat=4096)
    t = c["tokens"][0, :6].long()
    c["logits"][:, t[0]], c["logits"][:, t[1]], c["logits"][:, t[2]] = math.nan, math.inf, -math.inf
    c["logits"][:, 100:140], c["logits"][1, 200:300] = math.nan, -math.inf
    c["logits"][:, 300] = torch.finfo(dtype).min
    c["allowed"][2] = 0
    c["allowed"][3] = -1
    for place in (False, True):
        check(c, run(c, place=place))


@pytest.mark.parametrize("place", [False, True])
def test_histories(place):
    """Ids outside the vocabulary, lengths past the tensor or negative, a prompt longer than the history; a token many times."""
    c = make(6, 3000, 300, 0, None, repeat=3000)
    c["tokens"][:, ::7] = -1
    c["tokens"][:, 3::7] = 3000
    c["tokens"][:, 4::9] = 2 ** 31 - 1
    c["tokens"][:, 5::11] = -2 ** 31
    c["lengths"] = torch.tensor([300, 301, 2 ** 31 - 1, -4, 0, 150], dtype=I32)
    c["prompt_lengths"] = torch.tensor([0, -9, 100, 0, 0, 2 ** 31 - 1], dtype=I32)
    check(c, run(c, place=place))
    c["prompt_lengths"] = None
    check(c, run(c, place=place))
    c = make(2, 500, 140000, 0, None, repeat=2)
    check(c, run(c, place=place))


@pytest.mark.parametrize("only", ["repetition", "frequency", "presence"])
def test_one_penalty(only):
    c = make(3, 5000, 200)
    for k in ("repetition", "frequency", "presence"):
        if k != only:
            c[k] = None
    check(c, run(c))


@pytest.mark.parametrize("place", [False, True])
def test_biases_of_one_token(place):
    """A token's several biases add up in the list's order, the same in every run; ids outside are passed over."""
    c = make(3, 2000, 0, 64)
    c["bias_ids"][0] = 77
    c["bias_ids"][1, ::2] = 78
    c["bias_ids"][2, :5] = torch.tensor([-1, 2000, 2 ** 31 - 1, -2 ** 31, 1999], dtype=I32)
    c["bias_lengths"] = torch.tensor([64, 100, 7], dtype=I32)
    out = run(c, place=place)
    check(c, out)
    x = c["logits"][0, 77].clone()
    for b in c["bias"][0]:
        x = x + b
    assert out[0, 77] == x
    c["bias_lengths"] = torch.tensor([-3, 0, 1], dtype=I32)
    check(c, run(c, place=place))


def test_masks_shared_and_missing():
    c = make(7, 777, 0, 0, 3)
    c["mask_rows"] = torch.tensor([2, 2, 0, -1, 3, 2 ** 31 - 1, 1], dtype=I32)
    check(c, run(c))
    check(c, run(c, place=True))
    c["mask_rows"] = None  # rows 3.. have no mask of their own
    check(c, run(c))
    wide = torch.zeros(3, 40, dtype=I32)
    wide[:, :25] = c["allowed"]
    c["allowed"] = wide
    check(c, run(c))


@pytest.mark.parametrize("place", [False, True])
def test_more_rows_than_a_grid_is_high(place):
    R, V = 70001, 40
    g = torch.Generator().manual_seed(2)
    x = torch.randn(R, V, generator=g).cuda()
    allowed = torch.randint(-2 ** 31, 2 ** 31, (R - 3, 2), generator=g, dtype=I32).cuda()   # the last rows have no mask
    tokens = torch.randint(0, V, (R, 3), generator=g, dtype=I32).cuda()
    presence = torch.rand(R, generator=g).cuda()
    lengths = torch.full((R,), 3, dtype=I32, device="cuda")
    want = x - presence[:, None] * torch.zeros(R, V, device="cuda").scatter_(1, tokens.long(), 1.0)
    v = torch.arange(V, device="cuda")
    want[:R - 3][((allowed[:, v // 32] >> (v % 32)) & 1) == 0] = -math.inf
    out = x if place else torch.empty_like(x)
    uw.edit_logits(x, R, V, out, tokens=tokens, lengths=lengths, presence=presence, allowed=allowed)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_strides_and_streams():
    """Columns of a wider tensor, in and out side by side in one tensor; a captured graph and its replay on new tokens."""
    c = make(5, 1000, 60, 4, 5)
    big = torch.zeros(5, 2048, device="cuda")
    big[:, :1000] = c["logits"].cuda()
    e = {k: c[k].cuda() if c[k] is not None else None for k in EDITS}
    uw.edit_logits(big, 5, 1000, big[:, 1024:], **e)
    torch.cuda.synchronize()
    assert torch.equal(big[:, 1024:2024].cpu(), run(c))
    assert (big[:, 2024:] == 0).all() and torch.equal(big[:, :1000].cpu(), c["logits"])
    out = torch.zeros(5, 1000, device="cuda")
    x = c["logits"].cuda()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        uw.edit_logits(x, 5, 1000, out, **e)
    e["tokens"].copy_((e["tokens"] + 1) % 1000)
    c["tokens"] = e["tokens"].cpu()
    g.replay()
    torch.cuda.synchronize()
    check(c, out.cpu())


def test_then_logprobs():
    """Edits, then the log probabilities of the edited row."""
    c = make(4, 3001, 90, 5, 4)
    x = c["logits"].cuda()
    e = {k: c[k].cuda() if c[k] is not None else None for k in EDITS}
    uw.edit_logits(x, 4, 3001, x, **e)
    lp, ids, top = torch.empty(4, device="cuda"), torch.empty(4, 5, dtype=I32, device="cuda"), torch.empty(4, 5, device="cuda")
    target = torch.tensor([1, 2, 3, 4], dtype=I32, device="cuda")
    uw.token_logprobs(x, 4, 3001, lp, targets=target, n_top=5, top_ids=ids, top_logprobs=top)
    torch.cuda.synchronize()
    ref, b, _ = plain(c)
    want = torch.log_softmax(ref, 1)
    tol = 2 * float(b[torch.isfinite(ref)].max()) + 1e-5
    t = want[torch.arange(4), target.cpu().long()]
    assert torch.equal(torch.isinf(lp.cpu()), torch.isinf(t))
    assert ((lp.cpu().to(F64) - t).abs()[torch.isfinite(t)] <= tol).all()
    assert ((top.cpu().to(F64) - want.gather(1, ids.cpu().long())).abs() <= tol).all()


def test_tensor_refusals():
    x = torch.zeros(2, 64, device="cuda")
    for kw in (dict(tokens=torch.zeros(2, 4, device="cuda"), lengths=torch.zeros(2, dtype=I32, device="cuda")),
               dict(allowed=torch.zeros(2, 1, dtype=I32, device="cuda")), dict(repetition=torch.ones(1, device="cuda")),
               dict(bias_ids=torch.zeros(2, 3, dtype=I32, device="cuda"), bias=torch.zeros(2, 2, device="cuda")),
               dict(tokens=torch.zeros(2, 4, dtype=I32), lengths=torch.zeros(2, dtype=I32, device="cuda"))):
        with pytest.raises(ValueError):
            uw.edit_logits(x, 2, 64, x, **kw)
    with pytest.raises(ValueError):
        uw.edit_logits(x, 3, 64, x)
    with pytest.raises(ValueError):
        uw.edit_logits(x, 2, 65, x)
    with pytest.raises(ValueError):
        uw.edit_logits(x, 2, 64, x.bfloat16())
