"""Token log probabilities, entropies and top tokens against 64 bits; token ids exactly.

Tolerance: a thread adds at most vocab / 512 + 8 powers in sequence and a tree of 13 joins follows, each off by 2^-24, and
each power is off by 2^-22 plus 2^-23 of its argument's magnitude |z - m| (which its own smallness outweighs: at most 1 on
average over the distribution, entropy-like).  The logarithm and the differences add 2^-23 of their values.  So with
r = (vocab / 512 + 40) 2^-24 + 2^-20 a log probability is within r + 2^-21 |lp| and an entropy, whose second term is a
quotient of two such sums, within 2 r (1 + entropy)."""
import numpy as np
import pytest

import lossless_bf16_weight_exponent_gb300 as uw

pytestmark = pytest.mark.gpu


def torch():
    import torch as t
    return t


def run(x, targets=None, n=0, ld=0, vocab=None, T=1.0, entropy=True, stream=None):
    """x: tensor on the host; returns lp, entropy, ids, top_lp as numpy."""
    t = torch()
    xd = x.cuda()
    R, V = x.shape[0], vocab or x.shape[1]
    lp = t.full((R,), 7.0, device="cuda") if targets is not None else None
    H = t.full((R,), 7.0, device="cuda") if entropy else None
    ids = t.full((R, n), -7, dtype=t.int32, device="cuda") if n else None
    top = t.full((R, n), 7.0, device="cuda") if n else None
    tg = t.as_tensor(targets, dtype=t.int32).cuda() if targets is not None else None
    if stream is not None:
        stream.wait_stream(t.cuda.current_stream())
    uw.token_logprobs(xd, R, V, lp, tg, H, n, ids, top, uw.OUT_BF16 if x.dtype == t.bfloat16 else uw.OUT_F32, ld, T, stream)
    t.cuda.synchronize()
    return [None if v is None else v.cpu().numpy() for v in (lp, H, ids, top)]


def plain(x, targets, n, T):
    """x: float64 [R, V]"""
    z = x / T
    with np.errstate(invalid="ignore", divide="ignore"):
        m = z.max(1, keepdims=True)
        e = np.exp(z - np.where(np.isneginf(m), 0, m))
        s = e.sum(1, keepdims=True)
        logp = np.where(s == 0, -np.inf, z - m - np.log(s))
        H = -np.where(e > 0, e / s * logp, 0).sum(1)
    lp = None
    if targets is not None:
        tg = np.asarray(targets)
        lp = np.where(tg < 0, 0, np.where(tg >= x.shape[1], np.nan, logp[np.arange(len(tg)), np.clip(tg, 0, x.shape[1] - 1)]))
    order = np.argsort(-x, axis=1, kind="stable")[:, :n]
    return lp, H, order, np.take_along_axis(logp, order, 1)


def check(got, want, V):
    r = (V / 512 + 40) * 2.0 ** -24 + 2.0 ** -20
    for g, w in ((got[0], want[0]), (got[3], want[3] if got[3] is not None else None)):
        if g is None:
            continue
        fin = np.isfinite(w)
        assert np.array_equal(g[~fin], w[~fin], equal_nan=True)
        err = np.abs(g[fin] - w[fin])
        assert (err <= r + 2.0 ** -21 * np.abs(w[fin])).all(), err.max()
    if got[1] is not None:
        assert (np.abs(got[1] - want[1]) <= 2 * r * (1 + want[1])).all(), np.abs(got[1] - want[1]).max()
    if got[2] is not None:
        assert np.array_equal(got[2], want[2])


def logits(R, V, seed, bf16=False, scale=3.0):
    t = torch()
    x = t.randn(R, V, generator=t.Generator().manual_seed(seed)) * scale
    return x.bfloat16() if bf16 else x


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [0, 1, 5, 32])
@pytest.mark.parametrize("R,V", [(1, 32), (2, 33), (3, 517), (1, 5000), (7, 32003), (1, 128256), (400, 1001), (160, 9000)])
def test_logprobs(R, V, n, bf16):
    x = logits(R, V, R + V + n, bf16)
    tg = np.random.default_rng(V).integers(0, V, R)
    check(run(x, tg, n, T=0.7), plain(x.double().numpy(), tg, n, 0.7), V)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows", ["ordinary", "rising", "few_values"])
def test_long_lists_in_many_rows(rows, bf16):
    R, V, n = 650, 20011, 32
    x = logits(R, V, 9, bf16)
    if rows == "rising":  # the first part's bound is below most of what follows
        x = (x.float() + torch().linspace(0, 40, V)).to(x.dtype)
    elif rows == "few_values":  # many equal logits at the bound
        x = x.round()
    tg = np.random.default_rng(V).integers(0, V, R)
    check(run(x, tg, n, T=1.0), plain(x.double().numpy(), tg, n, 1.0), V)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V,ld,shift", [(1, 1, 0), (5, 7, 1), (1000, 1003, 3), (4097, 4099, 0), (30001, 30017, 1)])
def test_unaligned_rows(V, ld, shift, bf16):
    # rows begin at any element; what lies between them is not read as part of one
    t = torch()
    buf = t.full((4 * ld + shift,), 60.0).to(t.bfloat16 if bf16 else t.float32)
    x = logits(4, V, V, bf16)
    for r in range(4):
        buf[shift + r * ld:shift + r * ld + V] = x[r]
    d = buf.cuda()
    lp, H, n = t.empty(4, device="cuda"), t.empty(4, device="cuda"), min(V, 9)
    ids, top = t.empty(4, n, dtype=t.int32, device="cuda"), t.empty(4, n, device="cuda")
    tg = np.array([0, V - 1, V // 2, V // 3])
    uw.token_logprobs(d[shift:], 4, V, lp, t.as_tensor(tg, dtype=t.int32).cuda(), H, n, ids, top, uw.OUT_BF16 if bf16 else uw.OUT_F32, ld)
    check([v.cpu().numpy() for v in (lp, H, ids, top)], plain(x.double().numpy(), tg, n, 1.0), V)


@pytest.mark.parametrize("V", [40, 3000, 70000])
def test_equal_logits_go_to_the_lower_index(V):
    t = torch()
    x = t.zeros(3, V)
    x[1] = t.randint(-2, 3, (V,), generator=t.Generator().manual_seed(1)).float()
    x[1][x[1] == 0] = -0.0
    x[1][V // 2:][x[1][V // 2:] == 0] = 0.0
    x[2] = -5.0
    x[2, -1] = 1.0
    check(run(x, [0, 1, 2], 32), plain(x.double().numpy(), [0, 1, 2], 32, 1.0), V)


@pytest.mark.parametrize("V", [50, 5000, 128256])
def test_masked_tokens(V):
    t = torch()
    x = logits(6, V, 9)
    keep = t.rand(6, V, generator=t.Generator().manual_seed(2)) < 0.02
    keep[:, 3] = True
    x[~keep] = -float("inf")
    x[2] = -float("inf")            # nothing is left
    x[3] = -float("inf")
    x[3, V - 1] = -2.0              # one token is
    x[4] = torch().finfo(t.float32).min  # the type's lowest value is not a mask
    tg = [3, 4, 0, V - 1, 5, 3]
    got = run(x, tg, 8)
    check(got, plain(x.double().numpy(), tg, 8, 1.0), V)
    assert np.isneginf(got[0][2]) and got[1][2] == 0 and np.array_equal(got[2][2], np.arange(8))
    assert got[0][3] == 0 and got[1][3] == 0


def test_peaked_and_wide_distributions():
    V = 20000
    x = logits(4, V, 11)
    x[0, 77] = 5000.0   # everything else underflows
    x[1] *= 300
    x[2] -= 30000.0     # far from zero
    x[3] *= 1e-6        # nearly uniform: the entropy is near log V
    check(run(x, [77, 5, 6, 7], 4), plain(x.double().numpy(), [77, 5, 6, 7], 4, 1.0), V)


@pytest.mark.parametrize("V", [60, 40000])
def test_nan_and_infinity_stay_in_their_row(V):
    x = logits(5, V, 13)
    x[1, 0], x[1, 20], x[3, 9] = float("nan"), float("inf"), float("inf")
    got = run(x, [1] * 5, 3)
    ok = [0, 2, 4]
    check([g[ok] for g in got], plain(x.double().numpy()[ok], [1] * 3, 3, 1.0), V)
    assert np.isnan(got[0][[1, 3]]).all() and np.isnan(got[1][[1, 3]]).all() and np.isnan(got[3][[1, 3]]).all()
    order = np.argsort(-x[1].numpy()[1:], kind="stable") + 1
    assert list(got[2][1][:2]) == [0, 20] and got[2][3][0] == 9 and got[2][1][2] == order[1]


def test_targets_outside_the_vocabulary():
    x = logits(4, 300, 15)
    got = run(x, [-1, -100, 300, 2 ** 31 - 1])
    assert (got[0][:2] == 0).all() and np.isnan(got[0][2:]).all()


def test_parts_streams_and_repeats():
    t = torch()
    x = logits(3, 50000, 17)
    want = plain(x.double().numpy(), [1, 2, 3], 6, 2.0)
    a = run(x, [1, 2, 3], 6, T=2.0, stream=t.cuda.Stream())
    check(a, want, 50000)
    check(run(x, None, 6, T=2.0, entropy=False), want, 50000)
    check(run(x, [1, 2, 3], 0, T=2.0, entropy=False), want, 50000)
    b = run(x, [1, 2, 3], 6, T=2.0)
    assert all(np.array_equal(p, q) for p, q in zip(a, b))


def test_rows_beyond_32_bit_offsets():
    t = torch()
    R, V = 34000, 128256  # 4.4e9 logits of 2 bytes
    x = t.zeros(R, V, dtype=t.bfloat16, device="cuda")
    x[-1, 5], x[-1, V - 1], x[17000, 9] = 3.0, 2.0, 1.0
    ids, top = t.empty(R, 2, dtype=t.int32, device="cuda"), t.empty(R, 2, device="cuda")
    uw.token_logprobs(x, R, V, n_top=2, top_ids=ids, top_logprobs=top, dtype=uw.OUT_BF16)
    assert ids[-1].tolist() == [5, V - 1] and ids[17000].tolist() == [9, 0] and ids[16999].tolist() == [0, 1]


def test_refusals():
    t = torch()
    x, o, i = t.zeros(2, 100, device="cuda"), t.zeros(64, device="cuda"), t.zeros(64, dtype=t.int32, device="cuda")

    def status(logits=x, rows=2, vocab=100, **k):
        with pytest.raises(uw.UwError) as e:
            uw.token_logprobs(logits, rows, vocab, **k)
        return e.value.status

    assert status(logprob=o) == status(targets=i) == uw.ERR_INVALID_ARG
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert status(entropy=o, temperature=T) == uw.ERR_INVALID_ARG
    assert status(n_top=33, top_ids=i, top_logprobs=o) == status(n_top=-1) == status(n_top=3) == uw.ERR_INVALID_ARG
    assert status(vocab=4, n_top=5, top_ids=i, top_logprobs=o) == uw.ERR_INVALID_ARG
    assert status(entropy=o, dtype=9) == status(logits=x.data_ptr() + 2, entropy=o) == status(logits=None, entropy=o) == uw.ERR_INVALID_ARG
    assert status(vocab=0, entropy=o) == status(vocab=2 ** 24 + 1, entropy=o) == status(entropy=o, ld=99) == status(rows=-1, entropy=o) == uw.ERR_SHAPE


def test_clusters_behind_one_another():
    # Few rows: the CTAs of a row exchange their parts through each other's shared memory.  Calls of one, two, four and
    # eight CTAs a row follow each other without a wait, so that CTAs begin while others end.
    t = torch()
    V, n = 40000, 4
    xs = [logits(R, V, 100 + R) for R in (1, 2, 40, 70, 140, 3)]
    dev, outs = [x.cuda() for x in xs], []
    for _ in range(20):
        for x in dev:
            R = x.shape[0]
            H, ids, top = t.empty(R, device="cuda"), t.empty(R, n, dtype=t.int32, device="cuda"), t.empty(R, n, device="cuda")
            uw.token_logprobs(x, R, V, None, None, H, n, ids, top)
            outs.append((H, ids, top))
    t.cuda.synchronize()
    for i, x in enumerate(xs):
        want = plain(x.double().numpy(), None, n, 1.0)
        for H, ids, top in outs[i::len(xs)]:
            check([None, H.cpu().numpy(), ids.cpu().numpy(), top.cpu().numpy()], want, V)


def as_f32(want):
    with np.errstate(over="ignore"):
        return [None if w is None else w if w.dtype.kind == "i" else w.astype(np.float32) for w in want]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [1.0, 4.0])
@pytest.mark.parametrize("V", [60, 20000, 70000])
def test_logits_of_the_types_largest_value(V, T, bf16):
    # finite logits over the type's whole range, beside masked tokens: differences to the maximum may be past the range
    t = torch()
    x = logits(5, V, 21, bf16)
    big = t.finfo(x.dtype).max
    x[0, 7] = big                                     # one forced token
    x[1, 7], x[1, 9:40] = big, -float("inf")
    x[2, 3:5], x[2, 20:30] = big, -big                # two of them, and the lowest
    x[3] = -float("inf")
    x[3, 5], x[3, 11], x[3, V - 1] = big, -big, -1.5e37
    x[4], x[4, 12] = -1.5e37, -1e36
    for tg in ([7, 7, 4, 5, 12], [3, 8, 20, 11, 13], [0, 10, 0, V - 1, 0]):
        check(run(x, tg, 6, T=T), as_f32(plain(x.double().numpy(), tg, 6, T)), V)


@pytest.mark.parametrize("T", [1e-30, 1e10, 1e30, 1e36, 3e38])
@pytest.mark.parametrize("V", [60, 20000])
def test_temperatures_far_from_one(V, T):
    t = torch()
    x = logits(4, V, 23) * max(1.0, min(T, 1e37)) if T > 1 else logits(4, V, 23) * T
    x[1, 5:50] = -float("inf")
    x[2, ::3] = t.finfo(t.float32).min
    x[3, 1:] = -float("inf")
    T = float(np.float32(T))
    tg = [2, 3, 4, 0]
    check(run(x, tg, 4, T=T), as_f32(plain(x.double().numpy(), tg, 4, T)), V)


@pytest.mark.parametrize("rest", [-float("inf"), -2e38])
@pytest.mark.parametrize("special", [float("nan"), float("inf")])
def test_masked_tokens_behind_a_nan_or_infinity_go_by_index(special, rest):
    # few rows: a row is several CTAs', and only one of them sees the NaN or infinity
    x = torch().full((2, 40000), rest)
    x[0, 30000] = special
    x[1, 30000], x[1, 39999] = special, -2.0
    got = run(x, None, 5)
    assert got[2].tolist() == [[30000, 0, 1, 2, 3], [30000, 39999, 0, 1, 2]]
