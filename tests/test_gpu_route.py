"""The router against a plain one in 64 bits: experts, order and ranks exactly (equal logits by the lower index), weights
within 1e-5 relative (two exponentials and a division of a few 2^-23 each, arguments up to 30 rounded to 2^-24, sums of
at most 32 + 5 steps of 2^-24)."""
import numpy as np
import pytest

import lossless_bf16_weight_exponent_gb300 as uw

pytestmark = pytest.mark.gpu


def torch():
    import torch as t
    return t


def plain(z, k, score, bias, renorm, scale):
    """ids, weights, offsets, row_src, pos; z fp32 [T, E]."""
    T, E = z.shape
    key = z if bias is None else (z + bias).astype(np.float32)
    ids = np.argsort(-key.astype(np.float64), axis=1, kind="stable")[:, :k]
    zd = z.astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        if score == uw.SCORE_SOFTMAX:
            m = zd.max(1, keepdims=True)
            e = np.exp(zd - np.where(np.isneginf(m), 0, m))
            s = e.sum(1, keepdims=True)
            p = np.where(s == 0, 0, e / np.where(s == 0, 1, s))
        else:
            p = 1 / (1 + np.exp(-zd))
    w = np.take_along_axis(p, ids, 1)
    if renorm:
        s = w.sum(1, keepdims=True)
        w = np.where(s == 0, 0, w / np.where(s == 0, 1, s))
    flat = ids.reshape(-1)
    rows = np.argsort(flat, kind="stable")
    pos = np.empty(T * k, np.int64)
    pos[rows] = np.arange(T * k)
    offsets = np.searchsorted(flat[rows], np.arange(E + 1))
    return ids, w * scale, offsets, rows // k, pos.reshape(T, k)


def run(z, k, score=uw.SCORE_SOFTMAX, bias=None, renorm=True, scale=1.0, bf16=False, ld=0, stream=None):
    t = torch()
    T, E = z.shape[0], (z.shape[1] if not ld else None)
    return _run(t.from_numpy(np.ascontiguousarray(z)).cuda(), T, E, k, score, bias, renorm, scale, bf16, ld, stream)


def _run(zd, T, E, k, score, bias, renorm, scale, bf16, ld, stream=None):
    t = torch()
    i32 = lambda *s: t.full(s, -7, dtype=t.int32, device="cuda")  # noqa: E731
    ids, src, pos, off = i32(T, k), i32(T * k), i32(T, k), i32(E + 1)
    w = t.full((T, k), float("nan"), device="cuda")
    r = uw.Router(E, k, score, None if bias is None else t.from_numpy(bias).cuda(), renorm, scale)
    n = r.workspace_size(T)
    ws = t.full((max(n, 16),), 0xEE, dtype=t.uint8, device="cuda")  # needs no initialisation
    r.route(zd, T, ids, w, off, src, pos, uw.OUT_BF16 if bf16 else uw.OUT_F32, ld, ws, n, stream)
    t.cuda.synchronize()
    return [v.cpu().numpy() for v in (ids, w, off, src, pos)]


def check(got, want):
    for i in (0, 2, 3, 4):
        assert np.array_equal(got[i], want[i]), i
    assert np.allclose(got[1], want[1], rtol=1e-5, atol=1e-37, equal_nan=True)


@pytest.mark.parametrize("score", [uw.SCORE_SOFTMAX, uw.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm,biased", [(True, False), (False, True)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 33, 2), (127, 8, 8), (128, 100, 4), (129, 128, 8), (1000, 257, 16), (2500, 64, 6),
                                   (300, 1024, 16)])
def test_route(T, E, k, renorm, biased, score):
    rng = np.random.default_rng(T + E)
    z = (rng.standard_normal((T, E)) * 3).astype(np.float32)
    b = rng.standard_normal(E).astype(np.float32) if biased else None
    check(run(z, k, score, b, renorm, 2.5), plain(z, k, score, b, renorm, 2.5))


@pytest.mark.parametrize("T", [50, 700])
def test_equal_logits_go_to_the_lower_index(T):
    rng = np.random.default_rng(T)
    z = rng.integers(-1, 2, (T, 40)).astype(np.float32)  # many ties, among them -0 and +0
    z[z == 0] = np.where(rng.random((z == 0).sum()) < 0.5, -0.0, 0.0)
    check(run(z, 8), plain(z, 8, uw.SCORE_SOFTMAX, None, True, 1.0))
    z[:] = 4.0
    check(run(z, 8), plain(z, 8, uw.SCORE_SOFTMAX, None, True, 1.0))  # every token takes experts 0..7


@pytest.mark.parametrize("T,E,k", [(60, 100, 8), (300, 256, 16), (40, 1000, 16)])
@pytest.mark.parametrize("values", [2, 30, 1000])
def test_equal_logits_among_many_experts(T, E, k, values):
    rng = np.random.default_rng(E + values)
    z = rng.integers(0, values, (T, E)).astype(np.float32)  # a few equal keys at the bound, or more than a warp can hold
    z[0, 5:] = -np.inf
    z[1] = -np.inf
    check(run(z, k), plain(z, k, uw.SCORE_SOFTMAX, None, True, 1.0))


@pytest.mark.parametrize("T,E,k", [(2049, 1024, 3), (8200, 256, 8), (65000, 33, 2)])
def test_counts_added_up_by_the_scan(T, E, k):
    rng = np.random.default_rng(T)
    z = (rng.standard_normal((T, E)) + 2 * rng.standard_normal(E)).astype(np.float32)
    check(run(z, k), plain(z, k, uw.SCORE_SOFTMAX, None, True, 1.0))


def test_masked_experts_and_non_finite_logits():
    rng = np.random.default_rng(3)
    z = rng.standard_normal((200, 32)).astype(np.float32)
    z[:, 5:] = -np.inf                      # three tokens' worth of experts fewer than k
    z[10] = -np.inf                         # nothing is left
    z[11] = np.finfo(np.float32).min        # the type's lowest value everywhere
    got, want = run(z, 8), plain(z, 8, uw.SCORE_SOFTMAX, None, True, 1.0)
    check(got, want)
    assert (got[1][10] == 0).all() and np.allclose(got[1][11], 0.125)
    z[12, 3] = np.nan
    got = run(z, 8)
    assert got[0][12, 0] == 3 and np.isnan(got[1][12]).all()
    assert np.array_equal(np.sort(got[4].ravel()), np.arange(1600))  # the rows are a permutation all the same
    assert np.isfinite(got[1][np.arange(200) != 12]).all()


@pytest.mark.parametrize("T", [5, 400])
def test_bf16_logits_stride_stream_and_repeat(T):
    t = torch()
    E, k, ld = 60, 4, 72
    z = t.randn(T, ld, generator=t.Generator().manual_seed(1)).bfloat16()
    want = plain(z[:, :E].float().numpy(), k, uw.SCORE_SIGMOID, None, True, 1.0)
    s = t.cuda.Stream()
    zd = z.cuda()
    s.wait_stream(t.cuda.current_stream())
    got = _run(zd, T, E, k, uw.SCORE_SIGMOID, None, True, 1.0, True, ld, s)
    check(got, want)
    again = _run(zd, T, E, k, uw.SCORE_SIGMOID, None, True, 1.0, True, ld)
    assert all(np.array_equal(a, b) for a, b in zip(got, again))


def test_no_tokens_leave_empty_experts():
    t = torch()
    got = _run(t.empty(0, 9, device="cuda"), 0, 9, 2, uw.SCORE_SOFTMAX, None, True, 1.0, False, 0)
    assert np.array_equal(got[2], np.zeros(10, np.int32))


def test_refusals():
    t = torch()
    z = t.zeros(200, 16, device="cuda")
    o = [t.empty(4000, dtype=t.int32, device="cuda") for _ in range(5)]
    ws = t.empty(4096, dtype=t.uint8, device="cuda")

    def status(E=16, k=2, tokens=200, score=0, dtype=uw.OUT_F32, ld=0, outs=o, w=ws, n=4096, logits=z):
        with pytest.raises(uw.UwError) as e:
            uw.Router(E, k, score).route(logits, tokens, *outs, dtype, ld, w, n)
        return e.value.status

    assert status(E=0) == status(E=1025) == status(k=0) == status(k=17) == status(E=4, k=5) == status(score=2) == uw.ERR_INVALID_ARG
    assert status(dtype=3) == uw.ERR_INVALID_ARG
    assert status(tokens=-1) == status(ld=8) == status(tokens=2 ** 30) == uw.ERR_SHAPE
    assert status(n=16) == status(w=None) == uw.ERR_WORKSPACE
    assert status(outs=[None] + o[1:]) == status(outs=o[:4] + [None]) == status(logits=None) == uw.ERR_INVALID_ARG
    assert status(logits=z.data_ptr() + 2) == status(w=ws.data_ptr() + 4) == uw.ERR_INVALID_ARG


@pytest.mark.parametrize("score", [uw.SCORE_SOFTMAX, uw.SCORE_SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 3, 1), (7, 33, 2), (100, 64, 8), (129, 128, 8), (700, 257, 16), (2500, 40, 6), (300, 1024, 4)])
def test_choice_by_score(T, E, k, biased, score):
    # A score is within 2^-21 of its value (an exponential, a sum of at most 40 steps, a division), its sum with the bias off by half
    # a unit in the last place of it: experts whose exact keys differ by less may come in either order.
    rng = np.random.default_rng(T + E)
    z = (rng.standard_normal((T, E)) * 3).astype(np.float32)
    b = (rng.standard_normal(E) * 0.5).astype(np.float32) if biased else None
    got = run(z, k, score + uw.SCORE_CHOOSES, b, True, 1.5)
    zd = z.astype(np.float64)
    p = 1 / (1 + np.exp(-zd)) if score == uw.SCORE_SIGMOID else np.exp(zd - zd.max(1, keepdims=True))
    if score == uw.SCORE_SOFTMAX:
        p /= p.sum(1, keepdims=True)
    key = p + b if biased else p
    slack = 2.0 ** -21 + 2.0 ** -23 * np.abs(key).max()
    ids = got[0]
    chosen = np.take_along_axis(key, ids, 1)
    assert (np.sort(ids, 1)[:, 1:] != np.sort(ids, 1)[:, :-1]).all()
    assert (chosen[:, 1:] <= chosen[:, :-1] + slack).all()
    left = key.copy()
    np.put_along_axis(left, ids, -np.inf, 1)
    assert (left.max(1) <= chosen[:, -1] + slack).all()
    # the rest follows from the experts chosen
    w = np.take_along_axis(p, ids, 1)
    flat = ids.reshape(-1)
    rows = np.argsort(flat, kind="stable")
    pos = np.empty(T * k, np.int64)
    pos[rows] = np.arange(T * k)
    check(got, (ids, 1.5 * w / w.sum(1, keepdims=True), np.searchsorted(flat[rows], np.arange(E + 1)), rows // k, pos.reshape(T, k)))


def test_choice_by_score_is_not_that_by_logit():
    z, b = np.array([[4.0, 8.0, -1.0]], np.float32), np.array([0.125, 0.0, 0.0], np.float32)
    # sigmoid(4) + 0.125 > sigmoid(8), while 4 + 0.125 < 8
    assert run(z, 1, uw.SCORE_SIGMOID, b)[0].tolist() == [[1]]
    got = run(z, 1, uw.SCORE_SIGMOID + uw.SCORE_CHOOSES, b, renorm=False)
    assert got[0].tolist() == [[0]] and abs(got[1][0, 0] - 1 / (1 + np.exp(-4.0))) < 1e-6  # the bias is not in the weight


@pytest.mark.parametrize("score", [uw.SCORE_SOFTMAX, uw.SCORE_SIGMOID])
def test_choice_by_score_of_masked_and_nan_logits(score):
    z = np.full((200, 70), -np.inf, np.float32)
    z[1, 40] = 0.0
    z[2, 9] = np.nan
    b = np.linspace(0, 0.01, 70, dtype=np.float32)
    got = run(z, 3, score + uw.SCORE_CHOOSES, b, True)
    assert got[0][0].tolist() == [69, 68, 67] and (got[1][0] == 0).all()  # nothing but the bias is left
    assert got[0][1].tolist() == [40, 69, 68] and got[1][1].tolist() == [1, 0, 0]
    assert got[0][2, 0] == (9 if score == uw.SCORE_SIGMOID else 0) and np.isnan(got[1][2, 0])  # a softmax is a NaN everywhere
    assert np.array_equal(np.sort(got[4].ravel()), np.arange(600))
