"""Keys and values appended to a paged cache, and attention over it, against plain forms in 64 bits.

Append: an element is a cos - b sin with cos and sin within 2^-22 (the reduced angle is within 2^-23 of a turn's pi, sincospi
within two units) and three fp32 operations, so within 1e-6 (|a| + |b|) of the exact one, and rounded to bf16 once: 2^-8
of the value.

Attention: a score is a sum of D products in fp32, in an order and with a truncation of the tensor core's, within
(D + 2) 2^-22 of the sum of their magnitudes A; its power's error is as much (relative), and 2^-21 for the power itself.  A
probability is rounded to bf16, 2^-8 of it at most; the sums over n keys in fp32 add n 2^-23.  So an output is within
(2^-8 + 2 e) sum_j p_j |v_j| with e = (D + 2) 2^-22 A + 2^-21 + n 2^-23, and 2^-8 of itself for its own rounding; the logarithm of the sum
is within e + 2^-22 |lse|."""
import math

import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw

pytestmark = pytest.mark.gpu
F32, BF16, I32, F64 = torch.float32, torch.bfloat16, torch.int32, torch.float64


def batch_of(new, past, page, seed=0, spare=3, garbage=float("nan"), H=2, D=128, heads_first=False, max_pages=None, starts_at=0):
    """A cache whose sequences' slots hold numbers and all others `garbage`, the batch, and k and v of each sequence [len, H, D]."""
    g = torch.Generator().manual_seed(seed + 7 * sum(new) + sum(past))
    S = len(new)
    lens = [a + b for a, b in zip(new, past)]
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    shape = (pages, H, page, D) if heads_first else (pages, page, H, D)
    caches = [torch.full(shape, garbage, dtype=BF16) for _ in range(2)]
    views = [c.transpose(1, 2) if heads_first else c for c in caches]
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((S, max_pages or max(1, max(held))), -7, dtype=I32)
    seqs, at = [], 0
    for s in range(S):
        mine = order[at:at + held[s]]
        at += held[s]
        table[s, :held[s]] = torch.tensor(mine, dtype=I32)
        kv = [torch.randn(lens[s], H, D, generator=g).to(BF16) for _ in range(2)]
        for p, i in enumerate(mine):
            for c, x in zip(views, kv):
                part = x[p * page:(p + 1) * page]
                c[i, :part.shape[0]] = part
        seqs.append(kv)
    starts = [starts_at]
    for n in new:
        starts.append(starts[-1] + n)
    dev = [c.cuda() for c in caches]
    k, v = [c.transpose(1, 2) if heads_first else c for c in dev]
    dt = dict(starts=torch.tensor(starts, dtype=I32).cuda(), lengths=torch.tensor(lens, dtype=I32).cuda(), table=table.cuda())
    return dict(k=k, v=v, seqs=seqs, batch=uw.KVBatch(dt["starts"], dt["lengths"], dt["table"]), cache=uw.KVCache(k, v), g=g, at=starts, **dt)


# ------------------------------------------------------------------------------------------------ attention
def plain_attend(q, k, v, n, scale, causal, window):
    """q [n, Hq, D] against k, v [len, H, D], in 64 bits: out, lse and their bounds."""
    L, H, D = k.shape
    Hq = q.shape[1]
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    k, v = k.repeat_interleave(Hq // H, 1), v.repeat_interleave(Hq // H, 1)
    z = torch.einsum("nhd,lhd->hnl", q, k) * scale
    A = torch.einsum("nhd,lhd->hnl", q.abs(), k.abs()) * abs(scale)
    pos, key = torch.arange(L - n, L)[:, None], torch.arange(L)[None]
    see = torch.ones(n, L, dtype=torch.bool)
    if causal:
        see = key <= pos
        if window:
            see &= pos - key < window
    z = z.masked_fill(~see, -math.inf)
    none = ~see.any(1)
    lse = torch.logsumexp(z, 2) if L else torch.full((Hq, n), -math.inf, dtype=F64)
    p = torch.where(see, torch.exp(z - lse.masked_fill(none, 0.0)[..., None]), 0.0)
    out = torch.einsum("hnl,lhd->nhd", p, v)
    mag = torch.einsum("hnl,lhd->nhd", p, v.abs())
    e = (D + 2) * 2.0 ** -22 * torch.where(see, A, 0.0).amax(2) + 2.0 ** -21 + L * 2.0 ** -23 if L else torch.zeros(Hq, n, dtype=F64)
    bound = (2.0 ** -8 + 2 * e.t()[..., None]) * mag + 2.0 ** -8 * out.abs() + 1e-30
    return out, lse.t(), bound, (e + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)).t() + 1e-6


def attend(c, q, Hq, causal=True, window=0, scale=None, rows=None, out=None, lse=True, ws=None, stream=None):
    rows = q.shape[0] if rows is None else rows
    out = torch.full_like(q, 7.0) if out is None else out
    l = torch.full((max(1, q.shape[0]), Hq), 7.0, device="cuda") if lse else None
    need = c["cache"].workspace_size(c["batch"], rows, Hq)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if ws is None else ws
    c["cache"].attend(c["batch"], rows, q, out, scale=scale, causal=causal, window=window, lse=l, workspace=ws, ws_bytes=need, stream=stream)
    c["cache"].check(stream=stream)
    return out, l


def check_attend(c, q, out, lse, new, causal=True, window=0, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    for s, n in enumerate(new):
        if not n:
            continue
        a = c["at"][s]
        ref, rl, b, bl = plain_attend(q[a:a + n].cpu(), *c["seqs"][s], n, scale, causal, window)
        d = (out[a:a + n].cpu().to(F64) - ref).abs()
        assert (d <= b).all(), (s, float((d / b).max()))
        if lse is not None:
            got = lse[a:a + n].cpu().to(F64)
            dead = torch.isinf(rl)
            assert (got[dead] == -math.inf).all()
            assert ((got - rl).abs()[~dead] <= bl[~dead]).all(), s


CASES = [
    # new, past, Hq, H, D, page, heads_first, causal, window
    ([1], [0], 4, 1, 128, 16, False, True, 0),
    ([1], [1], 8, 8, 64, 8, True, True, 0),
    ([1], [127], 32, 8, 128, 64, False, True, 0),
    ([1], [128], 32, 8, 128, 64, False, True, 0),
    ([1] * 5, [0, 15, 16, 17, 1000], 8, 2, 128, 16, False, True, 0),
    ([1, 0, 1, 0, 0], [300, 50, 0, 0, 2000], 4, 4, 64, 32, True, True, 0),
    ([4], [5000], 16, 2, 128, 128, True, True, 0),
    ([3, 5], [700, 11], 6, 2, 64, 24, False, True, 0),
    ([7], [260], 7, 1, 128, 40, False, True, 0),
    ([17, 1, 130], [3, 900, 0], 8, 2, 128, 64, False, True, 0),
    ([200], [0], 10, 2, 128, 64, True, True, 0),
    ([257], [513], 4, 1, 64, 256, False, True, 0),
    ([40, 9], [100, 600], 16, 4, 128, 16, False, False, 0),
    ([65], [200], 8, 2, 128, 64, False, True, 1),
    ([65, 1, 3], [400, 1000, 0], 8, 2, 128, 16, False, True, 33),
    ([300], [300], 8, 2, 64, 32, True, True, 129),
    ([2], [64], 64, 1, 128, 16, False, True, 0),
    ([1] * 300, [(7 * i) % 61 for i in range(300)], 4, 2, 64, 16, False, True, 0),
    ([600, 300], [0, 77], 8, 2, 128, 48, False, True, 0),
    ([520], [130], 12, 4, 64, 64, False, False, 0),
    ([385], [1000], 24, 8, 128, 128, True, True, 500),
    ([1, 700, 1, 1, 90], [3000, 0, 128, 5, 1000], 32, 4, 64, 32, False, True, 256),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attend(case):
    new, past, Hq, H, D, page, hf, causal, window = case
    c = batch_of(new, past, page, H=H, D=D, heads_first=hf)
    q = (torch.randn(sum(new), Hq, D, generator=c["g"]) * 1.5).to(BF16).cuda()
    out, lse = attend(c, q, Hq, causal, window)
    check_attend(c, q, out, lse, new, causal, window)


@pytest.mark.parametrize("case", [
    ([9, 2, 5], [700, 64, 0], 12, 3, 64, 16, False, True, 0),
    ([4, 4, 4], [30000, 200, 3], 32, 4, 128, 64, True, True, 0),
    ([5, 3, 0, 5], [1000, 90, 4, 2000], 20, 4, 128, 16, False, True, 70),
    ([6, 1], [300, 1], 8, 1, 64, 8, False, False, 0),
    ([2] * 80, [(37 * i) % 700 for i in range(80)], 16, 1, 128, 32, False, True, 0)], ids=str)
def test_attend_up_to_32_rows(case):
    new, past, Hq, H, D, page, hf, causal, window = case
    c = batch_of(new, past, page, H=H, D=D, heads_first=hf)
    q = (torch.randn(sum(new), Hq, D, generator=c["g"]) * 1.5).to(BF16).cuda()
    out, lse = attend(c, q, Hq, causal, window)
    check_attend(c, q, out, lse, new, causal, window)


def test_attend_long_split():
    """One sequence over all CTAs, and a batch whose items are cut in many places."""
    for new, past, Hq, H in (([1], [40000], 8, 1), ([2, 1, 1], [9000, 20000, 3], 8, 2)):
        c = batch_of(new, past, 64, H=H, D=128)
        q = (torch.randn(sum(new), Hq, 128, generator=c["g"]) * 3).to(BF16).cuda()
        out, lse = attend(c, q, Hq)
        check_attend(c, q, out, lse, new)


@pytest.mark.parametrize("S,most,H", [(64, 500, 8), (200, 900, 4), (500, 40, 8), (150, 3000, 2)])
def test_attend_many_sequences(S, most, H):
    """More ranges of work than CTAs, some of them shorter than a CTA's copies reach ahead."""
    new, past = [1 + i % 2 for i in range(S)], [(i * 7919) % most for i in range(S)]
    c = batch_of(new, past, 16, H=H, D=64)
    q = torch.randn(sum(new), 4 * H, 64, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, 4 * H)
    check_attend(c, q, out, lse, new)


@pytest.mark.parametrize("S,few,page", [(600, 1, 8), (600, 20, 16), (2500, 1, 16)])
def test_attend_more_sequences_than_the_small_plan_takes(S, few, page):
    """The first kernel's general form, one sequence with many tiles of rows among them, some that bring nothing."""
    new = [0 if i % 7 == 3 else few for i in range(S)]
    new[5] = 400
    past = [(i * 37) % 50 for i in range(S)]
    past[11] = 3000
    c = batch_of(new, past, page, H=1, D=64)
    q = torch.randn(sum(new), 2, 64, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, 2)
    check_attend(c, q, out, lse, new)


def test_attend_many_tiles_of_one_sequence():
    """More tiles of rows than the small form of the first kernel holds."""
    new, past = [600] * 7, [0, 5, 100, 0, 0, 9, 40]
    c = batch_of(new, past, 32, H=2, D=64)
    q = torch.randn(sum(new), 128, 64, generator=c["g"]).to(BF16).cuda()
    need = c["cache"].workspace_size(c["batch"], 4200, 128)
    assert need > 0
    out, lse = attend(c, q, 128)
    check_attend(c, q, out, lse, new)


def test_keys_and_values_in_one_tensor():
    kv = torch.randn(6, 2, 16, 2, 64, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    k, v = kv[:, 0], kv[:, 1]
    cache = uw.KVCache(k, v)
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    batch = uw.KVBatch(i32([0, 3]), i32([40]), i32([[4, 1, 2]]))
    g = torch.Generator().manual_seed(4)
    q, kn, vn = (torch.randn(3, n, 64, generator=g).to(BF16).cuda() for n in (4, 2, 2))
    was = kv.clone()
    cache.append(batch, 3, kn, vn)
    was[2, 0, 5:8], was[2, 1, 5:8] = kn, vn
    assert torch.equal(kv, was)
    out = torch.zeros_like(q)
    need = cache.workspace_size(batch, 3, 4)
    cache.attend(batch, 3, q, out, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"), ws_bytes=need)
    cache.check()
    kk, vv = (t[[4, 1, 2]].reshape(48, 2, 64)[:40].cpu() for t in (k, v))
    ref, _, b, _ = plain_attend(q.cpu(), kk, vv, 3, 0.125, True, 0)
    assert ((out.cpu().to(F64) - ref).abs() <= b).all()


def test_attend_peaked_scores():
    """Scores up to hundreds: the running maximum moves, probabilities underflow."""
    new, past = [5, 260], [900, 300]
    c = batch_of(new, past, 32, H=2, D=128)
    q = (torch.randn(sum(new), 8, 128, generator=c["g"]) * 40).to(BF16).cuda()
    out, lse = attend(c, q, 8)
    check_attend(c, q, out, lse, new)
    out, lse = attend(c, q, 8, scale=-0.05)
    check_attend(c, q, out, lse, new, scale=-0.05)
    out, lse = attend(c, q, 8, scale=0.0)
    check_attend(c, q, out, lse, new, scale=0.0)


@pytest.mark.parametrize("new,past", [([300], [0]), ([3], [0])])
def test_attend_rising_scores(new, past):
    """Every later key has a higher score, by much: each step moves the maximum."""
    c = batch_of(new, [700], 32, H=1, D=64)
    n = 700 + new[0]
    ramp = torch.linspace(-60, 60, n).to(BF16)
    k = torch.zeros(n, 1, 64, dtype=BF16)
    k[:, 0, 0] = ramp
    c["seqs"][0][0] = k
    for p, i in enumerate(c["table"][0].tolist()):
        part = k[p * 32:(p + 1) * 32].cuda()
        c["k"][i, :part.shape[0]] = part
    q = torch.zeros(new[0], 4, 64, dtype=BF16)
    q[:, 0::2, 0] = 8.0
    q[:, 1::2, 0] = -8.0
    q = q.cuda()
    out, lse = attend(c, q, 4)
    check_attend(c, q, out, lse, new)


@pytest.mark.parametrize("n", [9, 400])
def test_attend_rows_that_see_nothing(n):
    """A sequence that holds fewer tokens than it brings: the first rows have negative positions; and one that holds none."""
    c = batch_of([n, 2, 1], [0, 0, 30], 16, H=2, D=64)
    L = n - 5
    c["lengths"].copy_(torch.tensor([L, 0, 31], dtype=I32))
    q = torch.randn(n + 3, 4, 64, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, 4)
    assert (out[:5] == 0).all() and (lse[:5] == -math.inf).all() and (out[n:n + 2] == 0).all() and (lse[n:n + 2] == -math.inf).all()
    ref, rl, b, bl = plain_attend(q[5:n].cpu(), *[x[:L] for x in c["seqs"][0]], L, 0.125, True, 0)
    assert ((out[5:n].cpu().to(F64) - ref).abs() <= b).all() and ((lse[5:n].cpu().to(F64) - rl).abs() <= bl).all()
    out, lse = attend(c, q, 4, causal=False)
    assert (lse[:n] > -math.inf).all() and (out[n:n + 2] == 0).all()


@pytest.mark.parametrize("n,window", [(1, 40), (300, 100)])
def test_attend_pages_a_window_left(n, window):
    """Pages in front of the window are free: their entries are no pages, or hold anything."""
    page, past = 16, 1000
    c = batch_of([n], [past], page, H=2, D=128)
    q = torch.randn(n, 8, 128, generator=c["g"]).to(BF16).cuda()
    want, wl = attend(c, q, 8, window=window)
    check_attend(c, q, want, wl, [n], window=window)
    first = (past - window + 1) // page
    for p in c["table"][0, :first].tolist():
        c["k"][p], c["v"][p] = float("nan"), float("nan")
    edge = (past - window + 1) % page
    c["k"][c["table"][0, first], :edge] = float("inf")
    c["v"][c["table"][0, first], :edge] = float("nan")
    out, lse = attend(c, q, 8, window=window)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    c["table"][0, :first] = -1
    out, lse = attend(c, q, 8, window=window)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    c["table"][0, :first] = 2 ** 31 - 1
    out, lse = attend(c, q, 8, window=window)
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("n,H", [(3, 2), (20, 1), (300, 2)])
def test_attend_a_key_that_is_not_finite(n, H):
    """The rows that see it have no answer; those that do not have theirs."""
    c = batch_of([n], [70], 16, H=H, D=64)
    q = torch.randn(n, 4, 64, generator=c["g"]).to(BF16).cuda()
    at = 70 + n - 1                                  # the last token's key
    for bad in (float("nan"), float("inf")):
        c["k"][c["table"][0, at // 16].item(), at % 16] = bad
        out, lse = attend(c, q, 4)
        k, v = c["seqs"][0]
        ref, rl, b, bl = plain_attend(q[:n - 1].cpu(), k[:-1], v[:-1], n - 1, 0.125, True, 0)
        assert ((out[:n - 1].cpu().to(F64) - ref).abs() <= b).all() and ((lse[:n - 1].cpu().to(F64) - rl).abs() <= bl).all()
        if math.isnan(bad):
            assert torch.isnan(out[n - 1].float()).all() and torch.isnan(lse[n - 1]).all()


@pytest.mark.parametrize("n", [1, 300])
def test_attend_pages_outside_read_as_zeros(n):
    page, past = 32, 500
    c = batch_of([n], [past], page, H=2, D=64)
    q = torch.randn(n, 4, 64, generator=c["g"]).to(BF16).cuda()
    for i, bad in ((1, -5), (3, c["cache"].pages), (4, 2 ** 31 - 1), (5, -2 ** 31)):
        c["table"][0, i] = bad
        for x in c["seqs"][0]:
            x[i * page:(i + 1) * page] = 0
    out, lse = attend(c, q, 4)
    check_attend(c, q, out, lse, [n])


@pytest.mark.parametrize("n", [2, 200])
def test_attend_table_shorter_than_the_length(n):
    """A length that the table does not reach: keys up to its end."""
    c = batch_of([n], [600 - n], 32, H=1, D=64, max_pages=19)
    short = uw.KVBatch(c["starts"], c["lengths"], c["table"][:, :10])
    q = torch.randn(n, 4, 64, generator=c["g"]).to(BF16).cuda()
    c["batch"] = short
    out, lse = attend(c, q, 4)
    k, v = (x[:320] for x in c["seqs"][0])
    ref, rl, b, bl = plain_attend(q.cpu(), k, v, n, 0.125, False, 0)
    assert ((out.cpu().to(F64) - ref).abs() <= b).all() and ((lse.cpu().to(F64) - rl).abs() <= bl).all()


@pytest.mark.parametrize("n", [1, 150])
def test_attend_strides_and_rows_outside(n):
    """Columns of wider tensors, rows in front of and behind the sequences': those are left as they were."""
    new = [n, 2]
    c = batch_of(new, [100, 40], 16, H=2, D=128, starts_at=3)
    rows = n + 9
    wide = torch.randn(rows, 4 * 128 + 264, generator=c["g"]).to(BF16).cuda()
    q = wide[:, 256:256 + 512]
    big = torch.full((rows, 1000), 7.0, dtype=BF16, device="cuda")
    out = big[:, 8:8 + 512]
    lse = torch.full((rows, 4), 7.0, device="cuda")
    need = c["cache"].workspace_size(c["batch"], rows, 4)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    c["cache"].attend(c["batch"], rows, q, out, lse=lse, workspace=ws, ws_bytes=need)
    c["cache"].check()
    check_attend(c, q.reshape(rows, 4, 128), out.reshape(rows, 4, 128), lse, new)
    o = big.cpu()
    assert (o[:3] == 7).all() and (o[3 + n + 2:] == 7).all() and (o[:, :8] == 7).all() and (o[:, 520:] == 7).all()
    assert (lse[:3] == 7).all() and (lse[n + 5:] == 7).all()


@pytest.mark.parametrize("n", [1, 300])
def test_attend_starts_are_clamped(n):
    """Starts past the call's rows: nothing outside them is read or written."""
    c = batch_of([n, n], [50, 60], 16, H=1, D=64)
    q = torch.randn(2 * n, 2, 64, generator=c["g"]).to(BF16).cuda()
    out, lse = attend(c, q, 2, rows=n)
    check_attend(c, q, out, lse, [n, 0])
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    c["starts"].copy_(torch.tensor([-5, n, 2 ** 31 - 1], dtype=I32))
    out, lse = attend(c, q, 2)
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("new,past", [([1] * 9, [1000] * 9), ([300, 5], [100, 2000])])
def test_attend_same_bits_graphs_and_streams(new, past):
    c = batch_of(new, past, 16, H=2, D=128)
    q = torch.randn(sum(new), 8, 128, generator=c["g"]).to(BF16).cuda()
    want, wl = attend(c, q, 8)
    need = c["cache"].workspace_size(c["batch"], sum(new), 8)
    torch.cuda.synchronize()
    # two streams at once, a workspace each
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in streams]
    lses = [torch.zeros_like(wl) for _ in streams]
    wss = [torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, o, l, w in zip(streams, outs, lses, wss):
            c["cache"].attend(c["batch"], sum(new), q, o, lse=l, workspace=w, ws_bytes=need, stream=st)
    torch.cuda.synchronize()
    for o, l in zip(outs, lses):
        assert torch.equal(o, want) and torch.equal(l, wl)
    # a captured graph, replayed after the lengths changed; a second graph with the same workspace
    graphs, gouts = [], [torch.zeros_like(q) for _ in range(2)]
    side = torch.cuda.Stream()
    for o in gouts:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c["cache"].attend(c["batch"], sum(new), q, o, workspace=wss[0], ws_bytes=need)
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gouts[0], want) and torch.equal(gouts[1], want)
    c["lengths"] -= 7
    less, _ = attend(c, q, 8)
    assert not torch.equal(less, want)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gouts[0], less) and torch.equal(gouts[1], less)


# ------------------------------------------------------------------------------------------------ append
def turned(x, pos, dim, layout, freq, scale):
    """x [rows, heads, D] in 64 bits, the first dim elements turned by pos * freq; and the magnitudes that meet in an element."""
    x = x.to(F64)
    y, m = x.clone(), x.abs()
    ang = pos.to(F64)[:, None] * torch.from_numpy(freq)
    cs, sn = (torch.cos(ang) * scale)[:, None], (torch.sin(ang) * scale)[:, None]
    i = torch.arange(dim // 2)
    a, b = (i, i + dim // 2) if layout == uw.ROTARY_HALF else (2 * i, 2 * i + 1)
    y[..., a], y[..., b] = x[..., a] * cs - x[..., b] * sn, x[..., a] * sn + x[..., b] * cs
    m[..., a] = m[..., b] = (x[..., a].abs() + x[..., b].abs()) * scale
    return y, m


def close(got, ref, mag):
    d = (got.cpu().to(F64) - ref).abs()
    assert (d <= 2.0 ** -8 * ref.abs() + 1e-6 * mag + 1e-38).all(), float(d.max())


APPENDS = [
    # new, past, Hq, H, D, page, heads_first, dtype, rot, layout, scaling
    ([1], [0], 4, 1, 128, 16, False, F32, 128, 0, 0),
    ([1], [100000], 32, 8, 128, 64, False, F32, 128, 0, 3),
    ([1] * 70, [(13 * i) % 200 for i in range(70)], 8, 2, 64, 8, True, BF16, 64, 1, 0),
    ([300, 0, 17], [5, 9, 0], 8, 2, 128, 24, False, BF16, 64, 1, 4),
    ([33, 700], [1000, 3], 5, 5, 64, 64, True, F32, 32, 0, 2),
    ([2] * 40, [7] * 40, 64, 8, 128, 16, False, BF16, 16, 0, 1),
    ([2500], [30], 16, 4, 128, 32, False, BF16, 96, 0, 0),
]


def append_case(new, past, Hq, H, D, page, hf, dtype, rot, layout, scaling, starts_at=0, extra=0):
    c = batch_of(new, past, page, H=H, D=D, heads_first=hf, garbage=5.0, starts_at=starts_at)
    rows = starts_at + sum(new) + extra
    c["qkv"] = torch.randn(rows, (Hq + 2 * H) * D, generator=c["g"]).to(dtype).cuda()
    c["q"], c["kn"], c["vn"] = c["qkv"].view(rows, Hq + 2 * H, D).split([Hq, H, H], 1)
    args = dict(base=10000.0, scaling=scaling, factor=1.0 if scaling == 0 else 8.0, low=1.0, high=32.0 if scaling == 4 else 4.0, original=4096)
    c["rotary"] = uw.Rotary(rot, layout=layout, **args) if rot else None
    c["rot"], c["layout"] = rot, layout
    c["rows"], c["dt"] = rows, uw.OUT_F32 if dtype == F32 else uw.OUT_BF16
    return c


def cache_want(c, new, past, page, kref, kmag, vref, before, positions=None):
    """The cache after the append, where the new tokens stand in it, and the bounds' magnitudes."""
    k, v = (t.cpu().to(F64).clone() for t in before)
    mk = torch.zeros_like(k)
    hit = torch.zeros(k.shape[:2], dtype=torch.bool)
    for s, n in enumerate(new):
        for i in range(n):
            p, row = past[s] + i, c["at"][s] + i
            if p < 0 or p // page >= c["table"].shape[1]:
                continue
            pg = int(c["table"][s, p // page])
            if not 0 <= pg < c["cache"].pages:
                continue
            k[pg, p % page], v[pg, p % page], mk[pg, p % page] = kref[row], vref[row], kmag[row]
            hit[pg, p % page] = True
    return k, v, mk, hit


def check_append(c, new, past, page, q_out, before, pos=None):
    rows, rot = c["rows"], c["rot"]
    if pos is None:
        pos = torch.zeros(rows, dtype=torch.int64)
        for s, n in enumerate(new):
            pos[c["at"][s]:c["at"][s] + n] = torch.arange(past[s], past[s] + n)
    f = (lambda x: turned(x.cpu(), pos, rot, c["layout"], c["rotary"].freq, c["rotary"].scale)) if rot else (lambda x: (x.cpu().to(F64), x.cpu().to(F64).abs()))
    a, b = c["at"][0], c["at"][-1]
    if q_out is not None:
        qr, qm = f(c["q"])
        close(q_out[a:b], qr[a:b], qm[a:b])
    kr, km = f(c["kn"])
    k, v, mk, hit = cache_want(c, new, past, page, kr, km, c["vn"].cpu().to(F64), before)
    close(c["k"], k, mk)
    assert torch.equal(c["v"].cpu(), v.to(BF16))
    for got, was in ((c["k"], before[0]), (c["v"], before[1])):
        assert torch.equal(got.cpu()[~hit], was.cpu()[~hit])


@pytest.mark.parametrize("case", APPENDS, ids=[str(i) for i in range(len(APPENDS))])
def test_append(case):
    new, past, page = case[0], case[1], case[5]
    c = append_case(*case)
    q_out = torch.full((c["rows"],) + c["q"].shape[1:], 7.0, dtype=BF16, device="cuda")
    before = c["k"].clone(), c["v"].clone()
    c["cache"].append(c["batch"], c["rows"], c["kn"], c["vn"], q=c["q"], q_out=q_out, rotary=c["rotary"], dtype=c["dt"])
    c["cache"].check()
    check_append(c, new, past, page, q_out, before)


@pytest.mark.parametrize("rot", [0, 64])
def test_append_parts(rot):
    """Queries alone, keys and values alone, without a rotation, in place; rows outside the sequences are left."""
    case = ([3, 40], [20, 0], 8, 2, 64, 16, False, BF16, rot, 0, 0)
    c = append_case(*case, starts_at=2, extra=5)
    before = c["k"].clone(), c["v"].clone()
    q_out = torch.full((c["rows"], 8, 64), 7.0, dtype=BF16, device="cuda")
    c["cache"].append(c["batch"], c["rows"], q=c["q"], q_out=q_out, rotary=c["rotary"])
    c["cache"].check()
    assert torch.equal(c["k"], before[0]) and torch.equal(c["v"], before[1])
    assert (q_out[:2] == 7).all() and (q_out[45:] == 7).all()
    c["cache"].append(c["batch"], c["rows"], c["kn"], c["vn"], rotary=c["rotary"])
    c["cache"].check()
    check_append(c, case[0], case[1], 16, q_out, before)
    was = c["qkv"].clone()
    c["cache"].append(c["batch"], c["rows"], q=c["q"], q_out=c["q"], rotary=c["rotary"])
    c["cache"].check()
    assert torch.equal(c["q"][2:45], q_out[2:45])
    was.view(c["rows"], 12, 64)[2:45, :8] = q_out[2:45]
    assert torch.equal(c["qkv"], was)


def test_append_given_positions():
    """The angles go by the given positions, far and negative ones too; the slots by the cache's."""
    case = ([6, 3], [10, 40], 4, 2, 128, 16, False, F32, 128, 1, 0)
    c = append_case(*case)
    pos = torch.tensor([0, 1, -3, 2 ** 31 - 1, -2 ** 31, 1 << 20, 131071, 7, 0], dtype=I32)
    q_out = torch.zeros(9, 4, 128, dtype=BF16, device="cuda")
    before = c["k"].clone(), c["v"].clone()
    c["cache"].append(c["batch"], 9, c["kn"], c["vn"], q=c["q"], q_out=q_out, rotary=c["rotary"], positions=pos.cuda(), dtype=c["dt"])
    c["cache"].check()
    check_append(c, case[0], case[1], 16, q_out, before, pos=pos.long())


def test_append_tokens_without_a_slot():
    """Negative positions, pages outside the cache and positions past the table are not stored; their queries are turned."""
    case = ([8, 20, 4], [0, 10, 30], 4, 2, 64, 8, False, BF16, 64, 0, 0)
    c = append_case(*case)
    c["lengths"][0] = 5                     # positions -3..4
    c["table"][1, 2] = -1
    c["table"][1, 3] = c["cache"].pages
    c["table"] = c["table"][:, :4]          # sequence 2: positions 30, 31 are in the table
    c["batch"] = uw.KVBatch(c["starts"], c["lengths"], c["table"])
    before = c["k"].clone(), c["v"].clone()
    q_out = torch.zeros(32, 4, 64, dtype=BF16, device="cuda")
    c["cache"].append(c["batch"], 32, c["kn"], c["vn"], q=c["q"], q_out=q_out, rotary=c["rotary"])
    c["cache"].check()
    check_append(c, case[0], [-3, 10, 30], 8, q_out, before)


def test_append_graph():
    case = ([1] * 6, [3, 8, 15, 16, 17, 100], 4, 2, 64, 8, False, BF16, 64, 0, 0)
    c = append_case(*case)
    before = c["k"].clone(), c["v"].clone()
    q_out = torch.zeros(6, 4, 64, dtype=BF16, device="cuda")
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        c["cache"].append(c["batch"], 6, c["kn"], c["vn"], q=c["q"], q_out=q_out, rotary=c["rotary"])
    c["qkv"].copy_(torch.randn(c["qkv"].shape, generator=c["g"]).to(BF16))
    g.replay()
    torch.cuda.synchronize()
    check_append(c, case[0], case[1], 8, q_out, before)


# ------------------------------------------------------------------------------------------------ together
def test_chunks_and_tokens_of_a_sequence():
    """A prompt appended in chunks and then token by token, with attention after each, as a whole prompt at once."""
    H, Hq, D, page, n = 2, 8, 128, 16, 300
    g = torch.Generator().manual_seed(5)
    k, v = (torch.full((40, page, H, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    cache, rotary = uw.KVCache(k, v), uw.Rotary(D)
    qkv = torch.randn(n, (Hq + 2 * H) * D, generator=g).to(BF16).cuda().view(n, Hq + 2 * H, D)
    table = torch.randperm(40, generator=g)[:19].to(I32).view(1, 19).cuda()
    out = torch.zeros(n, Hq, D, dtype=BF16, device="cuda")
    q_all = torch.zeros_like(out)
    at = 0
    for m in (130, 1, 64, 99, 1, 1, 4):
        batch = uw.KVBatch(torch.tensor([0, m], dtype=I32).cuda(), torch.tensor([at + m], dtype=I32).cuda(), table)
        q, kk, vv = qkv[at:at + m].split([Hq, H, H], 1)
        need = cache.workspace_size(batch, m, Hq)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        cache.append(batch, m, kk, vv, q=q, q_out=q_all[at:at + m], rotary=rotary)
        cache.attend(batch, m, q_all[at:at + m], out[at:at + m], workspace=ws, ws_bytes=need)
        at += m
    cache.check()
    kr, vr = (t[table[0].long()].reshape(-1, H, D)[:n].cpu() for t in (k, v))
    kw, km = turned(qkv[:, Hq:Hq + H].cpu(), torch.arange(n), D, 0, rotary.freq, 1.0)
    close(kr, kw, km)
    assert torch.equal(vr, qkv[:, Hq + H:].cpu())
    ref, _, b, _ = plain_attend(q_all.cpu(), kr, vr, n, D ** -0.5, True, 0)
    assert ((out.cpu().to(F64) - ref).abs() <= b).all()


# ------------------------------------------------------------------------------------------------ refusals
def test_refusals():
    c = batch_of([2], [30], 16, H=2, D=64)
    q, out = torch.zeros(2, 4, 64, dtype=BF16, device="cuda"), torch.zeros(2, 4, 64, dtype=BF16, device="cuda")
    need = c["cache"].workspace_size(c["batch"], 2, 4)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")

    def bad(status, f, *a, **kw):
        with pytest.raises(uw.UwError) as e:
            f(*a, **kw)
        assert e.value.status == status, str(e.value)

    at, ap, bt = c["cache"].attend, c["cache"].append, c["batch"]
    ok = dict(workspace=ws, ws_bytes=need)
    bad(uw.ERR_WORKSPACE, at, bt, 2, q, out, workspace=ws, ws_bytes=need - 1)
    bad(uw.ERR_WORKSPACE, at, bt, 2, q, out)
    bad(uw.ERR_INVALID_ARG, at, bt, 2, q, out, workspace=ws[1:], ws_bytes=need)
    bad(uw.ERR_INVALID_ARG, at, bt, 2, q, q, **ok)
    bad(uw.ERR_INVALID_ARG, at, bt, 2, q, out, scale=float("inf"), **ok)
    bad(uw.ERR_INVALID_ARG, at, bt, 2, q, out, scale=float("nan"), **ok)
    bad(uw.ERR_INVALID_ARG, at, bt, 2, q, out, window=-1, **ok)
    bad(uw.ERR_INVALID_ARG, at, bt, 2, q, out, window=4, causal=False, **ok)
    bad(uw.ERR_INVALID_ARG, at, bt, 2, q.data_ptr() + 2, out, q_heads=4, **ok)
    bad(uw.ERR_INVALID_ARG, at, bt, 2, 0, out, q_heads=4, **ok)
    bad(uw.ERR_SHAPE, at, bt, 2, q.data_ptr(), out.data_ptr(), q_heads=3, **ok)
    bad(uw.ERR_SHAPE, at, bt, 2, q.data_ptr(), out.data_ptr(), q_heads=0, **ok)
    bad(uw.ERR_SHAPE, at, bt, 2, q.data_ptr(), out.data_ptr(), q_heads=130, **ok)
    bad(uw.ERR_SHAPE, at, bt, -1, q.data_ptr(), out.data_ptr(), q_heads=4, **ok)
    bad(uw.ERR_SHAPE, at, bt, 2, q.data_ptr(), out.data_ptr(), q_heads=4, ldq=255, **ok)
    bad(uw.ERR_SHAPE, at, bt, 2, q.data_ptr(), out.data_ptr(), q_heads=4, ldo=248, **ok)
    at(bt, 0, 0, 0, q_heads=4, **ok)
    k = torch.zeros(2, 2, 64, dtype=BF16, device="cuda")
    bad(uw.ERR_INVALID_ARG, ap, bt, 2, k, None)
    bad(uw.ERR_INVALID_ARG, ap, bt, 2, k, k, q=q)
    bad(uw.ERR_INVALID_ARG, ap, bt, 2)
    bad(uw.ERR_INVALID_ARG, ap, bt, 2, k.data_ptr(), k.data_ptr(), dtype=5)
    bad(uw.ERR_INVALID_ARG, ap, bt, 2, k.data_ptr() + 8, k.data_ptr())
    bad(uw.ERR_INVALID_ARG, ap, bt, 2, q=q.data_ptr(), q_out=q.data_ptr(), q_heads=4, dtype=uw.OUT_F32)
    bad(uw.ERR_SHAPE, ap, bt, 2, k.data_ptr(), k.data_ptr(), ldk=120)
    bad(uw.ERR_SHAPE, ap, bt, 2, k.data_ptr(), k.data_ptr(), ldv=129)
    bad(uw.ERR_SHAPE, ap, bt, 2, k, k, rotary=uw.Rotary(128))
    bad(uw.ERR_INVALID_ARG, ap, bt, 2, k, k, rotary=uw.Rotary(64, layout=7))
    for a in ((torch.zeros(2, 4, 32, dtype=BF16, device="cuda"), out), (q[:1], out), (q.float(), out), (q, out[:, :2]), (q.cpu(), out), (q[:, :, ::2], out)):
        with pytest.raises(ValueError):
            at(bt, 2, *a, **ok)
    with pytest.raises(ValueError):
        uw.KVBatch(c["starts"], c["lengths"][:0], c["table"])
    with pytest.raises(ValueError):
        uw.KVBatch(c["starts"].long(), c["lengths"], c["table"])
    with pytest.raises(ValueError):
        uw.KVCache(c["k"], c["v"][:1])
    e = torch.zeros(4, 16, 2, 96, dtype=BF16, device="cuda")
    bad(uw.ERR_UNSUPPORTED, uw.KVCache, e, e)
    e = torch.zeros(4, 12, 2, 64, dtype=BF16, device="cuda")
    bad(uw.ERR_SHAPE, uw.KVCache, e, e)
    e = torch.zeros(4, 16, 2, 68, dtype=BF16, device="cuda")[..., :64]
    bad(uw.ERR_INVALID_ARG, uw.KVCache, e, e)
