"""Groups of compressed expert matrices and their grouped product: the form is lossless for every bit pattern, and
the product matches a plain 64-bit one for ragged rows per expert, odd sizes, strides, padding rows and both output
types, gated and not.

Tolerance of a product: fp32 accumulation in a tree of at most K / 16 sequential steps of 16 products each, every step
off by at most 2^-22 of the running sum of magnitudes (the tensor pipe may truncate), is within K 2^-26 sum |w x|,
6e-5 of it at the largest K here; the suite's 1e-4 sum |w x| + 1e-6 covers that.  A bf16 output adds half a unit in the
last place, at most 2^-8 |y|.  A gated output a/(1+e^-a) b moves by at most 1.1 |b| per unit of a and |a| per unit of b, and
the exponential and division add a few 2^-23 |y| (4e-6 taken)."""
import numpy as np
import pytest

import lossless_bf16_weight_exponent_gb300 as uw
import synth

pytestmark = pytest.mark.gpu


def torch():
    import torch as t
    return t


def dev(a, dtype=None):
    t = torch()
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return t.from_numpy(a.view(np.int16)).cuda().view(t.bfloat16)
    r = t.from_numpy(a).cuda()
    return r if dtype is None else r.to(dtype)


def f64(bits):
    return synth.bf16_to_f32(bits).astype(np.float64)


def weights(E, N, K, seed, outliers=2e-3):
    return synth.fill((E, N, K), seed=seed, scale=0.02, p1=outliers, f1=300.0)


def offsets_of(counts, start=0):
    return np.concatenate([[start], start + np.cumsum(counts)]).astype(np.int32)


def reference(w, w_up, x, src, offsets, rows):
    """(y, bound of its fp32 error) of every row of [0, rows); NaN rows are not written."""
    E, N, K = w.shape
    y = np.full((rows, N), np.nan)
    bound = np.zeros((rows, N))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi <= lo:
            continue
        s = src[lo:hi]
        ok = (s >= 0) & (s < x.shape[0])
        xe = np.where(ok[:, None], x[np.clip(s, 0, x.shape[0] - 1)], 0.0)
        a, ea = xe @ f64(w[e]).T, 1e-4 * (np.abs(xe) @ np.abs(f64(w[e])).T) + 1e-6
        if w_up is None:
            y[lo:hi], bound[lo:hi] = a, ea
            continue
        b, eb = xe @ f64(w_up[e]).T, 1e-4 * (np.abs(xe) @ np.abs(f64(w_up[e])).T) + 1e-6
        silu = a / (1 + np.exp(-a))
        y[lo:hi] = silu * b
        bound[lo:hi] = 1.1 * ea * (np.abs(b) + eb) + np.abs(silu) * eb + 4e-6 * np.abs(silu * b) + 1e-6
    return y, bound


def check(y, ref, bound, bf16):
    wr = ~np.isnan(ref)
    assert np.array_equal(np.isnan(y), ~wr)
    b = bound + (2.0 ** -8 * (np.abs(ref) + bound) if bf16 else 0)
    err = np.abs(y - ref)[wr]
    assert (err <= b[wr]).all(), float((err / b[wr]).max())


def run(g, x, offsets, rows, out_bf16, src=None, x_rows=None, ldx=0, ldy=0, stream=None):
    t = torch()
    y = t.full((rows, ldy or g.N), float("nan"), dtype=t.bfloat16 if out_bf16 else t.float32, device="cuda")
    g.matmul(x, offsets, rows, y, row_src=src, x_rows=x_rows, out_dtype=uw.OUT_BF16 if out_bf16 else uw.OUT_F32, ldx=ldx, ldy=ldy,
             stream=stream)
    g.check(stream)
    return y.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------------------------------------ the form
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,K", [(1, 64), (15, 128), (16, 192), (17, 64), (130, 1408), (257, 320)])
@pytest.mark.parametrize("kind", ["normal", "bits", "zeros", "wide"])
def test_form_is_lossless(kind, N, K, gated):
    t = torch()
    E = 3

    def make(seed):
        if kind == "bits":
            return synth.random_bits((E, N, K), seed)
        if kind == "zeros":
            w = weights(E, N, K, seed)
            w[:, :, ::7] = 0
            w[1] = 0x8000
            return w
        w = weights(E, N, K, seed)
        if kind == "wide":  # every fourth row spans all exponents
            w[:, ::4] = (w[:, ::4] & 0x807F) | ((np.arange(K) % 256).astype(np.uint16) << 7)
        return w

    w, u = make(5), make(6)
    g = uw.Group(dev(w), dev(u) if gated else None)
    for e in range(E):
        for up, ref in ((False, w), (True, u)) if gated else ((False, w),):
            out = t.full((N, K), 0x5555, dtype=t.int16, device="cuda")
            g.decode(e, out, up=up)
            assert np.array_equal(out.cpu().numpy().view(np.uint16), ref[e]), (e, up)


@pytest.mark.parametrize("outliers", [0.0, 2e-3])
def test_form_size_and_verbatim_runs(outliers):
    # 12 bits a weight, 32 bytes a step of 8192, and 64 bytes for each run that the 16 consecutive exponents that cover
    # the most weights of its matrix do not hold: counted here from the bits
    E, N, K = 2, 1024, 1024
    w = weights(E, N, K, 3, outliers)
    g = uw.Group(dev(w))
    runs = 0
    for e in range(E):
        exps = (w[e] >> 7) & 255
        cover = np.convolve(np.bincount(exps.ravel(), minlength=256), np.ones(16, np.int64), "valid")
        base = int(np.argmax(cover))
        runs += int(((exps < base) | (exps > base + 15)).reshape(-1, 64).any(1).sum())
    assert g.info["n_verbatim"] == runs
    steps = E * (N // 128) * (K // 64)
    assert steps * (12288 + 32) + 64 * runs <= g.info["device_bytes"] <= steps * (12288 + 32) + 64 * runs + 8192


@pytest.mark.parametrize("codec,resident", [(uw.CODEC_PALETTE, "both"), (uw.CODEC_HUFFMAN, "huffman"), (uw.CODEC_HUFFMAN, "palette")])
def test_group_of_loaded_matrices(codec, resident):
    t = torch()
    E, N, K = 3, 100, 320
    w, u = weights(E, N, K, 21), weights(E, N, K, 22)
    ms = [[uw.Matrix(uw.encode(a[e], codec), resident=resident) for e in range(E)] for a in (w, u)]
    g = uw.Group(ms[0], ms[1])
    for m in ms[0] + ms[1]:
        m.close()  # the group holds its own copy
    for up, ref in ((False, w), (True, u)):
        for e in range(E):
            out = t.empty((N, K), dtype=t.int16, device="cuda")
            g.decode(e, out, up=up)
            assert np.array_equal(out.cpu().numpy().view(np.uint16), ref[e])


# ------------------------------------------------------------------------------------------------ the product
COUNTS = {"one": [1], "single_row": [0, 0, 1, 0], "few": [3, 0, 8, 9, 1], "ragged": [0, 17, 1, 130, 0, 64, 5, 300],
          "all_in_last": [0, 0, 0, 40], "even": [16] * 6, "many_empty": [0] * 70 + [2] + [0] * 30 + [11]}


@pytest.mark.parametrize("out_bf16", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("N,K", [(48, 256), (130, 448), (1, 64)])
def test_product(N, K, counts, gated, out_bf16):
    c = COUNTS[counts]
    E, rows = len(c), sum(c)
    w = weights(E, N, K, N + rows)
    u = weights(E, N, K, N + rows + 1) if gated else None
    x = synth.fill((rows, K), seed=rows)
    off = offsets_of(c)
    ref, bound = reference(w, u, f64(x), np.arange(rows), off, rows)
    g = uw.Group(dev(w), dev(u) if gated else None)
    check(run(g, dev(x), dev(off), rows, out_bf16), ref, bound, out_bf16)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows_each", [2, 40, 600])
def test_gathered_rows_strides_and_padding(rows_each, gated):
    t = torch()
    rng = np.random.default_rng(rows_each)
    E, N, K, T, ldx, ldy = 5, 70, 192, 37, 208, 75
    c = rng.integers(0, 2 * rows_each, E)
    off = offsets_of(c, start=3)  # the first three rows belong to nobody
    rows = int(off[-1]) + 2       # nor do the last two
    src = rng.integers(0, T, rows).astype(np.int32)
    src[::5] = -1
    src[1::11] = T                # past the end
    src[2::13] = 2 ** 31 - 1
    w, u = weights(E, N, K, 31), weights(E, N, K, 32) if gated else None
    x = synth.fill((T, ldx), seed=33)
    ref, bound = reference(w, u, f64(x)[:, :K], src.astype(np.int64), off, rows)
    g = uw.Group(dev(w), dev(u) if gated else None)
    y = run(g, dev(x), dev(off), rows, False, src=dev(src), ldx=ldx, ldy=ldy)
    check(y[:, :N], ref, bound, False)
    assert np.isnan(y[:, N:]).all()  # nothing is written between the rows


def test_offsets_outside_the_rows_are_clamped():
    E, N, K, rows = 3, 32, 64, 20
    w, x = weights(E, N, K, 41), synth.fill((rows, K), seed=42)
    off = np.array([-5, 8, 8, 1000], np.int32)
    ref, bound = reference(w, None, f64(x), np.arange(rows), np.clip(off, 0, rows), rows)
    check(run(uw.Group(dev(w)), dev(x), dev(off), rows, False), ref, bound, False)


@pytest.mark.parametrize("rows_each", [3, 48, 300])
def test_exact_integers(rows_each):
    # small integers: every partial sum is exact, so the result is, whatever the order
    rng = np.random.default_rng(7)
    E, N, K = 4, 100, 512
    wi = (rng.integers(-3, 4, (E, N, K)) * 2.0 ** rng.integers(0, 3, (E, N, K))).astype(np.float32)
    c = [rows_each, 0, rows_each + 1, 2]
    rows = sum(c)
    xi = rng.integers(-4, 5, (rows, K)).astype(np.float32)
    off = offsets_of(c)
    g = uw.Group(dev((wi.view(np.uint32) >> 16).astype(np.uint16)))
    y = run(g, dev((xi.view(np.uint32) >> 16).astype(np.uint16)), dev(off), rows, False)
    for e in range(E):
        assert np.array_equal(y[off[e]:off[e + 1]], xi[off[e]:off[e + 1]].astype(np.float64) @ wi[e].astype(np.float64).T)


def test_non_finite_weights_stay_in_their_outputs():
    E, N, K, rows = 2, 40, 128, 20
    w, x = weights(E, N, K, 51, 0.0), np.abs(f64(synth.fill((rows, K), seed=52)))
    xb = (np.maximum(x, 0.1).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    w[0, 5, 9], w[0, 7, 3], w[1, 33, 100] = 0x7F80, 0x7FC0, 0xFF80  # inf, NaN, -inf
    off = offsets_of([12, 8])
    y = run(uw.Group(dev(w)), dev(xb), dev(off), rows, False)
    assert np.isposinf(y[:12, 5]).all() and np.isnan(y[:12, 7]).all() and np.isneginf(y[12:, 33]).all()
    ok = np.isfinite(y)
    ok[:12, [5, 7]] = ok[12:, 33] = True
    assert ok.all()


def test_rows_do_not_depend_on_other_rows_or_runs():
    t = torch()
    E, N, K = 6, 96, 256
    w, u = weights(E, N, K, 61), weights(E, N, K, 62)
    g = uw.Group(dev(w), dev(u))
    x = synth.fill((200, K), seed=63)
    a = run(g, dev(x), dev(offsets_of([40, 40, 40, 40, 20, 20])), 200, False)
    b = run(g, dev(x), dev(offsets_of([40, 40, 40, 40, 20, 20])), 200, False)
    assert np.array_equal(a, b)
    x2 = x.copy()
    x2[40:] = synth.fill((160, K), seed=64)
    assert np.array_equal(run(g, dev(x2), dev(offsets_of([40, 40, 40, 40, 20, 20])), 200, False)[:40], a[:40])


def test_other_stream_and_graph():
    t = torch()
    E, N, K, rows = 4, 64, 192, 50
    w, x = weights(E, N, K, 71), synth.fill((rows, K), seed=72)
    off = offsets_of([10, 0, 33, 7])
    ref, bound = reference(w, None, f64(x), np.arange(rows), off, rows)
    g = uw.Group(dev(w))
    xd, od = dev(x), dev(off)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    check(run(g, xd, od, rows, False, stream=s), ref, bound, False)
    y = t.zeros((rows, N), dtype=t.float32, device="cuda")
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=s):
        g.matmul(xd, od, rows, y, out_dtype=uw.OUT_F32, stream=s)
    # the rows per expert are read when the graph runs
    off2 = offsets_of([0, 45, 0, 5])
    od.copy_(dev(off2))
    y.fill_(float("nan"))
    graph.replay()
    t.cuda.synchronize()
    ref, bound = reference(w, None, f64(x), np.arange(rows), off2, rows)
    check(y.cpu().numpy().astype(np.float64), ref, bound, False)


def test_no_rows_is_a_no_op():
    g = uw.Group(dev(weights(2, 16, 64, 81)))
    t = torch()
    y = t.full((1, 16), 7.0, device="cuda")
    g.matmul(y, dev(np.zeros(3, np.int32)), 0, y, x_rows=0, out_dtype=uw.OUT_F32)
    # rows exist, but no expert has them and there is nothing to read
    g.matmul(0, dev(np.zeros(3, np.int32)), 1, y, x_rows=0, out_dtype=uw.OUT_F32)
    t.cuda.synchronize()
    assert (y == 7.0).all()


def test_refusals():
    t = torch()
    w = dev(weights(2, 32, 128, 91))
    g = uw.Group(w)
    x, off = dev(synth.fill((4, 128), seed=1)), dev(offsets_of([2, 2]))
    y = t.empty((4, 32), device="cuda")

    def status(fn):
        with pytest.raises(uw.UwError) as e:
            fn()
        return e.value.status

    assert status(lambda: uw.Group(w.view(2, 64, 64)[:, :, :32].contiguous())) == uw.ERR_SHAPE
    assert status(lambda: uw.Group(w[:0])) == uw.ERR_INVALID_ARG
    ms = [uw.Matrix(uw.encode(synth.fill(s, seed=2))) for s in ((32, 64), (32, 128))]
    assert status(lambda: uw.Group(ms)) == uw.ERR_SHAPE
    assert status(lambda: uw.Group([])) == uw.ERR_INVALID_ARG
    f = dict(out_dtype=uw.OUT_F32)
    assert status(lambda: g.matmul(x, off, -1, y, **f)) == uw.ERR_SHAPE
    assert status(lambda: g.matmul(x, off, 4, y, ldx=120, **f)) == uw.ERR_SHAPE
    assert status(lambda: g.matmul(x, off, 4, y, ldx=132, **f)) == uw.ERR_SHAPE
    assert status(lambda: g.matmul(x, off, 4, y, ldy=16, **f)) == uw.ERR_SHAPE
    assert status(lambda: g.matmul(x, off, 4, y, out_dtype=7)) == uw.ERR_INVALID_ARG
    assert status(lambda: g.matmul(x, None, 4, y, **f)) == uw.ERR_INVALID_ARG
    assert status(lambda: g.matmul(x, off, 4, None, **f)) == uw.ERR_INVALID_ARG
    assert status(lambda: g.matmul(x.data_ptr() + 2, off, 4, y, x_rows=3, **f)) == uw.ERR_INVALID_ARG
    assert status(lambda: g.matmul(x, off, 4, y.data_ptr() + 4, **f)) == uw.ERR_INVALID_ARG
    assert status(lambda: g.decode(2, w)) == uw.ERR_INVALID_ARG
    assert status(lambda: g.decode(0, w, up=True)) == uw.ERR_UNSUPPORTED


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows_each", [3, 20, 150])
def test_long_sums_in_fp32(rows_each, gated):
    # An fp32 output is summed in segments of 512: 32 products of 16 that each cut at most 2^-24 of a running sum no larger
    # (in the norm) than the result, and 16 additions of segments at K = 8192, 2^-24 each: 48 2^-24 of the result's norm
    # (a gated result has two such factors; its activation passes errors on at most 1.1-fold).  One sum of all of K would be off by
    # several times that.
    t = torch()
    E, N, K = 3, 64, 8192
    w, u = weights(E, N, K, 101, 0.0), weights(E, N, K, 102, 0.0)
    rows = E * rows_each
    x, off = synth.fill((rows, K), seed=103), offsets_of([rows_each] * E)
    y = run(uw.Group(dev(w), dev(u) if gated else None), dev(x), dev(off), rows, False)
    ref, _ = reference(w, u if gated else None, f64(x), np.arange(rows), off, rows)
    assert np.linalg.norm(y - ref) <= (2.1 if gated else 1.0) * 48 * 2.0 ** -24 * np.linalg.norm(ref)


# More units than CTAs in each of the tcgen05 shapes, K no multiple of a segment of 512, an odd number of weight tiles, so that
# every ring and both accumulators go on from one unit to the next: pairs of 192 rows, single CTAs of 64, sums of segments.
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,mean,N,out_bf16", [(6, 450, 2180, True), (20, 20, 1300, True), (6, 380, 1700, False)])
def test_many_units(E, mean, N, out_bf16, gated, gather):
    K, rng = 704, np.random.default_rng(mean)
    N = N // 2 if gated else N
    c = rng.integers(mean // 2, mean + mean // 2, E)
    c[E // 2] = 0
    off, rows = offsets_of(c), int(sum(c))
    assert 2 * E < rows and (rows <= 24 * E) == (mean == 20)
    T = rows // 3 if gather else rows
    src = rng.integers(-1, T + 1, rows) if gather else np.arange(rows)
    w, u = weights(E, N, K, 111), weights(E, N, K, 112) if gated else None
    x = synth.fill((T, K), seed=113)
    ref, bound = reference(w, u, f64(x), src, off, rows)
    g = uw.Group(dev(w), dev(u) if gated else None)
    a = run(g, dev(x), dev(off), rows, out_bf16, src=dev(src.astype(np.int32)) if gather else None)
    check(a, ref, bound, out_bf16)
    assert np.array_equal(a, run(g, dev(x), dev(off), rows, out_bf16, src=dev(src.astype(np.int32)) if gather else None))


def test_a_group_that_does_not_fit_leaves_no_error_behind():
    import ctypes
    w = dev(weights(2, 32, 128, 181))
    h = ctypes.c_void_p()
    # 413 GB of steps: refused before a weight is read
    s = uw.lib().uw_group_create_dense(w.data_ptr(), None, 1, 2 ** 24, 2 ** 14, 0, ctypes.byref(h))
    assert s == uw.ERR_NO_MEMORY and not h.value
    assert torch().cuda.is_available() and uw.Group(w).N == 32


@pytest.mark.parametrize("each", [1, 9, 60, 300])
def test_gate_over_its_whole_range(each):
    # One weight of 1 in the gate matrix and one in the up matrix: both factors are exact.  Of silu(g) u, e^-|g| is off by an ulp,
    # the quotient by two, the sum and the two products by half a one each: 4.5 2^-23, and 2^-149 of each rounding below the
    # smallest normal number, multiplied by what follows it.
    E, N, K = 40, 33, 64
    w, u = np.zeros((E, N, K), np.uint16), np.zeros((E, N, K), np.uint16)
    w[:, :, 0] = u[:, :, 1] = 0x3F80
    rows = E * each
    gate = np.linspace(-115, 115, rows).astype(np.float32)
    up = np.where(np.arange(rows) % 3 == 0, 1e30, np.where(np.arange(rows) % 3 == 1, -1.5, 1.0)).astype(np.float32)
    x = np.zeros((rows, K), np.float32)
    x[:, 0], x[:, 1] = gate, up
    xb = (x.view(np.uint32) >> 16).astype(np.uint16)
    g, b = f64(xb)[:, 0], f64(xb)[:, 1]
    want = g / (1 + np.exp(-g)) * b
    group = uw.Group(dev(w), dev(u))
    y = run(group, dev(xb), dev(offsets_of([each] * E)), rows, False)
    assert (y == y[:, :1]).all()
    bound = 5 * 2.0 ** -23 * np.abs(want) + 2.0 ** -149 * (2 + (np.abs(g) + 2) * np.abs(b))
    assert (np.abs(y[:, 0] - want) <= bound).all(), (np.abs(y[:, 0] - want) / bound).max()


@pytest.mark.parametrize("each", [1, 9, 60, 300])
def test_gate_over_its_whole_range_in_bf16(each):
    # half a unit in the last place of bf16 (of the smallest normal number's below it), and 2^-15 of the faster power and
    # quotient (2 + 1.173 |g| and 2 units in the last place)
    E, N, K = 40, 33, 64
    w, u = np.zeros((E, N, K), np.uint16), np.zeros((E, N, K), np.uint16)
    w[:, :, 0] = u[:, :, 1] = 0x3F80
    rows = E * each
    x = np.zeros((rows, K), np.float32)
    x[:, 0], x[:, 1] = np.linspace(-115, 115, rows), np.where(np.arange(rows) % 3 == 0, 1e30, -1.5)
    xb = (x.view(np.uint32) >> 16).astype(np.uint16)
    g, b = f64(xb)[:, 0], f64(xb)[:, 1]
    want = g / (1 + np.exp(-g)) * b
    y = run(uw.Group(dev(w), dev(u)), dev(xb), dev(offsets_of([each] * E)), rows, True)
    assert (y == y[:, :1]).all()
    bound = (2.0 ** -8 + 2.0 ** -15) * np.abs(want) + 2.0 ** -134 + 2.0 ** -149 * (2 + (np.abs(g) + 2) * np.abs(b))
    assert (np.abs(y[:, 0] - want) <= bound).all(), (np.abs(y[:, 0] - want) / bound).max()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N", [64, 1300])
def test_few_rows_of_long_sums_in_fp32(N, gated):
    # The bound of the test above, on the matrix-vector kernel: sums of 512 products there too.
    E, K, c = 10, 8192, [1, 0, 5, 2, 0, 9, 1, 0, 0, 2]
    w, u = weights(E, N, K, 161, 0.0), weights(E, N, K, 162, 0.0)
    rows, off = sum(c), offsets_of(c)
    x = np.abs(synth.bf16_to_f32(synth.fill((rows, K), seed=163)))  # one sign: the sums grow
    xb = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    w[:, ::2] &= 0x7FFF
    u[:, ::2] &= 0x7FFF
    y = run(uw.Group(dev(w), dev(u) if gated else None), dev(xb), dev(off), rows, False)
    ref, _ = reference(w, u if gated else None, f64(xb), np.arange(rows), off, rows)
    err = np.linalg.norm(y - ref) / np.linalg.norm(ref)
    assert err <= (2.1 if gated else 1.0) * 48 * 2.0 ** -24


# ------------------------------------------------------------------------------------------------ up to two rows an expert
# the matrix-vector kernel: CTAs of eight warps for a small grid, of four for a large one (N)
@pytest.mark.parametrize("out_bf16", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N", [70, 3000])
def test_few_rows_gathered_with_strides_and_padding(N, gated, out_bf16):
    K, T, ldx, ldy = 192, 37, 208, N + 5
    c = [1, 0, 3, 2, 0, 9, 1, 0, 0, 2, 0, 1]
    off = offsets_of(c, start=3)  # the first three rows belong to nobody
    E, rows = len(c), int(off[-1]) + 2
    assert rows <= 2 * E
    rng = np.random.default_rng(N)
    src = rng.integers(0, T, rows).astype(np.int32)
    src[4], src[9], src[10], src[14] = -1, T, 2 ** 31 - 1, -2 ** 31
    w, u = weights(E, N, K, 121), weights(E, N, K, 122) if gated else None
    x = synth.fill((T, ldx), seed=123)
    ref, bound = reference(w, u, f64(x)[:, :K], src.astype(np.int64), off, rows)
    y = run(uw.Group(dev(w), dev(u) if gated else None), dev(x), dev(off), rows, out_bf16, src=dev(src), ldx=ldx, ldy=ldy)
    check(y[:, :N], ref, bound, out_bf16)
    assert np.isnan(y[:, N:]).all()


@pytest.mark.parametrize("E", [3, 12])
def test_few_rows_with_offsets_outside_them(E):
    N, K, rows = 32, 64, 2 * E
    w, x = weights(E, N, K, 131), synth.fill((rows, K), seed=132)
    off = np.array([-5] + [2] * (E - 1) + [1000], np.int32)
    ref, bound = reference(w, None, f64(x), np.arange(rows), np.clip(off, 0, rows), rows)
    check(run(uw.Group(dev(w)), dev(x), dev(off), rows, False), ref, bound, False)


@pytest.mark.parametrize("N", [100, 3100])
def test_few_rows_of_exact_integers(N):
    rng = np.random.default_rng(8)
    c = [3, 0, 9, 2, 0, 1, 0, 0]
    E, K, rows, off = len(c), 1088, sum(c), offsets_of(c)
    wi = (rng.integers(-3, 4, (E, N, K)) * 2.0 ** rng.integers(0, 3, (E, N, K))).astype(np.float32)
    xi = rng.integers(-4, 5, (rows, K)).astype(np.float32)
    g = uw.Group(dev((wi.view(np.uint32) >> 16).astype(np.uint16)))
    y = run(g, dev((xi.view(np.uint32) >> 16).astype(np.uint16)), dev(off), rows, False)
    for e in range(E):
        assert np.array_equal(y[off[e]:off[e + 1]], xi[off[e]:off[e + 1]].astype(np.float64) @ wi[e].astype(np.float64).T)


def test_few_rows_keep_non_finite_weights_in_their_outputs():
    E, N, K, rows = 10, 40, 128, 20
    w, x = weights(E, N, K, 141, 0.0), np.abs(f64(synth.fill((rows, K), seed=142)))
    xb = (np.maximum(x, 0.1).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    w[0, 5, 9], w[0, 7, 3], w[1, 33, 100] = 0x7F80, 0x7FC0, 0xFF80  # inf, NaN, -inf
    y = run(uw.Group(dev(w)), dev(xb), dev(offsets_of([12, 8] + [0] * 8)), rows, False)
    assert np.isposinf(y[:12, 5]).all() and np.isnan(y[:12, 7]).all() and np.isneginf(y[12:, 33]).all()
    ok = np.isfinite(y)
    ok[:12, [5, 7]] = ok[12:, 33] = True
    assert ok.all()


def test_few_rows_in_a_graph_that_finds_other_experts():
    t = torch()
    E, N, K, rows = 30, 64, 192, 50
    w, x = weights(E, N, K, 151), synth.fill((rows, K), seed=152)
    g = uw.Group(dev(w))
    xd, od, s = dev(x), dev(offsets_of([10, 0, 33, 7] + [0] * 26)), t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    run(g, xd, od, rows, False, stream=s)
    y = t.zeros((rows, N), dtype=t.float32, device="cuda")
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=s):
        g.matmul(xd, od, rows, y, out_dtype=uw.OUT_F32, stream=s)
    for c in ([0] * 29 + [50], [2] * 20 + [1] * 10):
        off = offsets_of(c)
        od.copy_(dev(off))
        y.fill_(float("nan"))
        graph.replay()
        t.cuda.synchronize()
        ref, bound = reference(w, None, f64(x), np.arange(rows), off, rows)
        check(y.cpu().numpy().astype(np.float64), ref, bound, False)


@pytest.mark.parametrize("E,mine,rows,out_bf16", [(30, 5, 60, False), (8, 40, 160, True), (8, 40, 160, False), (4, 130, 700, True)])
def test_rows_do_not_depend_on_how_the_others_are_shared_out(E, mine, rows, out_bf16):
    # at a fixed number of rows, in each kernel and shape, bit for bit; another number may choose another order of sums
    N, K, rng = 96, 704, np.random.default_rng(rows)
    w, u = weights(E, N, K, 171), weights(E, N, K, 172)
    g, x = uw.Group(dev(w), dev(u)), synth.fill((3 * rows, K), seed=173)
    rest = rows - mine
    shares = [[rest] + [0] * (E - 2), [0] * (E - 2) + [rest], list(np.bincount(rng.integers(0, E - 1, rest), minlength=E - 1))]
    ys = [run(g, dev(x[:rows]), dev(offsets_of([mine] + s)), rows, out_bf16)[:mine] for s in shares]
    assert np.array_equal(ys[0], ys[1]) and np.array_equal(ys[0], ys[2])
    off = offsets_of([mine, 3 * rows - mine] + [0] * (E - 2))
    ref, bound = reference(w, u, f64(x), np.arange(3 * rows), off, 3 * rows)
    check(run(g, dev(x), dev(off), 3 * rows, out_bf16)[:mine], ref[:mine], bound[:mine], out_bf16)


@pytest.mark.skipif("__import__('torch').cuda.device_count() < 2", reason="one device")
def test_a_group_is_used_on_its_own_device():
    t = torch()
    w = weights(2, 32, 64, 191)
    with t.cuda.device(1):
        g = uw.Group(dev(w))
    x, off, y = dev(synth.fill((4, 64), seed=1)), dev(offsets_of([2, 2])), t.empty((4, 32), device="cuda")
    for call in (lambda: g.matmul(x, off, 4, y, out_dtype=uw.OUT_F32), lambda: g.decode(0, t.empty((32, 64), dtype=t.int16, device="cuda"))):
        with pytest.raises(uw.UwError) as e:
            call()
        assert e.value.status == uw.ERR_INVALID_ARG
