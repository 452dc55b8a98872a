"""The norms around a block with gate and residual against a plain form in 64 bits.

Tolerance: a sum of squares joins at most 64 elements a thread in sequence and ten levels of a tree, so it is within
75 2^-24 of its value, its root half that, and the reciprocal root and the products add a few 2^-23 each; the weighted sum
of up to 16 expert rows adds 17 2^-24 of its magnitudes.  1e-5 of the magnitudes that meet in an element covers these;
u also takes what the error of h' does to the second norm.  A bf16 output adds half a unit in the last place, at most
2^-8 of the value."""
import numpy as np
import pytest

import lossless_bf16_weight_exponent_gb300 as uw

pytestmark = pytest.mark.gpu
REL = 1e-5


def torch():
    import torch as t
    return t


def make(T, D, topk=0, y_rows=None, res="bf16", block="bf16", post=False, gate_every=0, pre=True, seed=0, h=True, y=True):
    t = torch()
    g = t.Generator().manual_seed(seed + T * 7 + D)
    dt = {"bf16": t.bfloat16, "f32": t.float32}
    r = lambda *s: t.randn(*s, generator=g)  # noqa: E731
    y_rows = y_rows or T * max(1, topk)
    c = dict(T=T, D=D, topk=topk, y_rows=y_rows, eps=1e-5, a=0.9, s=0.7, gate_every=gate_every)
    c["h"] = (r(T, D) * 2).to(dt[res]) if h else None
    c["y"] = r(y_rows, D).to(dt[block]) if y else None
    c["post"] = (1 + 0.2 * r(D)).bfloat16() if post else None
    c["pre"] = (1 + 0.2 * r(D)).bfloat16() if pre else None
    c["gate"] = (0.5 * r(-(-T // gate_every), D)).bfloat16() if gate_every else None
    c["pos"] = t.randperm(y_rows, generator=g)[:T * topk].to(t.int32).view(T, topk) if topk else None
    c["p"] = t.rand(T, topk, generator=g) if topk else None
    c["res"], c["block"] = res, block
    return c


def n64(v):
    return v.double().numpy()


def plain(c):
    """h', u and their bounds."""
    T, D = c["T"], c["D"]
    o = np.zeros((T, D))
    om = np.zeros((T, D))
    if c["topk"]:
        pos = c["pos"].numpy()
        for j in range(c["topk"]):
            ok = (pos[:, j] >= 0) & (pos[:, j] < c["y_rows"])
            v = n64(c["p"])[:, j, None] * n64(c["y"])[np.clip(pos[:, j], 0, c["y_rows"] - 1)] * ok[:, None]
            o += v
            om += np.abs(v)
    elif c["y"] is not None:
        o = n64(c["y"])
        om = np.abs(o)
    f = np.full((T, D), c["s"])
    if c["post"] is not None:
        f = f * n64(c["post"]) / np.sqrt((o * o).mean(1, keepdims=True) + c["eps"])
    if c["gate"] is not None:
        f = f * n64(c["gate"])[np.arange(T) // c["gate_every"]]
    h = f * o
    m = np.abs(f) * om
    if c["h"] is not None:
        h = h + c["a"] * n64(c["h"])
        m = m + np.abs(c["a"] * n64(c["h"]))
    if c["pre"] is None:
        return h, REL * m, None, None
    rms = np.sqrt((h * h).mean(1, keepdims=True) + c["eps"])
    w = n64(c["pre"])
    u = w * h / rms
    ub = REL * (np.abs(w) * m / rms + np.abs(u) * (1 + np.sqrt((m * m).mean(1, keepdims=True)) / rms))
    return h, REL * m, u, ub


def run(c, in_place=False, stream=None, store=True):
    t = torch()
    d = {k: v.cuda() if isinstance(v, t.Tensor) else v for k, v in c.items()}
    od = {"bf16": uw.OUT_BF16, "f32": uw.OUT_F32}
    n = uw.BlockNorm(c["D"], d["post"], d["gate"], c["gate_every"], d["pre"], c["a"], c["s"], c["eps"], od[c["res"]], od[c["block"]])
    dt = t.bfloat16 if c["res"] == "bf16" else t.float32
    h_out = None
    if store:
        h_out = d["h"] if in_place else t.full((c["T"], c["D"]), float("nan"), dtype=dt, device="cuda")
    u = None
    if c["pre"] is not None:
        u = d["y"] if in_place and not c["topk"] else t.full((c["T"], c["D"]), float("nan"), dtype=t.bfloat16, device="cuda")
    if stream is not None:
        stream.wait_stream(t.cuda.current_stream())
    n.run(c["T"], d["h"], h_out, d["y"], d["pos"], d["p"], c["topk"], c["y_rows"], u, stream)
    t.cuda.synchronize()
    return h_out, u


def check(c, got):
    h, hb, u, ub = plain(c)
    for v, ref, b, bf in ((got[0], h, hb, c["res"] == "bf16"), (got[1], u, ub, True)):
        if v is None:
            continue
        err = np.abs(v.double().cpu().numpy() - ref)
        bound = b + (2.0 ** -8 * (np.abs(ref) + b) if bf else 0) + 1e-30
        assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("res", ["bf16", "f32"])
@pytest.mark.parametrize("block", ["bf16", "f32"])
@pytest.mark.parametrize("topk", [0, 1, 8, 16])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (5, 64), (17, 1000), (33, 2048), (2, 4099)])
def test_block_norm(T, D, topk, block, res):
    c = make(T, D, topk, res=res, block=block, post=True, gate_every=2)
    check(c, run(c))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate_every", [0, 1, 5, 1000])
@pytest.mark.parametrize("pre", [False, True])
def test_parts(post, gate_every, pre):
    c = make(12, 520, post=post, gate_every=gate_every, pre=pre)
    check(c, run(c))


@pytest.mark.parametrize("D", [8192, 8193, 14336, 28672, 65536])
def test_long_rows(D):
    for topk in (0, 2):
        c = make(3, D, topk, post=True, gate_every=3)
        check(c, run(c))


def test_first_norm_no_residual_and_nothing_stored():
    c = make(9, 264, y=False)
    h, u = run(c, store=False)
    assert h is None
    check(c, (None, u))
    c = make(9, 264, h=False, post=True)
    check(c, run(c))


def test_in_place_and_other_stream():
    t = torch()
    c = make(40, 776, post=True, gate_every=40)
    check(c, run(c, in_place=True))
    c = make(40, 776, 4, post=True)
    check(c, run(c, in_place=True, stream=t.cuda.Stream()))


def test_positions_outside_add_nothing():
    c = make(20, 96, 3, y_rows=60)
    c["pos"][::2, 1] = -1
    c["pos"][3] = 60
    c["pos"][4] = 2 ** 31 - 1
    c["pos"][5] = -2 ** 31
    check(c, run(c))


def test_rows_of_zeros_and_of_large_values():
    t = torch()
    c = make(6, 512, post=True, res="f32", block="f32")
    c["h"][0], c["y"][0] = 0, 0  # rms 0: eps keeps the quotient finite
    c["y"][1] = 0
    c["h"][2] *= 1e15            # squares near the end of the range
    c["y"][3] *= 1e15
    h, u = run(c)
    check(c, (h, u))
    assert t.isfinite(u).all() and (u[0] == 0).all()


def test_non_finite_values_stay_in_their_row():
    t = torch()
    c = make(8, 256, post=True)
    c["y"][3, 17] = float("nan")
    c["h"][5, 0] = float("inf")
    h, u = run(c)
    rows = [0, 1, 2, 4, 6, 7]
    assert t.isfinite(u[rows]).all() and t.isfinite(h[rows]).all() and t.isnan(u[3]).all() and t.isinf(h[5, 0])


def test_refusals():
    t = torch()
    x = t.zeros(4, 64, dtype=t.bfloat16, device="cuda")
    p = t.zeros(64, dtype=t.int32, device="cuda")

    def status(n=None, rows=4, h=x, h_out=x, y=x, **k):
        with pytest.raises(uw.UwError) as e:
            uw.BlockNorm(64, **(n or {})).run(rows, h, h_out, y, **k)
        return e.value.status

    w = x[0]
    assert status(u=x) == status(n=dict(pre_weight=w)) == uw.ERR_INVALID_ARG  # u and its weight go together
    assert status(h_out=None) == status(h=None, y=None) == uw.ERR_INVALID_ARG
    assert status(n=dict(gate=w, gate_every=0)) == status(n=dict(res_dtype=5)) == status(n=dict(block_dtype=-1)) == uw.ERR_INVALID_ARG
    assert status(topk=2) == status(topk=17, pos=p, weights=p, y_rows=4) == status(topk=-1) == uw.ERR_INVALID_ARG
    assert status(h=x.data_ptr() + 2) == status(n=dict(post_weight=w.data_ptr() + 8)) == uw.ERR_INVALID_ARG
    assert status(rows=-1) == status(y_rows=-1) == uw.ERR_SHAPE
    with pytest.raises(uw.UwError) as e:
        uw.BlockNorm(65537).run(1, x, x, x)
    assert e.value.status == uw.ERR_SHAPE
    uw.BlockNorm(64).run(0, x, x, x)
