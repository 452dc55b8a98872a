"""The block and head example: every stage against a plain form in 64 bits on the stage's own inputs, and a graph of the
whole step against the plain calls.

Products within 1e-4 sum |w x| + 1e-6, the suite's bound, plus 2^-8 of the value where the output is bf16; the gated
product as in the group tests; norms within 1e-5 of the magnitudes that meet, log probabilities within 2^-14 (fp32 sums of
at most 5003 terms of 2^-24 each, and as much again for the powers)."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def n64(t):
    return t.double().cpu().numpy()


def product(x, w):
    return x @ w.T, 1e-4 * (np.abs(x) @ np.abs(w).T) + 1e-6


def near(got, want, bound, bf16=False):
    b = bound + (2.0 ** -8 * (np.abs(want) + bound) if bf16 else 0)
    err = np.abs(n64(got) - want)
    assert (err <= b).all(), float((err / b).max())


@pytest.mark.parametrize("tokens", [1, 7, 200])
def test_block_and_head(tokens):
    import moe_block
    import torch
    m = moe_block.MoeBlock()
    g = torch.Generator(device="cuda").manual_seed(tokens)
    h = torch.randn(tokens, m.dim, device="cuda", generator=g)
    targets = torch.randint(0, m.vocab, (tokens,), dtype=torch.int32, device="cuda", generator=g)
    lp, ent = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    ids, top = torch.empty(tokens, 5, dtype=torch.int32, device="cuda"), torch.empty(tokens, 5, device="cuda")
    out, v = m.block(h, tokens)
    m.score(tokens, targets, lp, ent, 5, ids, top)
    m.gate_up.check()
    m.down.check()
    d, rows, k = m.dense, tokens * m.topk, m.topk

    def norm(x, w):
        return n64(w) * x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-5)

    u = norm(n64(h), d["norm"])
    near(m.u[:tokens], u, 1e-5 * np.abs(u), True)
    u = n64(m.u[:tokens])
    logits, b = product(u, n64(d["router"]))
    near(m.router_logits[:tokens], logits, b)
    z = n64(m.router_logits[:tokens])
    order = np.argsort(-z, axis=1, kind="stable")[:, :k]
    assert np.array_equal(m.ids[:rows].cpu().numpy().reshape(tokens, k), order)
    p = np.take_along_axis(np.exp(z - z.max(1, keepdims=True)), order, 1)
    weights = n64(m.weights[:rows]).reshape(tokens, k)
    assert np.allclose(weights, p / p.sum(1, keepdims=True), rtol=1e-5)
    off, src, pos = (t.cpu().numpy() for t in (m.offsets, m.row_src[:rows], m.pos[:rows]))
    assert off[0] == 0 and off[-1] == rows and np.array_equal(src[pos.reshape(tokens, k)], np.repeat(np.arange(tokens)[:, None], k, 1))
    act, rowsv = n64(m.act[:rows]), n64(m.rows[:rows])
    for e in range(m.experts):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        assert (order[src[lo:hi]] == e).any(1).all()
        a, ea = product(u[src[lo:hi]], n64(d["gate"][e]))
        c, ec = product(u[src[lo:hi]], n64(d["up"][e]))
        silu = a / (1 + np.exp(-a))
        near(m.act[lo:hi], silu * c, 1.1 * ea * (np.abs(c) + ec) + np.abs(silu) * ec + 4e-6 * np.abs(silu * c) + 1e-6, True)
        y, ey = product(act[lo:hi], n64(d["down"][e]))
        near(m.rows[lo:hi], y, ey)
    joined = (weights[:, :, None] * rowsv[pos.reshape(tokens, k)]).sum(1)
    mag = np.abs(n64(h)) + (weights[:, :, None] * np.abs(rowsv[pos.reshape(tokens, k)])).sum(1)
    near(out, n64(h) + joined, 1e-5 * mag)
    hn = n64(h) + joined
    rms = np.sqrt((hn * hn).mean(1, keepdims=True) + 1e-5)
    w = norm(hn, d["final"])
    near(v, w, 1e-5 * (np.abs(n64(d["final"])) * mag / rms + np.abs(w) * (1 + np.sqrt((mag * mag).mean(1, keepdims=True)) / rms)), True)
    logits, b = product(n64(v), n64(d["head"]))
    near(m.logits[:tokens], logits, b)
    z = n64(m.logits[:tokens])
    logp = z - z.max(1, keepdims=True)
    logp -= np.log(np.exp(logp).sum(1, keepdims=True))
    best = np.argsort(-z, axis=1, kind="stable")[:, :5]
    assert np.array_equal(ids.cpu().numpy(), best)
    near(top, np.take_along_axis(logp, best, 1), 2.0 ** -14)
    near(lp, logp[np.arange(tokens), targets.cpu().numpy()], 2.0 ** -14)
    near(ent, -(np.exp(logp) * logp).sum(1), 2.0 ** -12)

    # the same step as one graph, on other inputs
    h2 = torch.randn(tokens, m.dim, device="cuda", generator=g)
    m.block(h2, tokens)
    m.score(tokens, targets, lp, ent, 5, ids, top)
    want = [t.clone() for t in (m.out[:tokens], lp, ent, ids, top)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    x = h.clone()
    with torch.cuda.graph(graph, stream=s):
        m.block(x, tokens)
        m.score(tokens, targets, lp, ent, 5, ids, top)
    x.copy_(h2)
    graph.replay()
    torch.cuda.synchronize()
    for got, w in zip((m.out[:tokens], lp, ent, ids, top), want):
        assert got.dtype == torch.int32 and torch.equal(got, w) or torch.allclose(got.float(), w.float(), rtol=1e-4, atol=1e-4)
