"""A decoder's attention block and its answers, as they are used together on compressed weights: the qkv product, the append
with its rotation, attention, the output product with the residual and norm, the head, edits of its logits and their log
probabilities - for a batch of prompts, then for single tokens, eagerly and as one captured graph.

Each stage is checked against a plain form in 64 bits of what the stage before left.  Products: 1e-4 of the sums of magnitudes, as
the matrices' own tests have it, and half a unit of bf16 (2^-8) for a bf16 output; the others as in their own tests."""
import numpy as np
import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw
from test_gpu_edit import plain as plain_edits
from test_gpu_kv import close, plain_attend, turned

pytestmark = pytest.mark.gpu
F32, BF16, I32, F64 = torch.float32, torch.bfloat16, torch.int32, torch.float64
DIM, HQ, H, D, VOCAB, PAGE = 512, 8, 2, 64, 1003, 16


def compressed(w):
    return uw.Matrix(uw.encode(w.view(torch.int16).numpy().view(np.uint16)), resident="palette")


class Step:
    """The block's weights, cache and buffers for up to `rows` tokens of `seqs` sequences."""

    def __init__(self, rows, seqs, g):
        w = lambda n, k: (torch.randn(n, k, generator=g) * k ** -0.5).to(BF16)  # noqa: E731
        self.w = dict(qkv=w((HQ + 2 * H) * D, DIM), out=w(DIM, HQ * D), head=w(VOCAB, DIM))
        self.m = {k: compressed(v) for k, v in self.w.items()}
        self.norm_w = (1 + 0.1 * torch.randn(DIM, generator=g)).to(BF16).cuda()
        self.norm = uw.BlockNorm(DIM, pre_weight=self.norm_w, res_dtype=uw.OUT_BF16, block_dtype=uw.OUT_F32)
        self.rotary = uw.Rotary(D, base=10000.0, scaling=uw.ROTARY_LINEAR, factor=2.0)
        self.k, self.v = (torch.full((64, PAGE, H, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
        self.cache = uw.KVCache(self.k, self.v)
        z = lambda n, dt: torch.zeros(rows, n, dtype=dt, device="cuda")  # noqa: E731
        self.qkv, self.q, self.att, self.o, self.h2, self.u, self.logits, self.edited = (
            z((HQ + 2 * H) * D, F32), z(HQ * D, BF16), z(HQ * D, BF16), z(DIM, F32), z(DIM, BF16), z(DIM, BF16), z(VOCAB, F32), z(VOCAB, F32))
        self.lp, self.top_lp, self.top = torch.zeros(rows, device="cuda"), torch.zeros(rows, 4, device="cuda"), torch.zeros(rows, 4, dtype=I32, device="cuda")
        self.ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")

    def product(self, name, x, rows, y):
        m = self.m[name]
        need = m.workspace_size(rows)
        m.matmul(x, rows, y, uw.OUT_F32, uw.STRAT_AUTO, self.ws, need)

    def run(self, h, rows, batch, edits, target):
        self.product("qkv", h, rows, self.qkv)
        q, k, v = self.qkv[:rows].view(rows, HQ + 2 * H, D).split([HQ, H, H], 1)
        self.cache.append(batch, rows, k, v, q=q, q_out=self.q[:rows], rotary=self.rotary, dtype=uw.OUT_F32)
        need = self.cache.workspace_size(batch, rows, HQ)
        assert need <= self.ws.numel()
        self.cache.attend(batch, rows, self.q[:rows], self.att[:rows], workspace=self.ws, ws_bytes=need)
        self.product("out", self.att, rows, self.o)
        self.norm.run(rows, h, self.h2, y=self.o, u=self.u)
        self.product("head", self.u, rows, self.logits)
        uw.edit_logits(self.logits, rows, VOCAB, self.edited, **edits)
        uw.token_logprobs(self.edited, rows, VOCAB, self.lp, targets=target, n_top=4, top_ids=self.top, top_logprobs=self.top_lp)

    def check(self, h, rows, positions, seq_of, table, lens, edits, target):
        c = lambda t: t[:rows].cpu()  # noqa: E731

        def product(x, w, y):
            x, w = x.to(F64), w.to(F64)
            assert ((y.to(F64) - x @ w.t()).abs() <= 1e-4 * (x.abs() @ w.abs().t())).all()

        product(h.cpu(), self.w["qkv"], c(self.qkv))
        x = c(self.qkv).view(rows, HQ + 2 * H, D)
        want, mag = turned(x[:, :HQ + H], positions, D, uw.ROTARY_HALF, self.rotary.freq, 1.0)
        close(self.q[:rows].view(rows, HQ, D), want[:, :HQ], mag[:, :HQ])
        for s, n in enumerate(lens):
            mine = (seq_of == s).nonzero()[:, 0]
            k, v = (t[table[s].long().cuda()].reshape(-1, H, D)[:n].cpu() for t in (self.k, self.v))
            at = positions[mine]
            close(k[at], want[mine, HQ:], mag[mine, HQ:])
            assert torch.equal(v[at], x[mine, HQ + H:].to(BF16))
            ref, _, b, _ = plain_attend(c(self.q).view(rows, HQ, D)[mine], k, v, len(mine), D ** -0.5, True, 0)
            assert ((c(self.att).view(rows, HQ, D)[mine].to(F64) - ref).abs() <= b).all()
        product(c(self.att), self.w["out"], c(self.o))
        h2 = h.cpu().to(F64) + c(self.o).to(F64)
        assert ((c(self.h2).to(F64) - h2).abs() <= 2.0 ** -8 * h2.abs() + 1e-5 * (h.cpu().to(F64).abs() + c(self.o).to(F64).abs())).all()
        u = self.norm_w.cpu().to(F64) * h2 / (h2.pow(2).mean(1, keepdim=True) + 1e-5).sqrt()
        assert ((c(self.u).to(F64) - u).abs() <= 2.0 ** -8 * u.abs() + 4e-5 * u.abs().amax()).all()
        product(c(self.u), self.w["head"], c(self.logits))
        e = {k: v.cpu() if v is not None else None for k, v in edits.items()}
        full = dict(R=rows, V=VOCAB, logits=c(self.logits), bias_ids=None, bias=None, bias_lengths=None, **e)
        ref, b, _ = plain_edits(full)
        got, dead = c(self.edited).to(F64), torch.isinf(ref)
        assert torch.equal(torch.isinf(got), dead) and ((got - ref).abs()[~dead] <= b[~dead]).all()
        lp = torch.log_softmax(got, 1)
        t = lp[torch.arange(rows), target.cpu().long()]
        live = ~torch.isinf(t)
        assert torch.equal(torch.isinf(c(self.lp)), ~live) and ((c(self.lp).to(F64) - t).abs()[live] <= 1e-4).all()
        assert ((c(self.top_lp).to(F64) - lp.gather(1, c(self.top).long())).abs() <= 1e-4).all()


def edits_for(rows, g):
    allowed = torch.randint(-2 ** 31, 2 ** 31, (2, (VOCAB + 31) // 32), generator=g, dtype=I32)
    e = dict(tokens=torch.randint(0, VOCAB, (rows, 40), generator=g, dtype=I32), lengths=torch.randint(0, 41, (rows,), generator=g, dtype=I32),
             prompt_lengths=torch.full((rows,), 10, dtype=I32), repetition=1 + torch.rand(rows, generator=g) * 0.2,
             frequency=torch.rand(rows, generator=g), presence=torch.rand(rows, generator=g), allowed=allowed,
             mask_rows=torch.randint(-1, 2, (rows,), generator=g, dtype=I32))
    return {k: v.cuda() for k, v in e.items()}


def test_prompts_then_tokens():
    g = torch.Generator().manual_seed(11)
    prompts = [150, 33, 1]
    st = Step(sum(prompts), len(prompts), g)
    table = torch.randperm(64, generator=g)[:45].to(I32).view(3, 15)
    dt = table.cuda()
    i32 = lambda v: torch.tensor(v, dtype=I32).cuda()  # noqa: E731

    rows = sum(prompts)
    h = torch.randn(rows, DIM, generator=g).to(BF16).cuda()
    batch = uw.KVBatch(i32([0, 150, 183, 184]), i32(prompts), dt)
    edits, target = edits_for(rows, g), torch.randint(0, VOCAB, (rows,), generator=g, dtype=I32).cuda()
    st.run(h, rows, batch, edits, target)
    st.cache.check()
    seq_of = torch.repeat_interleave(torch.arange(3), torch.tensor(prompts))
    positions = torch.cat([torch.arange(n) for n in prompts])
    st.check(h, rows, positions, seq_of, table, prompts, edits, target)

    # single tokens: one eager step, then the same step as a graph, replayed for the tokens that follow
    lengths = i32(prompts)
    batch = uw.KVBatch(i32([0, 1, 2, 3]), lengths, dt)
    edits, target = edits_for(3, g), torch.randint(0, VOCAB, (3,), generator=g, dtype=I32).cuda()
    h = torch.zeros(3, DIM, dtype=BF16, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    for step in range(4):
        h.copy_(torch.randn(3, DIM, generator=g).to(BF16))
        lengths += 1
        torch.cuda.synchronize()
        if step == 0:
            st.run(h, 3, batch, edits, target)
        elif step == 1:
            with torch.cuda.graph(graph, stream=side):
                st.run(h, 3, batch, edits, target)
        if step:
            graph.replay()
        torch.cuda.synchronize()
        lens = [n + step + 1 for n in prompts]
        st.check(h, 3, torch.tensor(lens) - 1, torch.arange(3), table, lens, edits, target)
    st.cache.check()
