"""One mixture-of-experts block and the head of a decoder on losslessly compressed weights.

    python examples/moe_block.py [tokens]

Builds synthetic weights, compresses them, runs the block for a prompt and then, captured into one CUDA graph, for
single tokens, and prints the time of a step and the log probabilities of the chosen tokens with their alternatives.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import lossless_bf16_weight_exponent_gb300 as uw  # noqa: E402


def _weights(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * shape[-1] ** -0.5).bfloat16()


def _compress(w):
    return uw.Matrix(uw.encode(w.view(torch.int16).cpu().numpy().view("uint16")))


class MoeBlock:
    """norm -> router -> experts -> their weighted sum into the residual, and the norm in front of what follows; the
    head's log probabilities.  Buffers for up to max_tokens are made once."""

    def __init__(self, dim=512, hidden=704, experts=16, topk=4, vocab=5003, max_tokens=256, seed=1):
        self.dim, self.hidden, self.experts, self.topk, self.vocab = dim, hidden, experts, topk, vocab
        w = self.dense = dict(router=_weights(experts, dim, seed=seed), gate=_weights(experts, hidden, dim, seed=seed + 1),
                              up=_weights(experts, hidden, dim, seed=seed + 2), down=_weights(experts, dim, hidden, seed=seed + 3),
                              head=_weights(vocab, dim, seed=seed + 4), norm=1 + _weights(dim, seed=seed + 5).float(),
                              final=1 + _weights(dim, seed=seed + 6).float())
        w["norm"], w["final"] = w["norm"].bfloat16(), w["final"].bfloat16()
        # compressed: the router and the head as single matrices, the experts as groups
        self.router_w, self.head_w = _compress(w["router"]), _compress(w["head"])
        self.gate_up, self.down = uw.Group(w["gate"], w["up"]), uw.Group(w["down"])
        self.router = uw.Router(experts, topk)
        self.first = uw.BlockNorm(dim, pre_weight=w["norm"], res_dtype=uw.OUT_F32)
        self.join = uw.BlockNorm(dim, pre_weight=w["final"], res_dtype=uw.OUT_F32, block_dtype=uw.OUT_F32)
        n, f32, bf16, i32 = max_tokens, torch.float32, torch.bfloat16, torch.int32
        new = lambda *s, t=f32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        self.u, self.router_logits = new(n, dim, t=bf16), new(n, experts)
        self.ids, self.weights, self.offsets = new(n * topk, t=i32), new(n * topk), new(experts + 1, t=i32)
        self.row_src, self.pos = new(n * topk, t=i32), new(n * topk, t=i32)
        self.act, self.rows = new(n * topk, hidden, t=bf16), new(n * topk, dim)
        self.out, self.v, self.logits = new(n, dim), new(n, dim, t=bf16), new(n, vocab)
        self.route_ws = new(max(16, self.router.workspace_size(n)), t=torch.uint8)
        self.matmul_ws = new(max(m.workspace_size(b) for m in (self.router_w, self.head_w) for b in (1, n)), t=torch.uint8)

    def block(self, h, tokens):
        """h: fp32 [tokens, dim], the residual stream; returns it after the block, and the next block's normed input."""
        ws = self.matmul_ws
        self.first.run(tokens, h, None, u=self.u)
        self.router_w.matmul(self.u, tokens, self.router_logits, workspace=ws, ws_bytes=ws.numel())
        self.router.route(self.router_logits, tokens, self.ids, self.weights, self.offsets, self.row_src, self.pos,
                          workspace=self.route_ws, ws_bytes=self.route_ws.numel())
        rows = tokens * self.topk
        self.gate_up.matmul(self.u, self.offsets, rows, self.act, row_src=self.row_src, x_rows=tokens)
        self.down.matmul(self.act, self.offsets, rows, self.rows, x_rows=rows, out_dtype=uw.OUT_F32)
        self.join.run(tokens, h, self.out, y=self.rows, pos=self.pos, weights=self.weights, topk=self.topk, y_rows=rows, u=self.v)
        return self.out[:tokens], self.v[:tokens]

    def score(self, tokens, targets, logprob, entropy=None, n_top=0, top_ids=None, top_logprobs=None, temperature=1.0):
        """Log probabilities of `targets` under the head, on what block() left."""
        ws = self.matmul_ws
        self.head_w.matmul(self.v, tokens, self.logits, workspace=ws, ws_bytes=ws.numel())
        uw.token_logprobs(self.logits, tokens, self.vocab, logprob, targets, entropy, n_top, top_ids, top_logprobs,
                          temperature=temperature)


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 200
    m = MoeBlock(max_tokens=max(tokens, 1))
    h = torch.randn(tokens, m.dim, device="cuda")
    targets = torch.randint(0, m.vocab, (tokens,), dtype=torch.int32, device="cuda")
    lp, ent = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    ids, top = torch.empty(tokens, 5, dtype=torch.int32, device="cuda"), torch.empty(tokens, 5, device="cuda")
    m.block(h, tokens)
    m.score(tokens, targets, lp, ent, 5, ids, top)
    print(f"{tokens} tokens: mean log probability {lp.mean().item():.4f}, mean entropy {ent.mean().item():.4f}")
    print("rows per expert:", (m.offsets[1:] - m.offsets[:-1]).tolist())

    # one token at a time: the whole step in one graph
    step = lambda: (m.block(h[:1], 1), m.score(1, targets, lp, ent, 5, ids, top))  # noqa: E731
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(5):
        graph.replay()
    a.record()
    for _ in range(100):
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    print(f"one token: {a.elapsed_time(b) * 10:.1f} us a step; alternatives", list(zip(ids[0].tolist(), [round(v, 4) for v in top[0].tolist()])))


if __name__ == "__main__":
    main()
