"""Operators behind one another without a wait: each begins while the one before it ends and reads what that one wrote.
The same calls with a synchronisation after each give the same bits."""
import pytest

import lossless_bf16_weight_exponent_gb300 as uw

pytestmark = pytest.mark.gpu


# one launch of the router and the matrix-vector product; two launches and tcgen05; the scan between them
@pytest.mark.parametrize("tokens", [5, 700, 60000])
def test_chain_reads_what_the_kernel_before_it_wrote(tokens):
    import torch
    E, k, K, D = 40, 4, 64, 96
    g = torch.Generator(device="cuda").manual_seed(tokens)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    group = uw.Group(randn(E, D, K).bfloat16())
    bias = randn(E)
    router = uw.Router(E, k, bias=bias)
    norm = uw.BlockNorm(D, pre_weight=(1 + 0.1 * randn(D)).bfloat16(), res_dtype=uw.OUT_F32, block_dtype=uw.OUT_F32)
    i32, f32 = torch.int32, torch.float32
    new = lambda *s, t=f32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    ids, weights, pos, src, offsets = new(tokens, k, t=i32), new(tokens, k), new(tokens, k, t=i32), new(tokens * k, t=i32), new(E + 1, t=i32)
    y, h, u = new(tokens * k, D), new(tokens, D), new(tokens, D, t=torch.bfloat16)
    H, top_ids, top = new(tokens), new(tokens, 3, t=i32), new(tokens, 3)
    ws = new(max(16, router.workspace_size(tokens)), t=torch.uint8)
    inputs = [(randn(tokens, E), randn(tokens, K).bfloat16(), randn(tokens, D)) for _ in range(3)]

    def step(logits, x, res, after):
        for call in (lambda: router.route(logits, tokens, ids, weights, offsets, src, pos, workspace=ws, ws_bytes=ws.numel()),
                     lambda: group.matmul(x, offsets, tokens * k, y, row_src=src, out_dtype=uw.OUT_F32),
                     lambda: norm.run(tokens, res, h, y=y, pos=pos, weights=weights, topk=k, y_rows=tokens * k, u=u),
                     lambda: uw.token_logprobs(h, tokens, D, entropy=H, n_top=3, top_ids=top_ids, top_logprobs=top)):
            call()
            after()
        return [t.clone() for t in (ids, weights, offsets, src, pos, y, h, u, H, top_ids, top)]

    alone = [step(*i, torch.cuda.synchronize) for i in inputs]
    behind = [step(*inputs[j % 3], lambda: None) for j in range(30)]
    torch.cuda.synchronize()
    group.check()
    for j, got in enumerate(behind):
        for a, b in zip(alone[j % 3], got):
            assert torch.equal(a, b)
