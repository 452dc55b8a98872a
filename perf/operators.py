"""Cases, inputs and plain forms of the operators that surround the compressed products in a mixture-of-experts
decoder: the router, the experts' grouped products, the norms and residual around a block, and the log probabilities
on the head's logits.

``run`` computes a case in elementary torch operations in 32 bits, or, where ``own`` is true, through the library.
``exact`` computes it from the definition in 64 bits.
"""
import math

import torch

own = False  # set by the caller: run the library's operators instead of the plain forms

F32, BF16 = "f32", "bf16"
_DT = {F32: torch.float32, BF16: torch.bfloat16}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one new token through the gate and up projections of 8 of 64 experts: the latency of decoding
        dict(name="experts_glu_1tok", op="experts", tokens=1, experts=64, topk=8, K=2048, N=1408, glu=True, gather=True, out=BF16),
        # a decode batch through the down projections (K no multiple of 256): a few rows for each expert
        dict(name="experts_down_32tok", op="experts", tokens=32, experts=64, topk=8, K=1408, N=2048, glu=False, gather=False, out=F32),
        # a chunk of a prompt through the gate and up projections: hundreds of rows for each expert, ragged
        dict(name="experts_glu_4096tok", op="experts", tokens=4096, experts=64, topk=8, K=2048, N=1408, glu=True, gather=True, out=BF16),
        # few large experts of the 8B projection's shape, an odd number of tokens
        dict(name="experts_glu_333tok_8b", op="experts", tokens=333, experts=8, topk=2, K=4096, N=14336, glu=True, gather=True, out=BF16),
        # the router of a decode batch, then that of a prompt chunk
        dict(name="route_16tok", op="route", tokens=16, experts=64, topk=8, score="softmax", bias=False, renorm=True, dtype=F32),
        dict(name="route_8191tok", op="route", tokens=8191, experts=128, topk=8, score="sigmoid", bias=True, renorm=True, dtype=BF16),
        # residual and norms around a dense block: one token, and a prompt chunk with a gate for each channel
        dict(name="norm_1tok", op="norm", tokens=1, dim=4096, topk=0, res=BF16, block=BF16, post=False, gate=0, pre=True),
        dict(name="norm_4096tok_gate", op="norm", tokens=4096, dim=4096, topk=0, res=BF16, block=BF16, post=True, gate=4096, pre=True),
        # the experts' rows of each token joined on the way
        dict(name="norm_combine_4096tok", op="norm", tokens=4096, dim=2048, topk=8, res=F32, block=BF16, post=False, gate=0, pre=True),
        # one sampled token with its alternatives; a batch of them; a scored prompt with a padded vocabulary
        dict(name="logprobs_1row_top20", op="logprobs", rows=1, vocab=128256, pad=0, top=20, dtype=F32, masked=False),
        dict(name="logprobs_256rows_top5", op="logprobs", rows=256, vocab=128256, pad=0, top=5, dtype=F32, masked=True),
        dict(name="logprobs_2047rows", op="logprobs", rows=2047, vocab=32003, pad=61, top=0, dtype=BF16, masked=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["experts", "experts", "route", "norm", "logprobs"])
    if op == "experts":
        while True:
            glu = rng.random() < 0.5
            E = _log(rng, 1, 128)
            k = rng.randint(1, min(8, E))
            T, K, N = _log(rng, 1, 4096), 64 * _log(rng, 1, 64), _log(rng, 16, 4096)
            if E * K * N * (2 if glu else 1) <= 380e6 and T * k * K * N * (2 if glu else 1) <= 180e9:
                break
        return dict(op=op, tokens=T, experts=E, topk=k, K=K, N=N, glu=glu, gather=rng.random() < 0.5, out=rng.choice([F32, BF16]))
    if op == "route":
        E = _log(rng, 2, 256)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=E, topk=rng.randint(1, min(8, E)), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, renorm=rng.random() < 0.5, dtype=rng.choice([F32, BF16]))
    if op == "norm":
        T, D = _log(rng, 1, 8192), _log(rng, 64, 8192)
        return dict(op=op, tokens=T, dim=D, topk=rng.choice([0, 0, 1, 2, 4, 8]), res=rng.choice([F32, BF16]), block=rng.choice([F32, BF16]),
                    post=rng.random() < 0.5, gate=rng.choice([0, 1, T, max(1, T // 3)]), pre=rng.random() < 0.8)
    V = _log(rng, 200, 200000)
    return dict(op="logprobs", rows=min(_log(rng, 1, 2048), max(1, 60_000_000 // V)), vocab=V, pad=rng.choice([0, 0, 1, 64]),
                top=rng.choice([0, 1, 5, 20]), dtype=rng.choice([F32, BF16]), masked=rng.random() < 0.5)


def work(c):
    es = {F32: 4, BF16: 2}
    if c["op"] == "experts":
        T, E, k, K, N = c["tokens"], c["experts"], c["topk"], c["K"], c["N"]
        m = 2 if c["glu"] else 1
        active = E * (1.0 - (1.0 - k / E) ** T)  # experts that get rows, when all are as likely
        rows = T * k
        weights = active * N * K * m * 1.5  # a sign+mantissa byte and four bits of exponent for each weight
        return {"bytes": int(weights + (T if c["gather"] else rows) * K * 2 + rows * N * es[c["out"]] + rows * 4), "flops": 2 * rows * K * N * m}
    if c["op"] == "route":
        T, E, k = c["tokens"], c["experts"], c["topk"]
        return {"bytes": T * E * es[c["dtype"]] + T * k * 16 + 4 * E, "flops": T * E * 4}
    if c["op"] == "norm":
        T, D, k = c["tokens"], c["dim"], c["topk"]
        n = T * D * (2 * es[c["res"]] + max(1, k) * es[c["block"]] + (2 if c["pre"] else 0)) + T * k * 8
        n += 2 * D * (c["post"] + c["pre"]) + (2 * D * -(-T // c["gate"]) if c["gate"] else 0)
        return {"bytes": n, "flops": T * D * (8 + 2 * k)}
    return {"bytes": c["rows"] * (c["vocab"] * es[c["dtype"]] + 12 + 8 * c["top"]), "flops": c["rows"] * c["vocab"] * 6}


# ------------------------------------------------------------------------------------------------ inputs
def _inputs(c, seed):
    """The case's tensors on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, scale, generator=g)
        return t if dtype == torch.float32 else t.to(dtype)

    def uniform(*shape):
        return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(0.0, 1.0, generator=g)

    if c["op"] == "experts":
        T, E, k, K, N = c["tokens"], c["experts"], c["topk"], c["K"], c["N"]
        # tokens choose k experts each, some experts more popular than others; rows sorted by expert
        score = normal(T, E, dtype=torch.float32) + 0.4 * normal(E, dtype=torch.float32)
        ids = torch.topk(score, k, dim=1).indices.reshape(-1)
        order = torch.sort(ids, stable=True).indices
        counts = torch.bincount(ids, minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.cumsum(counts, 0)

        def weights():  # trained weights' bulk and a few large ones
            w = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
            for e in range(E):
                t = normal(N, K, scale=0.02, dtype=torch.float32)
                n = max(1, N * K // 10000)
                t.view(-1)[torch.randint(0, N * K, (n,), generator=g, device="cuda")] *= 100.0
                w[e] = t
            return w

        s = dict(x=normal(T if c["gather"] else T * k, K), offsets=offsets, counts=counts.tolist(), w=weights(),
                 src=(order // k).to(torch.int32) if c["gather"] else None)
        s["w_up"] = weights() if c["glu"] else None
        return s
    if c["op"] == "route":
        T, E = c["tokens"], c["experts"]
        return dict(logits=(normal(T, E, dtype=torch.float32) * 1.5 + normal(E, dtype=torch.float32) * 0.5).to(_DT[c["dtype"]]),
                    bias=normal(E, scale=0.3, dtype=torch.float32) if c["bias"] else None)
    if c["op"] == "norm":
        T, D, k = c["tokens"], c["dim"], c["topk"]
        s = dict(h=normal(T, D, scale=2.0, dtype=_DT[c["res"]]), y=normal(T * max(1, k), D, dtype=_DT[c["block"]]), pos=None, p=None)
        if k:
            s["pos"] = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
            s["p"] = torch.softmax(normal(T, k, dtype=torch.float32), 1)
        s["post_w"] = (1.0 + normal(D, scale=0.2, dtype=torch.float32)).bfloat16() if c["post"] else None
        s["pre_w"] = (1.0 + normal(D, scale=0.2, dtype=torch.float32)).bfloat16() if c["pre"] else None
        s["gate"] = normal(-(-T // c["gate"]), D, scale=0.5) if c["gate"] else None  # one row for each `gate` tokens
        s["a"], s["s"], s["eps"] = 1.0, 0.75, 1e-5
        return s
    R, V = c["rows"], c["vocab"]
    full = normal(R, V + c["pad"], scale=2.5, dtype=torch.float32)
    if c["masked"]:  # every third row is restricted to a grammar's few tokens
        allowed = uniform(R, V + c["pad"]) < 0.02
        allowed[:, 7] = True
        full[::3] = torch.where(allowed[::3], full[::3], torch.full_like(full[::3], -math.inf))
    target = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    return dict(logits=full.to(_DT[c["dtype"]]), target=target, temperature=0.8)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = c = case
    if not own:
        return s
    import lossless_bf16_weight_exponent_gb300 as uw
    dev, f32, i32 = "cuda", torch.float32, torch.int32
    dt = {F32: uw.OUT_F32, BF16: uw.OUT_BF16}
    if c["op"] == "experts":
        rows = c["tokens"] * c["topk"]
        s["group"] = uw.Group(s.pop("w"), s.pop("w_up"))
        s["y"] = torch.empty(rows, c["N"], dtype=_DT[c["out"]], device=dev)
        s["out"] = dt[c["out"]]
    elif c["op"] == "route":
        T, k = c["tokens"], c["topk"]
        s["ids"], s["src"], s["pos"] = (torch.empty(n, dtype=i32, device=dev) for n in ((T, k), (T * k,), (T, k)))
        s["weights"] = torch.empty(T, k, dtype=f32, device=dev)
        s["offsets"] = torch.empty(c["experts"] + 1, dtype=i32, device=dev)
        s["router"] = uw.Router(c["experts"], k, score=uw.SCORE_SIGMOID if c["score"] == "sigmoid" else uw.SCORE_SOFTMAX, bias=s["bias"],
                                renormalize=c["renorm"])
        s["ws_bytes"] = s["router"].workspace_size(T)
        s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device=dev)
        s["dt"] = dt[c["dtype"]]
    elif c["op"] == "norm":
        T, D = c["tokens"], c["dim"]
        s["h_out"] = torch.empty_like(s["h"])
        s["u"] = torch.empty(T, D, dtype=torch.bfloat16, device=dev) if c["pre"] else None
        s["norm"] = uw.BlockNorm(D, post_weight=s["post_w"], gate=s["gate"], gate_every=c["gate"], pre_weight=s["pre_w"], res_scale=s["a"],
                                 out_scale=s["s"], eps=s["eps"], res_dtype=dt[c["res"]], block_dtype=dt[c["block"]])
    else:
        R, n = c["rows"], c["top"]
        s["lp"], s["entropy"] = torch.empty(R, dtype=f32, device=dev), torch.empty(R, dtype=f32, device=dev)
        s["top_ids"] = torch.empty(R, n, dtype=i32, device=dev)
        s["top_lp"] = torch.empty(R, n, dtype=f32, device=dev)
        s["dt"] = dt[c["dtype"]]
    return s


# ------------------------------------------------------------------------------------------------ one pass
def _run_own(s):
    import lossless_bf16_weight_exponent_gb300 as uw
    c = s["case"]
    if c["op"] == "experts":
        s["group"].matmul(s["x"], s["offsets"], c["tokens"] * c["topk"], s["y"], row_src=s["src"], x_rows=s["x"].shape[0], out_dtype=s["out"])
        return s["y"]
    if c["op"] == "route":
        s["router"].route(s["logits"], c["tokens"], s["ids"], s["weights"], s["offsets"], s["src"], s["pos"], dtype=s["dt"], workspace=s["ws"],
                          ws_bytes=s["ws_bytes"])
        return [s["ids"], s["weights"], s["offsets"], s["src"], s["pos"]]
    if c["op"] == "norm":
        s["norm"].run(c["tokens"], s["h"], s["h_out"], y=s["y"], pos=s["pos"], weights=s["p"], topk=c["topk"], y_rows=s["y"].shape[0], u=s["u"])
        return [s["h_out"]] + ([s["u"]] if c["pre"] else [])
    uw.token_logprobs(s["logits"], c["rows"], c["vocab"], s["lp"], targets=s["target"], entropy=s["entropy"], n_top=c["top"],
                      top_ids=s["top_ids"], top_logprobs=s["top_lp"], dtype=s["dt"], ld=c["vocab"] + c["pad"], temperature=s["temperature"])
    return [s["lp"], s["entropy"]] + ([s["top_ids"], s["top_lp"]] if c["top"] else [])


def _silu(t):
    return t / (1.0 + torch.exp(-t))


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "experts":
        y = torch.empty(c["tokens"] * c["topk"], c["N"], dtype=_DT[c["out"]], device="cuda")
        at = 0
        for e, n in enumerate(s["counts"]):  # one product for each expert that has rows
            if not n:
                continue
            x = (s["x"][s["src"][at:at + n]] if c["gather"] else s["x"][at:at + n]).float()
            r = x @ s["w"][e].float().t()
            if c["glu"]:
                r = _silu(r) * (x @ s["w_up"][e].float().t())
            y[at:at + n] = r
            at += n
        return y
    if c["op"] == "route":
        T, E, k = c["tokens"], c["experts"], c["topk"]
        z = s["logits"].float()
        key = z + s["bias"] if c["bias"] else z
        ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
        if c["score"] == "softmax":
            e = torch.exp(z - z.amax(1, keepdim=True))
            p = e / e.sum(1, keepdim=True)
        else:
            p = 1.0 / (1.0 + torch.exp(-z))
        w = torch.gather(p, 1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        flat = ids.reshape(-1)
        order = torch.sort(flat, stable=True).indices
        pos = torch.empty_like(order)
        pos[order] = torch.arange(T * k, device="cuda")
        offsets = (flat[None, :] < torch.arange(E + 1, device="cuda")[:, None]).sum(1)
        i32 = torch.int32
        return [ids.to(i32), w, offsets.to(i32), (order // k).to(i32), pos.view(T, k).to(i32)]
    if c["op"] == "norm":
        T, D, k = c["tokens"], c["dim"], c["topk"]
        o = s["y"].float() if not k else (s["y"].float()[s["pos"].reshape(-1)].view(T, k, D) * s["p"][:, :, None]).sum(1)
        if c["post"]:
            o = o * torch.rsqrt((o * o).mean(1, keepdim=True) + s["eps"]) * s["post_w"].float()
        if c["gate"]:
            o = o * s["gate"].float()[torch.arange(T, device="cuda") // c["gate"]]
        h = s["a"] * s["h"].float() + s["s"] * o
        if not c["pre"]:
            return [h.to(_DT[c["res"]])]
        u = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["pre_w"].float()
        return [h.to(_DT[c["res"]]), u.bfloat16()]
    x = s["logits"][:, :c["vocab"]].float()
    z = x * (1.0 / s["temperature"])
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    lp = torch.gather(z, 1, s["target"].long()[:, None]) - lse
    entropy = lse[:, 0] - torch.where(e > 0, e * z, 0.0).sum(1) / total[:, 0]
    if not c["top"]:
        return [lp[:, 0], entropy]
    top = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top"]]
    return [lp[:, 0], entropy, top.to(torch.int32), torch.gather(z, 1, top) - lse]


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The case's outputs from the definitions, in 64 bits; None in the place of whole-number outputs."""
    c, s = case, _inputs(case, seed)
    f = torch.float64
    if c["op"] == "experts":
        rows, E = c["tokens"] * c["topk"], c["experts"]
        out = torch.zeros(rows, c["N"], dtype=f, device="cuda")
        which = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(s["counts"], device="cuda"))
        token = s["src"].long() if c["gather"] else torch.arange(rows, device="cuda")
        for e in which.unique().tolist():
            mine = (which == e).nonzero()[:, 0]
            x = s["x"][token[mine]].to(f)
            a = torch.einsum("rk,nk->rn", x, s["w"][e].to(f))
            out[mine] = a * torch.sigmoid(a) * torch.einsum("rk,nk->rn", x, s["w_up"][e].to(f)) if c["glu"] else a
        return out
    if c["op"] == "route":
        z = s["logits"].to(f)
        key = z.float() + s["bias"] if c["bias"] else z
        left, picked = key.double().clone(), []
        for _ in range(c["topk"]):  # the largest that is left, the lowest index of equals
            best = left.max(1, keepdim=True).values
            first = torch.where(left == best, torch.arange(c["experts"], device="cuda"), c["experts"]).amin(1, keepdim=True)
            picked.append(first)
            left.scatter_(1, first, -math.inf)
        ids = torch.cat(picked, 1)
        p = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
        w = p.gather(1, ids)
        return [None, w / w.sum(1, keepdim=True) if c["renorm"] else w, None, None, None]
    if c["op"] == "norm":
        T, k = c["tokens"], c["topk"]
        o = s["y"].to(f) if not k else sum(s["p"][:, j, None].to(f) * s["y"][s["pos"][:, j].long()].to(f) for j in range(k))
        if c["post"]:
            o = s["post_w"].to(f) * (o / (o.pow(2).mean(1) + s["eps"]).sqrt()[:, None])
        if c["gate"]:
            o = o * torch.repeat_interleave(s["gate"].to(f), c["gate"], 0)[:T]
        h = s["h"].to(f) * s["a"] + o * s["s"]
        u = s["pre_w"].to(f) * (h / (h.pow(2).mean(1) + s["eps"]).sqrt()[:, None]) if c["pre"] else None
        return [h] + ([u] if c["pre"] else [])
    z = s["logits"][:, :c["vocab"]].to(f) / s["temperature"]
    logp = torch.log_softmax(z, 1)
    lp = logp[torch.arange(c["rows"], device="cuda"), s["target"].long()]
    entropy = -(logp.exp() * logp.nan_to_num(neginf=0.0)).sum(1)
    if not c["top"]:
        return [lp, entropy]
    return [lp, entropy, None, torch.sort(logp, 1, descending=True).values[:, :c["top"]]]
