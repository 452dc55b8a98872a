"""Cases, inputs and plain forms of the operators of a decoder's attention and of its answers: keys and values rotated
and appended to a paged cache, attention of new tokens over that cache, and the edits of logits before a token is chosen.

``run`` computes a case in elementary torch operations in 32 bits (the rotation's angles in 64), or, where ``own`` is
true, through the library.  ``exact`` computes it from the definition in 64 bits.
"""
import math
import random

import torch

own = False  # set by the caller: run the library's operators instead of the plain forms

F32, BF16 = "f32", "bf16"
_DT = {F32: torch.float32, BF16: torch.bfloat16}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of one sequence, as the qkv product of an 8B layer leaves it: the latency of decoding
        dict(name="append_1tok", op="append", seqs=1, few=1, past=4000, ragged=False, q_heads=32, kv_heads=8, dim=128, page=64, heads_first=False, dtype=F32,
             rot=128, layout="half", scaling="none"),
        # a decode batch with a 70B layer's heads, pairs side by side, half of the head rotated
        dict(name="append_253seqs", op="append", seqs=253, few=1, past=1009, ragged=True, q_heads=64, kv_heads=8, dim=128, page=16,
             heads_first=False, dtype=BF16, rot=64, layout="interleaved", scaling="none"),
        # a chunk of a long prompt, far behind its beginning, frequencies scaled for long contexts
        dict(name="append_4096tok_far", op="append", seqs=1, few=4096, past=24575, ragged=False, q_heads=32, kv_heads=8, dim=128, page=64, heads_first=True, dtype=BF16,
             rot=128, layout="half", scaling="bands"),
        # one token of one sequence, 8k tokens of context
        dict(name="attend_1tok_8k", op="attend", seqs=1, few=1, past=8190, ragged=False, q_heads=32, kv_heads=8, dim=128, page=64, heads_first=False, causal=True,
             window=0),
        # a decode batch of ragged contexts
        dict(name="attend_64seqs", op="attend", seqs=64, few=1, past=8191, ragged=True, q_heads=32, kv_heads=8, dim=128, page=16,
             heads_first=False, causal=True, window=0),
        # one sequence of a very long context, a few drafted tokens to verify
        dict(name="attend_4tok_128k", op="attend", seqs=1, few=4, past=131067, ragged=False, q_heads=64, kv_heads=8, dim=128, page=128, heads_first=True, causal=True,
             window=0),
        # a chunk of a prompt over what came before it, an odd number of tokens
        dict(name="attend_509tok_over_7k", op="attend", seqs=1, few=509, past=7171, ragged=False, q_heads=64, kv_heads=8, dim=128, page=64, heads_first=False,
             causal=True, window=0),
        # a whole prompt
        dict(name="attend_8191tok", op="attend", seqs=1, few=8191, past=0, ragged=False, q_heads=32, kv_heads=8, dim=128, page=64, heads_first=False, causal=True,
             window=0),
        # a mixed batch: two prompts' chunks beside decoding sequences, heads of 64, a window
        dict(name="attend_mixed_window", op="attend", seqs=48, few=1, past=6000, ragged=True, chunks=2, chunk=755, q_heads=32,
             kv_heads=4, dim=64, page=32, heads_first=False, causal=True, window=1024),
        # the next token of one sequence with penalties on its 4000 tokens
        dict(name="logits_1row", op="logits", rows=1, vocab=128256, pad=0, history=4000, prompt=1500, bias=8, masked=0.0, dtype=F32),
        # a batch, every second row under a grammar
        dict(name="logits_256rows", op="logits", rows=256, vocab=128256, pad=0, history=3001, prompt=2000, bias=0, masked=0.5, dtype=F32),
        # bf16 logits of a smaller, padded vocabulary, with biases
        dict(name="logits_96rows_bf16", op="logits", rows=96, vocab=32003, pad=61, history=700, prompt=500, bias=300, masked=1.0, dtype=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(c):
    """New and earlier tokens of each sequence: `few` new ones each, `chunk` in the first `chunks` and none in the last `idle`;
    `past` earlier ones, or, ragged, up to as many."""
    rng = random.Random(c.get("mix", 1))
    S, chunks, idle = c["seqs"], c.get("chunks", 0), c.get("idle", 0)
    new = [c["chunk"] if i < chunks else 0 if i >= S - idle else c["few"] for i in range(S)]
    return new, [rng.randint(0, c["past"]) if c["ragged"] else c["past"] for _ in range(S)]


def _pairs(c):
    """(row, key) pairs that attention sees for each query head."""
    n = 0
    for new, past in zip(*_lengths(c)):
        if not c["causal"]:
            n += new * (new + past)
        elif not c["window"]:
            n += new * past + new * (new + 1) // 2
        else:
            n += sum(min(past + i + 1, c["window"]) for i in range(new))
    return n


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "logits"])
    if op == "logits":
        V = _log(rng, 200, 200000)
        rows = min(_log(rng, 1, 512), max(1, 32_000_000 // V))
        n = _log(rng, 1, 4096)
        return dict(op=op, rows=rows, vocab=V, pad=rng.choice([0, 0, 1, 64]), history=n, prompt=rng.randint(0, n), bias=rng.choice([0, 0, 5, 200]),
                    masked=rng.choice([0.0, 0.5, 1.0]), dtype=rng.choice([F32, BF16]))
    kv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, q_heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv, dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]),
             heads_first=rng.random() < 0.5)
    c.update(mix=rng.randrange(1 << 20), ragged=rng.random() < 0.7)
    if op == "append":
        S = _log(rng, 1, 64)
        c.update(seqs=S, few=_log(rng, 1, max(1, 4096 // S)), past=_log(rng, 1, 16384 // S) - 1, idle=rng.choice([0, 0, S // 4]), dtype=rng.choice([F32, BF16]))
        c.update(rot=c["dim"] // rng.choice([1, 1, 2, 4]), layout=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "stretched", "bands", "ramp"]))
        return c
    kind = rng.choice(["decode", "decode", "chunk", "mixed"])
    while True:
        S = _log(rng, 1, 128) if kind == "decode" else rng.choice([1, 1, 2, 3]) if kind == "chunk" else _log(rng, 2, 48)
        c.update(seqs=S, few=_log(rng, 16, 4096) if kind == "chunk" else rng.choice([1, 1, 1, 2, 5]), past=_log(rng, 1, 32768) - 1)
        if kind == "mixed":
            c.update(chunks=rng.randint(1, min(S, 4)), chunk=_log(rng, 2, 1024))
        if kind == "decode":
            c.update(idle=rng.choice([0, 0, S // 3]))
        c.update(causal=rng.random() < 0.85, window=0)
        if c["causal"] and rng.random() < 0.25:
            c["window"] = _log(rng, 16, 4096)
        new, past = _lengths(c)
        if ((sum(new) + sum(past)) * kv * c["dim"] * 4 <= 500e6 and _pairs(c) * c["q_heads"] * c["dim"] * 4 <= 250e9
                and sum(n * (n + p) for n, p in zip(new, past)) * c["q_heads"] <= 1.2e9):
            return c


def work(c):
    es = {F32: 4, BF16: 2}
    if c["op"] == "append":
        T = sum(_lengths(c)[0])
        n = T * (c["q_heads"] + 2 * c["kv_heads"]) * c["dim"]
        return {"bytes": n * (es[c["dtype"]] + 2), "flops": T * (c["q_heads"] + c["kv_heads"]) * c["rot"] * 3}
    if c["op"] == "attend":
        lengths = _lengths(c)
        T, keys = sum(lengths[0]), 0
        for new, past in zip(*lengths):
            if new:
                keys += min(new + past, new + c["window"] - 1) if c["window"] else new + past
        return {"bytes": keys * c["kv_heads"] * c["dim"] * 4 + T * c["q_heads"] * (c["dim"] * 4 + 4),
                "flops": _pairs(c) * c["q_heads"] * c["dim"] * 4}
    R, V = c["rows"], c["vocab"]
    return {"bytes": R * (2 * V * es[c["dtype"]] + 4 * c["history"] + 8 * c["bias"] + 20) + int(R * c["masked"]) * V // 8, "flops": R * V}


# ------------------------------------------------------------------------------------------------ inputs
def _inputs(c, seed):
    """The case's tensors on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)
    i32 = dict(dtype=torch.int32, device="cuda")

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, scale, generator=g)
        return t if dtype == torch.float32 else t.to(dtype)

    if c["op"] == "logits":
        R, V, n = c["rows"], c["vocab"], c["history"]
        s = dict(logits=normal(R, V + c["pad"], scale=2.5, dtype=torch.float32).to(_DT[c["dtype"]]))
        # text repeats its frequent tokens: ids fall off as a power
        u = torch.empty(R, n, dtype=torch.float32, device="cuda").uniform_(0.0, 1.0, generator=g)
        s["tokens"] = ((V * u ** 3).long().clamp(max=V - 1) * 7919 % V).to(torch.int32)
        s["lengths"] = torch.randint(n // 2, n + 1, (R,), generator=g, **i32)
        s["lengths"][R - 1] = n
        s["prompts"] = torch.minimum(torch.full((R,), c["prompt"], **i32), s["lengths"])
        s["repetition"] = 1.0 + 0.3 * torch.empty(R, device="cuda").uniform_(0.0, 1.0, generator=g)
        s["frequency"], s["presence"] = (torch.empty(R, device="cuda").uniform_(0.0, 0.8, generator=g) for _ in range(2))
        s["bias_ids"], s["bias"] = (torch.randint(0, V, (R, c["bias"]), generator=g, **i32), normal(R, c["bias"], scale=3.0, dtype=torch.float32)) if c["bias"] else (None, None)
        rows = int(round(R * c["masked"]))
        s["allowed"], s["mask_rows"] = None, None
        if rows:
            s["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (rows, (V + 31) // 32), generator=g, **i32)
            s["allowed"] &= torch.randint(-2 ** 31, 2 ** 31, (rows, (V + 31) // 32), generator=g, **i32)
            s["mask_rows"] = torch.full((R,), -1, **i32)  # which row of `allowed` holds for a row of logits
            s["mask_rows"][torch.arange(rows, device="cuda") * R // rows] = torch.arange(rows, **i32)
        return s
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    new, past = _lengths(c)
    S, T = len(new), sum(new)
    held = [-(-(a + b) // P) for a, b in zip(new, past)]  # pages of each sequence
    pages = sum(held) + 3  # and a few that are free
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, max(1, max(held))), -1, **i32)
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)

    def cache():
        return normal(pages, H, P, D).transpose(1, 2) if c["heads_first"] else normal(pages, P, H, D)  # [page, slot, head, element]

    s = dict(new=new, past=past, rows=T, table=table, starts=torch.tensor(starts, **i32), lengths=torch.tensor([a + b for a, b in zip(new, past)], **i32), k=cache(), v=cache())
    if c["op"] == "append":
        s["qkv"] = normal(T, (c["q_heads"] + 2 * H) * D, dtype=_DT[c["dtype"]])  # one product's output
        where = [(a, p) for a, (n, b) in enumerate(zip(new, past)) for p in range(b, b + n)]
        s["seq"], s["position"] = (torch.tensor([w[j] for w in where], dtype=torch.int64, device="cuda") for j in range(2))
    else:
        s["q"] = normal(T, c["q_heads"], D, scale=1.5)
    return s


def _groups(s):
    """The sequences with as many new tokens together: their indices, their rows one after the other, and the most keys of one."""
    groups = []
    for n in sorted(set(s["new"]) - {0}):
        seqs = [i for i, m in enumerate(s["new"]) if m == n]
        at = s["starts"][torch.tensor(seqs, device="cuda")].long()
        groups.append(dict(new=n, keys=max(n + s["past"][i] for i in seqs), seqs=torch.tensor(seqs, device="cuda"),
                           rows=(at[:, None] + torch.arange(n, device="cuda")).reshape(-1)))
    return groups


_ROTARY = dict(base=500000.0, factor=8.0, low=1.0, high=4.0, fast=32.0, slow=1.0, original=8192)


def _rotary_args(uw, c):
    kind = {"none": uw.ROTARY_PLAIN, "linear": uw.ROTARY_LINEAR, "stretched": uw.ROTARY_STRETCHED, "bands": uw.ROTARY_BANDS, "ramp": uw.ROTARY_RAMP}
    r = _ROTARY
    a = dict(base=r["base"], layout=uw.ROTARY_INTERLEAVED if c["layout"] == "interleaved" else uw.ROTARY_HALF, scaling=kind[c["scaling"]])
    if c["scaling"] != "none":
        a["factor"] = r["factor"]
    if c["scaling"] == "bands":
        a.update(low=r["low"], high=r["high"], original=r["original"])
    if c["scaling"] == "ramp":
        a.update(low=r["slow"], high=r["fast"], original=r["original"])
    return a


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = c = case
    if not own:
        if c["op"] == "append":
            s["freq"], s["scale"] = _frequencies(c)
        elif c["op"] == "attend":
            s["groups"] = _groups(s)
        return s
    import lossless_bf16_weight_exponent_gb300 as uw
    dt = {F32: uw.OUT_F32, BF16: uw.OUT_BF16}
    if c["op"] == "logits":
        s["out"] = torch.empty(c["rows"], c["vocab"], dtype=_DT[c["dtype"]], device="cuda")
        s["dt"] = dt[c["dtype"]]
        return s
    s["cache"] = uw.KVCache(s["k"], s["v"])
    s["batch"] = uw.KVBatch(s["starts"], s["lengths"], s["table"])
    T, Hq, H, D = s["rows"], c["q_heads"], c["kv_heads"], c["dim"]
    s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    if c["op"] == "append":
        s["rotary"] = uw.Rotary(c["rot"], **_rotary_args(uw, c))
        s["parts"] = s["qkv"].view(T, Hq + 2 * H, D).split([Hq, H, H], 1)
        s["dt"] = dt[c["dtype"]]
    else:
        s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device="cuda")
        s["ws_bytes"] = s["cache"].workspace_size(s["batch"], T, Hq)
        s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ one pass
def _run_own(s):
    import lossless_bf16_weight_exponent_gb300 as uw
    c = s["case"]
    if c["op"] == "append":
        q, k, v = s["parts"]
        s["cache"].append(s["batch"], s["rows"], k, v, q=q, q_out=s["out"], rotary=s["rotary"], dtype=s["dt"])
        return [s["out"], s["k"], s["v"]]
    if c["op"] == "attend":
        s["cache"].attend(s["batch"], s["rows"], s["q"], s["out"], causal=c["causal"], window=c["window"], lse=s["lse"], workspace=s["ws"],
                          ws_bytes=s["ws_bytes"])
        return [s["out"], s["lse"]]
    uw.edit_logits(s["logits"], c["rows"], c["vocab"], s["out"], tokens=s["tokens"], lengths=s["lengths"], prompt_lengths=s["prompts"],
                   repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"], bias=s["bias"],
                   allowed=s["allowed"], mask_rows=s["mask_rows"], dtype=s["dt"], out_dtype=s["dt"])
    return s["out"]


def _frequencies(c):
    """Frequencies in radians a position, 64 bits, and the factor on cos and sin."""
    d, r = c["rot"], _ROTARY
    m = torch.arange(0, d, 2, dtype=torch.float64, device="cuda")
    base, s = r["base"], r["factor"]
    if c["scaling"] == "stretched":
        base = base * s ** (d / (d - 2)) if d > 2 else base
    f = base ** (-m / d)
    if c["scaling"] == "linear":
        return f / s, 1.0
    if c["scaling"] == "bands":
        keep = ((r["original"] * f / (2 * math.pi) - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
        return keep * f + (1 - keep) * f / s, 1.0
    if c["scaling"] == "ramp":  # by the index of the pair whose angle makes so many turns over the original length
        at = [d * math.log(r["original"] / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (r["fast"], r["slow"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
        keep = 1 - ((m / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return keep * f + (1 - keep) * f / s, 0.1 * math.log(s) + 1.0
    return f, 1.0


def _rotate(x, cos, sin, layout):
    """x [tokens, heads, dims] with cos and sin [tokens, 1, dims / 2]."""
    if layout == "half":
        a, b = x.chunk(2, dim=2)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], 2)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], 3).flatten(2)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "append":
        T, Hq, H, D, rot, P = s["rows"], c["q_heads"], c["kv_heads"], c["dim"], c["rot"], c["page"]
        x = s["qkv"].float().view(T, Hq + 2 * H, D)
        angle = s["position"].double()[:, None] * s["freq"]
        cos, sin = ((f(angle) * s["scale"]).float()[:, None] for f in (torch.cos, torch.sin))
        qk = torch.cat([_rotate(x[:, :Hq + H, :rot], cos, sin, c["layout"]), x[:, :Hq + H, rot:]], 2)
        page, slot = s["table"][s["seq"], s["position"] // P].long(), s["position"] % P
        s["k"][page, slot] = qk[:, Hq:].bfloat16()
        s["v"][page, slot] = x[:, Hq + H:].bfloat16()
        return [qk[:, :Hq].bfloat16(), s["k"], s["v"]]
    if c["op"] == "attend":
        T, Hq, H, D, P = s["rows"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(T, Hq, dtype=torch.float32, device="cuda")
        for g in s["groups"]:  # the sequences with as many new tokens, padded to the longest
            n, L, S = g["new"], g["keys"], len(g["seqs"])
            pages = s["table"][g["seqs"], :-(-L // P)].clamp(min=0).long()
            k, v = (s[x][pages].reshape(S, -1, H, D)[:, :L].float().transpose(1, 2) for x in "kv")  # [sequence, head, key, element]
            q = s["q"][g["rows"]].float().view(S, n, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(S, H, -1, D)
            z = (q @ k.transpose(2, 3)).view(S, H, Hq // H, n, L) * D ** -0.5
            key = torch.arange(L, device="cuda")
            hidden = (key >= s["lengths"][g["seqs"]][:, None])[:, None]
            if c["causal"]:
                back = (s["lengths"][g["seqs"]] - n)[:, None, None] + torch.arange(n, device="cuda")[:, None] - key
                hidden = (back < 0) | (back >= c["window"]) if c["window"] else back < 0
            z.masked_fill_(hidden[:, None, None], -math.inf)
            m = z.amax(4, keepdim=True)
            z = torch.exp(z - m)
            total = z.sum(4, keepdim=True)
            o = (z.view(S, H, -1, L) @ v).view(S, H, Hq // H, n, D) / total
            out[g["rows"]] = o.permute(0, 3, 1, 2, 4).reshape(S * n, Hq, D).bfloat16()
            lse[g["rows"]] = (m + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(S * n, Hq)
        return [out, lse]
    R, V = c["rows"], c["vocab"]
    x = s["logits"][:, :V].float()
    place = torch.arange(c["history"], device="cuda")
    inside = place < s["lengths"][:, None]
    tokens = s["tokens"].long()
    seen = torch.zeros(R, V, device="cuda").scatter_add_(1, tokens, inside.float())
    count = torch.zeros(R, V, device="cuda").scatter_add_(1, tokens, (inside & (place >= s["prompts"][:, None])).float())
    rep = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias"] is not None:
        x = x.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if s["allowed"] is not None:
        bits = (s["allowed"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        allowed = bits.view(bits.shape[0], -1)[:, :V] != 0
        row = s["mask_rows"].long()
        x = torch.where(allowed[row.clamp(min=0)] | (row < 0)[:, None], x, -math.inf)
    return x.to(_DT[c["dtype"]])


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The case's outputs from the definitions, in 64 bits."""
    c, s = case, _inputs(case, seed)
    f = torch.float64
    if c["op"] == "append":
        Hq, H, D, rot, P = c["q_heads"], c["kv_heads"], c["dim"], c["rot"], c["page"]
        freq, scale = _frequencies(c)
        x = s["qkv"].to(f).unflatten(1, (Hq + 2 * H, D))
        half = rot // 2
        first = torch.arange(half, device="cuda") * (1 if c["layout"] == "half" else 2)
        second = first + (half if c["layout"] == "half" else 1)
        turn = torch.polar(torch.full_like(s["position"], scale, dtype=f)[:, None].expand(-1, half), torch.outer(s["position"].to(f), freq))
        z = torch.complex(x[:, :Hq + H, first], x[:, :Hq + H, second]) * turn[:, None]
        x[:, :Hq + H, first], x[:, :Hq + H, second] = z.real, z.imag
        k, v = s["k"].to(f), s["v"].to(f)
        flat = (s["table"][s["seq"], torch.div(s["position"], P, rounding_mode="floor")] * P + s["position"] % P).long()
        k, v = (t.contiguous().flatten(0, 1).index_copy(0, flat, u).view(t.shape) for t, u in ((k, x[:, Hq:Hq + H]), (v, x[:, Hq + H:])))
        return [x[:, :Hq], k, v]
    if c["op"] == "attend":
        Hq, H, D = c["q_heads"], c["kv_heads"], c["dim"]
        out, lse = torch.zeros(s["rows"], Hq, D, dtype=f, device="cuda"), torch.zeros(s["rows"], Hq, dtype=f, device="cuda")
        first = s["starts"].tolist()
        for i, (n, past) in enumerate(zip(s["new"], s["past"])):
            where = torch.arange(n + past, device="cuda")
            page, slot = s["table"][i].long()[where // c["page"]], where % c["page"]
            for b in range(0, n, 1024):  # blocks of rows
                rows = torch.arange(b, min(n, b + 1024), device="cuda")
                far = (past + rows)[:, None] - where
                seen = torch.ones_like(far, dtype=torch.bool) if not c["causal"] else (far >= 0) & (far < (c["window"] or n + past))
                keys = seen.any(0).nonzero()[:, 0]  # only what some row of the block sees
                lo, hi = int(keys[0]), int(keys[-1]) + 1
                for h in range(H):
                    k, v = s["k"][page[lo:hi], slot[lo:hi], h].to(f), s["v"][page[lo:hi], slot[lo:hi], h].to(f)
                    for j in range(h * (Hq // H), (h + 1) * (Hq // H)):
                        score = torch.einsum("rd,kd->rk", s["q"][first[i] + rows, j].to(f), k) / math.sqrt(D)
                        score = score.masked_fill(~seen[:, lo:hi], -math.inf)
                        l = torch.logsumexp(score, 1)
                        lse[first[i] + rows, j] = l
                        out[first[i] + rows, j] = torch.einsum("rk,kd->rd", torch.exp(score - l[:, None]), v)
        return [out, lse]
    R, V = c["rows"], c["vocab"]
    x = s["logits"][:, :V].to(f).contiguous()
    lengths, prompts = s["lengths"].tolist(), s["prompts"].tolist()
    for r in range(R):
        every = torch.unique(s["tokens"][r, :lengths[r]].long())
        z, rep = x[r, every], s["repetition"][r].to(f)
        x[r, every] = torch.maximum(z, z.new_zeros(())) / rep + torch.minimum(z, z.new_zeros(())) * rep
        made, count = torch.unique(s["tokens"][r, prompts[r]:lengths[r]].long(), return_counts=True)
        x[r, made] -= s["frequency"][r].to(f) * count + s["presence"][r].to(f)
    if s["bias"] is not None:
        x.scatter_add_(1, s["bias_ids"].long(), s["bias"].to(f))
    if s["allowed"] is not None:
        v = torch.arange(V, device="cuda")
        for r, m in enumerate(s["mask_rows"].tolist()):
            if m >= 0:
                x[r, ((s["allowed"][m].long()[v // 32] >> (v % 32)) & 1) == 0] = -math.inf
    return x
