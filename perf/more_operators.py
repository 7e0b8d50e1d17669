"""The attention half of a transformer block as a server runs it, operator by operator: rotary
positions, appending keys and values to a paged cache, attention of new tokens over that cache,
and the dense products on both sides of it with bias, activation and residual.

A case names one operator, its sizes and its types. prepare() draws what a program has in hand
(projected rows, a paged cache with its page tables, weights); run() computes the operator in its
plain form, or with the package's kernels where `own` is true. Both take the same inputs.

A batch holds `seqs` sequences. Sequence b has some new tokens, whose rows stand one sequence
after the other, and some tokens in the cache before them. Its keys lie on pages of `page` tokens,
anywhere in the cache, in the order that its row of the page table gives.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
      "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "none": 0}


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # one token's queries and keys are rotated: only latency counts
        dict(name="rope_token", op="rope", T=1, heads=40, D=128, dim=128, layout="half",
             type="bf16", scaling="none", longest=32768),
        # a long prompt's queries and keys, inside the rows that the QKV product wrote; half of
        # each head turns, neighbours in pairs, frequencies scaled for a longer context
        dict(name="rope_prompt", op="rope", T=16384, heads=40, D=128, dim=64,
             layout="interleaved", type="bf16", scaling="yarn", longest=131072),
        # four sequences decode: queries are rotated and one token each goes to the cache
        dict(name="append_decode", op="append", seqs=4, new=1, past=6000, page=16, Hq=64, Hkv=8,
             D=64, dim=64, layout="half", scaling="yarn", type="bf16", cache="bf16"),
        # a chunk of a long prompt goes to an 8-bit cache, from the middle of a page on
        dict(name="append_chunk", op="append", seqs=1, new=8192, past=20011, page=64, Hq=32,
             Hkv=4, D=128, dim=128, layout="half", scaling="none", type="bf16", cache="e4m3"),
        # one token decodes in a layer with a short window and a learned sink
        dict(name="attend_token", op="attend", seqs=1, new=1, past=999, page=16, Hq=64, Hkv=8,
             D=64, type="bf16", cache="bf16", window=128, keep=0, sinks=True),
        # a server's batch decodes at uneven lengths
        dict(name="attend_batch", op="attend", seqs=64, new=1, past=16384, page=16, Hq=32, Hkv=8,
             D=128, type="bf16", cache="bf16", window=0, keep=0, sinks=False),
        # one sequence decodes far into a long context, on an 8-bit cache
        dict(name="attend_long", op="attend", seqs=1, new=1, past=131071, page=64, Hq=32, Hkv=4,
             D=128, type="bf16", cache="e4m3", window=0, keep=0, sinks=False),
        # chunks of prompts of uneven lengths beside sequences that decode, in one batch
        dict(name="attend_mixed", op="attend", seqs=16, new=512, past=8192, page=32, Hq=32, Hkv=4,
             D=128, type="bf16", cache="bf16", window=0, keep=0, sinks=False),
        # the second half of a long prompt
        dict(name="attend_prompt", op="attend", seqs=1, new=8192, past=8192, page=64, Hq=32,
             Hkv=8, D=128, type="bf16", cache="bf16", window=0, keep=0, sinks=False),
        # four sequences decode: the QKV product's weights are read once
        dict(name="linear_decode", op="linear", M=4, N=5120, K=2880, type="bf16", bias="bf16",
             act="none", resid="none", out="bf16"),
        # a ragged batch of tokens: the output product adds to the residual stream
        dict(name="linear_ragged", op="linear", M=333, N=2880, K=4096, type="bf16", bias="bf16",
             act="none", resid="fp32", out="fp32"),
        # a long prompt's product with an activation behind it
        dict(name="linear_prompt", op="linear", M=16384, N=5120, K=2880, type="bf16", bias="fp32",
             act="silu", resid="none", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "attend", "linear", "linear"))
    D = rng.choice((64, 64, 80, 96, 128, 128, 128, 256))
    kind = dict(layout=rng.choice(("half", "interleaved")),
                scaling=rng.choice(("none", "linear", "yarn")))
    if op == "rope":
        heads = rng.randint(1, 80)
        return dict(op=op, T=_log_int(rng, 1, 160_000_000 // 2 // (heads * D)), heads=heads, D=D,
                    dim=rng.choice((D, D, D // 2)), type=rng.choice(("bf16", "fp16", "fp32")),
                    longest=_log_int(rng, 1000, 1_000_000), **kind)
    Hkv, G = rng.choice((1, 2, 4, 8, 8, 12)), rng.choice((1, 2, 3, 4, 7, 8, 8, 16))
    types = dict(type=rng.choice(("bf16", "bf16", "fp16")))
    types["cache"] = rng.choice((types["type"], types["type"], "e4m3"))
    page = rng.choice((16, 16, 32, 64, 128, 48, 1))
    if op == "append":
        seqs = _log_int(rng, 1, 256)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, 40_000_000 // (
            seqs * Hkv * (G + 2) * D)))
        return dict(op=op, seqs=seqs, new=new, past=_log_int(rng, 1, max(2, 400_000 // seqs)),
                    page=page, Hq=Hkv * G, Hkv=Hkv, D=D, dim=rng.choice((D, D, D // 2)), **kind,
                    **types)
    if op == "attend":
        shape = rng.choice(("token", "batch", "chunk", "prompt"))
        seqs = {"token": 1, "batch": _log_int(rng, 2, 128), "chunk": _log_int(rng, 2, 24),
                "prompt": 1}[shape]
        new = {"token": 1, "batch": 1, "chunk": _log_int(rng, 2, 700),
               "prompt": _log_int(rng, 100, 8192)}[shape]
        # the keys, and the products of a padded batch, of the largest listed cases
        scores = 500_000_000_000 // (seqs * Hkv * G * D)
        new = min(new, math.isqrt(scores))
        most = min(1_000_000_000 // (seqs * Hkv * D), scores // new)
        past = _log_int(rng, 1, max(2, min(200_000, most) - new))
        window = rng.choice((0, 0, 0, 128, 2048, 100))
        return dict(op=op, seqs=seqs, new=new, past=past, page=page, Hq=Hkv * G, Hkv=Hkv, D=D,
                    window=window, keep=rng.choice((0, 4)) if window else 0,
                    sinks=rng.random() < 0.3, **types)
    N, K = _log_int(rng, 64, 16384), 8 * _log_int(rng, 8, 1792)
    M = _log_int(rng, 1, min(16384, 240_000_000_000 // (N * K)))
    resid = rng.choice(("none", "none", "bf16", "fp32"))
    return dict(op=op, M=M, N=N, K=K, type=types["type"], bias=rng.choice(("none", "same", "fp32"))
                .replace("same", types["type"]), act=rng.choice(("none", "none", "relu", "gelu",
                                                                 "gelu_tanh", "silu")),
                resid=resid, out=resid if resid != "none" else rng.choice((types["type"], "fp32")))


# ------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _frequencies(c):
    """Radians a position of each pair, and the factor on the turned values."""
    n, base = c["dim"], 150000.0
    i = torch.arange(n // 2, dtype=torch.float64)
    f = base ** (-2 * i / n)
    if c["scaling"] == "linear":
        return (f / 4).to(DEV), 1.0
    if c["scaling"] == "yarn":   # pairs that turn less than once in 4096 positions are slowed
        def pair(turns):
            return n * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), n - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return (f / 32 * (1 - keep) + f * keep).to(DEV), 0.1 * math.log(32) + 1
    return f.to(DEV), 1.0


def _lengths(c):
    """New and cached tokens of each sequence, the same for every seed: the first one has most
    of both; in a batch of chunks every second one decodes a single token."""
    new, past = [], []
    for b in range(c["seqs"]):
        u, v = (b * 0.6180339887) % 1, (b * 0.7548776662) % 1
        new.append(1 if b % 2 else max(1, round(c["new"] * (1 - 0.8 * u))))
        past.append(round(c["past"] * (1 - 0.75 * v)))
    return new, past


def _batch(g, c):
    """Page table and lengths of a batch; the pages that it needs, in random order."""
    new, past = _lengths(c)
    total = [n + p for n, p in zip(new, past)]
    pages = [-(-t // c["page"]) for t in total]
    order = torch.randperm(sum(pages), generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["seqs"], max(pages)), -1, dtype=torch.int32, device=DEV)
    start = [0]
    for b, n in enumerate(pages):
        table[b, :n] = order[sum(pages[:b]):sum(pages[:b]) + n]
        start.append(start[-1] + new[b])
    return dict(new=new, total=total, table=table, n_pages=sum(pages),
                q_start=torch.tensor(start, dtype=torch.int32, device=DEV),
                seq_len=torch.tensor(total, dtype=torch.int32, device=DEV),
                # sequence and position of every row, and its place among a padded batch's
                row_seq=torch.repeat_interleave(torch.arange(c["seqs"], device=DEV),
                                                torch.tensor(new, device=DEV)),
                row_at=torch.cat([torch.arange(n) for n in new]).to(DEV))


def _cache(g, c, n_pages, scale=None):
    """Pages of keys or values: unit normal values, divided by a head's scale if there is one."""
    rows = _randn(g, n_pages, c["page"], c["Hkv"], c["D"])
    if scale is not None:
        rows /= scale[:, None]
    return rows.to(DT[c["cache"]])


def _inputs(c, seed):
    g = _gen(seed)
    op = c["op"]
    if op == "rope":
        freq, scale = _frequencies(c)
        row = _randn(g, c["T"], c["heads"] + 8, c["D"], dtype=DT[c["type"]])   # values behind
        first = torch.randint(0, max(1, c["longest"] - c["T"]), (), generator=g, device=DEV)
        return dict(x=row[:, :c["heads"]], freq=freq, scale=scale,
                    positions=(first + torch.arange(c["T"], device=DEV)).to(torch.int32))
    if op in ("append", "attend"):
        d = _batch(g, c)
        T, Hq, Hkv, D, ty = sum(d["new"]), c["Hq"], c["Hkv"], c["D"], DT[c["type"]]
        d["k_scale"] = d["v_scale"] = None
        if c["cache"] == "e4m3" and op == "attend":
            d["k_scale"] = 0.02 + 0.03 * torch.rand(Hkv, generator=g, device=DEV)
            d["v_scale"] = 0.02 + 0.03 * torch.rand(Hkv, generator=g, device=DEV)
        d["k_cache"] = _cache(g, c, d["n_pages"], d["k_scale"])
        d["v_cache"] = _cache(g, c, d["n_pages"], d["v_scale"])
        if op == "append":
            row = _randn(g, T, Hq + 2 * Hkv, D, dtype=ty)      # what the QKV product wrote
            d["q"], d["k"], d["v"] = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
            d["freq"], d["scale"] = _frequencies(c)
            return d
        d["q"] = _randn(g, T, Hq, D, dtype=ty)
        d["sinks"] = _randn(g, Hq) if c["sinks"] else None
        d["scale"] = 1 / math.sqrt(D)
        return d
    ty = DT[c["type"]]
    return dict(x=_randn(g, c["M"], c["K"], dtype=ty),
                w=(_randn(g, c["N"], c["K"]) / math.sqrt(c["K"])).to(ty),
                bias=None if c["bias"] == "none" else _randn(g, c["N"], dtype=DT[c["bias"]]),
                resid=None if c["resid"] == "none" else 3 * _randn(g, c["M"], c["N"]).to(
                    DT[c["resid"]]))


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = case
    if own:   # what a program keeps: the frequencies' plan, the cache, a step's batch
        import quantized_routed_expert_gemv_amd as moe
        if "freq" in d:
            d["plan"] = moe.Rope(d["freq"], case["layout"], d["scale"])
        if "table" in d:
            d["kv"] = moe.KvCache(d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"])
            d["batch"] = moe.KvBatch(d["q_start"], d["seq_len"], d["table"], max(d["new"]),
                                     max(d["total"]))
    return d


# --------------------------------------------------------------------------------- run


def run(d):
    return (_own if own else _plain)(d, d["case"])


def _own(d, c):
    import quantized_routed_expert_gemv_amd as moe
    if c["op"] == "rope":
        return moe.rope(d["x"], d["positions"], d["plan"])
    if c["op"] == "append":
        q = moe.kv_append(d["kv"], d["batch"], d["k"], d["v"], rope=d["plan"], q=d["q"])
        return dict(q=q, k=d["k_cache"], v=d["v_cache"])
    if c["op"] == "attend":
        return moe.attend(d["q"], d["kv"], d["batch"], scale=d["scale"], window=c["window"],
                          keep_first=c["keep"], sinks=d["sinks"])
    return moe.linear(d["x"], d["w"], bias=d["bias"], act=c["act"], resid=d["resid"],
                      out_dtype=DT[c["out"]])


def _turned(x, positions, freq, scale, layout):
    """Rows [T, heads, D] with the first 2 * len(freq) values of each head turned, in fp32."""
    x = x.float()
    a = positions.double()[:, None, None] * freq        # far positions: angles in 64 bits
    c, s = (scale * torch.cos(a)).float(), (scale * torch.sin(a)).float()
    n = freq.numel()
    if layout == "half":
        u, v = x[..., :n], x[..., n:2 * n]
        turned = torch.cat((u * c - v * s, u * s + v * c), -1)
    else:
        u, v = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack((u * c - v * s, u * s + v * c), -1).flatten(-2)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _stored(x, dtype):
    return x.clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _plain(d, c):
    if c["op"] == "rope":
        return _turned(d["x"], d["positions"], d["freq"], d["scale"], c["layout"]).to(d["x"].dtype)
    if c["op"] == "linear":
        v = d["x"].float() @ d["w"].float().T
        if d["bias"] is not None:
            v = v + d["bias"].float()
        if c["act"] == "relu":
            v = torch.clamp(v, min=0)
        elif c["act"] == "gelu":
            v = 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
        elif c["act"] == "gelu_tanh":
            v = 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
        elif c["act"] == "silu":
            v = v / (1 + torch.exp(-v))
        if d["resid"] is not None:
            v = d["resid"].float() + v
        return v.to(DT[c["out"]])
    # sequence, position and page slot of every row
    seq, at, new = d["row_seq"], d["row_at"], d["q_start"].diff()
    pos = (d["seq_len"] - new)[seq] + at
    if c["op"] == "append":
        page = d["table"][seq, pos // c["page"]].long()
        turn = (d["freq"], d["scale"], c["layout"])
        d["k_cache"][page, pos % c["page"]] = _stored(_turned(d["k"], pos, *turn), d["k_cache"].dtype)
        d["v_cache"][page, pos % c["page"]] = _stored(d["v"].float(), d["v_cache"].dtype)
        return dict(q=_turned(d["q"], pos, *turn).to(d["q"].dtype), k=d["k_cache"], v=d["v_cache"])
    # attention of a padded batch: rows [sequence, KV head, new token * query head of it, D]
    B, Hkv, G, D = c["seqs"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    table = d["table"].long().clamp(min=0)
    k = d["k_cache"][table].flatten(1, 2).float()
    v = d["v_cache"][table].flatten(1, 2).float()
    if d["k_scale"] is not None:
        k, v = k * d["k_scale"][:, None], v * d["v_scale"][:, None]
    most = max(d["new"])
    q = torch.zeros(B, most, c["Hq"], D, device=DEV)
    q[seq, at] = d["q"].float()
    q = q.view(B, most, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, most * G, D)
    s = d["scale"] * (q @ k.permute(0, 2, 3, 1).contiguous())
    s = s.view(B, Hkv, most, G, -1)
    row = (d["seq_len"] - new)[:, None] + torch.arange(most, device=DEV)
    key = torch.arange(k.shape[1], device=DEV)
    seen = key <= row[..., None]                        # [sequence, new token, key]
    if c["window"]:
        seen &= (key > row[..., None] - c["window"]) | (key < c["keep"])
    s.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    if d["sinks"] is not None:
        sink = d["sinks"].view(Hkv, 1, G, 1)
        top = torch.maximum(top, sink)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    if d["sinks"] is not None:
        total = total + torch.exp(sink - top)
    inside = key < d["seq_len"][:, None]                # behind a sequence's end a page holds anything
    v = v.masked_fill(~inside[..., None, None], 0).permute(0, 2, 1, 3).contiguous()
    out = (s.view(B, Hkv, most * G, -1) @ v).view(B, Hkv, most, G, D) / total
    out = out.permute(0, 2, 1, 3, 4).reshape(B, most, c["Hq"], D)
    return out[seq, at].to(d["q"].dtype)


# -------------------------------------------------------------------------------- exact


def _rotation(x, positions, freq, scale, layout):
    """Each pair as a complex number times scale * e^(i angle), in 64 bits."""
    x, n = x.double(), freq.numel()
    z = torch.polar(torch.full_like(freq, scale).expand(len(positions), -1),
                    torch.outer(positions.double(), freq))[:, None]
    out = x.clone()
    re, im = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2),
                                                                     slice(1, 2 * n, 2))
    w = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * z
    out[..., re], out[..., im] = w.real, w.imag
    return out


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    if c["op"] == "rope":
        return _rotation(d["x"], d["positions"], d["freq"], d["scale"], c["layout"])
    if c["op"] == "linear":
        out = []
        w = d["w"].double().t().contiguous()
        for i in range(0, c["M"], 4096):
            v = torch.matmul(d["x"][i:i + 4096].double(), w)
            if d["bias"] is not None:
                v += d["bias"].double()
            v = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
                 "gelu": lambda v: v * torch.special.ndtr(v),
                 "gelu_tanh": lambda v: v * torch.sigmoid(
                     2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}[c["act"]](v)
            out.append(v if d["resid"] is None else v + d["resid"][i:i + 4096].double())
        return torch.cat(out)
    ends = d["q_start"].tolist()
    if c["op"] == "append":
        q = torch.empty(d["q"].shape, dtype=torch.float64, device=DEV)
        k, v = d["k_cache"].double(), d["v_cache"].double()
        top = 448.0 if c["cache"] == "e4m3" else math.inf
        for b, n in enumerate(d["new"]):
            rows = slice(ends[b], ends[b + 1])
            pos = torch.arange(d["total"][b] - n, d["total"][b], device=DEV)
            page = d["table"][b].long()[torch.div(pos, c["page"], rounding_mode="floor")]
            args = (pos, d["freq"], d["scale"], c["layout"])
            q[rows] = _rotation(d["q"][rows], *args)
            k[page, pos % c["page"]] = _rotation(d["k"][rows], *args).clamp(-top, top)
            v[page, pos % c["page"]] = d["v"][rows].double().clamp(-top, top)
        return dict(q=q, k=k, v=v)
    G = c["Hq"] // c["Hkv"]
    out = torch.empty(d["q"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(d["new"]):
        L = d["total"][b]
        pages = d["table"][b, :-(-L // c["page"])].long()
        pos = torch.arange(L - n, L, device=DEV)[:, None]
        key = torch.arange(L, device=DEV)
        hidden = key > pos
        if c["window"]:
            hidden |= (pos - key >= c["window"]) & (key >= c["keep"])
        for h in range(c["Hkv"]):
            k = d["k_cache"][pages, :, h].flatten(0, 1)[:L].double()
            v = d["v_cache"][pages, :, h].flatten(0, 1)[:L].double()
            if d["k_scale"] is not None:
                k, v = k * d["k_scale"][h].double(), v * d["v_scale"][h].double()
            kt = k.t().contiguous()
            for j in range(h * G, (h + 1) * G):
                s = torch.matmul(d["q"][ends[b]:ends[b + 1], j].double(), kt) * d["scale"]
                s = s.masked_fill(hidden, -math.inf)
                if d["sinks"] is not None:     # one more key, whose value is zero
                    s = torch.cat((s, d["sinks"][j].double().expand(n, 1)), 1)
                out[ends[b]:ends[b + 1], j] = torch.matmul(torch.softmax(s, 1)[:, :L], v)
    return out


# --------------------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * c["heads"]
        return dict(bytes=2 * n * c["D"] * SIZE[c["type"]] + 4 * c["T"] + 4 * c["dim"],
                    flops=n * c["dim"] * 3)
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return dict(bytes=(M * K + N * K) * SIZE[c["type"]] + N * SIZE[c["bias"]] +
                    M * N * (SIZE[c["resid"]] + SIZE[c["out"]]), flops=2 * M * N * K)
    new, past = _lengths(c)
    T, D, ty, kv = sum(new), c["D"], SIZE[c["type"]], SIZE[c["cache"]]
    if c["op"] == "append":
        return dict(bytes=T * D * (2 * c["Hq"] * ty + 2 * c["Hkv"] * (ty + kv)) + 4 * c["dim"],
                    flops=T * (c["Hq"] + c["Hkv"]) * c["dim"] * 3)
    pairs = keys = 0
    for n, p in zip(new, past):
        w = c["window"] or n + p
        # keys that each new token sees, and that any of them sees
        seen = [min(i + 1, w + min(c["keep"], max(0, i + 1 - w))) for i in range(p, p + n)]
        first = max(0, p + 1 - w)
        pairs += sum(seen)
        keys += n + p - first + min(c["keep"], first)
    return dict(bytes=2 * T * c["Hq"] * D * ty + 2 * keys * c["Hkv"] * D * kv,
                flops=4 * pairs * c["Hq"] * D)
