"""The FFN half of a transformer block in microscaled precision, operator by operator: the
norm before the block, quantisation to microscaled formats, the experts' products on
microscaled activations, and the combine with the norm, gate and scale after the block.

A case names one operator, its sizes and its types. prepare() draws what a program has in
hand (the residual stream, an expert pool, routed and bucketed tokens); run() computes the
operator in its plain form, or with the package's kernels where `own` is true. Both take the
same inputs: the plain forms read the canonical planes of the weights, the kernels the pool.

Microscaled formats: blocks of 32 values along a row share one scale byte s, meaning
2^(s - 127); MXFP4 holds E2M1 codes (4 bits), MXFP6 E2M3 codes (6 bits).
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# finest step, largest value and bits of a code; both formats have 2 as their largest exponent
MX = {"mxfp4": (0.5, 6.0, 4), "mxfp6": (0.125, 7.5, 6)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # one token leaves attention: the block's entry, where only latency counts
        dict(name="norm_decode", op="add_norm", T=1, H=2880, resid="bf16", delta="bf16",
             weight="bf16", scale=1.0),
        # a long prompt's tokens at the block's entry
        dict(name="norm_prefill", op="add_norm", T=16384, H=2880, resid="bf16", delta="bf16",
             weight="bf16", scale=1.0),
        # four sequences decode: the block's exit feeds the next layer's norm
        dict(name="exit_decode", op="combine_norm", T=4, H=2880, k=4, resid="bf16",
             weight="bf16", post=False, gate="none", next=True, scale=1.0),
        # a prompt at the exit of a block with norms on both sides, a gate and a scale
        dict(name="exit_prefill", op="combine_norm", T=8192, H=2048, k=8, resid="fp32",
             weight="fp32", post=True, gate="channel", next=True, scale=0.22),
        # a ragged batch of tokens becomes the products' operand
        dict(name="quantise_tokens", op="quantise", rows=1000, K=2880, src="bf16", fmt="mxfp6"),
        # a loader quantises 32 experts' matrices before they are packed into a pool
        dict(name="quantise_weights", op="quantise", rows=92160, K=2880, src="bf16",
             fmt="mxfp4"),
        # one token decodes: four experts' gate and up matrices are read once
        dict(name="gate_up_decode", op="gate_up", T=1, H=2880, I=2880, E=32, k=4, skew=0.0,
             fmt="mxfp6", missing=0),
        # sixteen sequences decode on fine-grained experts
        dict(name="gate_up_batch", op="gate_up", T=16, H=2048, I=768, E=128, k=8, skew=1.2,
             fmt="mxfp4", missing=0),
        # a long prompt with a skewed load
        dict(name="gate_up_prefill", op="gate_up", T=16384, H=2880, I=2880, E=32, k=4,
             skew=1.1, fmt="mxfp4", missing=0),
        # four sequences decode on a few wide experts
        dict(name="down_decode", op="down", T=4, H=4096, I=14336, E=8, k=2, skew=0.0,
             fmt="mxfp6", missing=0),
        # a short prompt over many experts, some of them not in the pool: small, odd groups
        dict(name="down_ragged", op="down", T=333, H=2048, I=768, E=128, k=8, skew=1.2,
             fmt="mxfp4", missing=16),
        # a long prompt's second product
        dict(name="down_prefill", op="down", T=16384, H=2880, I=2880, E=32, k=4, skew=1.1,
             fmt="mxfp6", missing=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("add_norm", "combine_norm", "quantise", "gate_up", "down"))
    if op in ("add_norm", "combine_norm"):
        H, k = 32 * _log_int(rng, 4, 400), rng.randint(1, 8)
        c = dict(op=op, T=_log_int(rng, 1, min(16384, (47_000_000 if op == "add_norm" else
                                                       134_000_000 // k) // H)), H=H,
                 resid=rng.choice(("bf16", "fp32")), weight=rng.choice(("bf16", "fp32")),
                 scale=rng.choice((1.0, 0.5, 0.22)))
        if op == "add_norm":
            c.update(delta=rng.choice(("none", "bf16", "fp32")))
        else:
            c.update(k=k, post=rng.random() < 0.5, next=rng.random() < 0.7,
                     gate=rng.choice(("none", "channel", "token")))
        return c
    if op == "quantise":
        K = 32 * _log_int(rng, 1, 448)
        return dict(op=op, rows=_log_int(rng, 1, 200_000_000 // K), K=K,
                    src=rng.choice(("bf16", "fp16", "fp32")), fmt=rng.choice(("mxfp4", "mxfp6")))
    E = rng.choice((4, 8, 17, 32, 64, 128))
    k = rng.randint(1, min(8, E))
    H, I = 32 * _log_int(rng, 4, 128), 32 * _log_int(rng, 4, 128)
    while E * H * I > 2.6e8:                     # the pool of the largest listed case
        H, I = max(128, H // 2 // 32 * 32), max(128, I // 2 // 32 * 32)
    T = _log_int(rng, 1, min(16384, 540_000_000_000 // (k * H * I)))   # and its products
    return dict(op=op, T=T, H=H, I=I, E=E, k=k,
                skew=rng.choice((0.0, 1.1)), fmt=rng.choice(("mxfp4", "mxfp6")),
                missing=rng.choice((0, 0, E // 8)))


# ------------------------------------------------- microscaled formats, in plain operations


def _steps(x, fmt):
    """Rows [..., K] -> (values over the scale, in whole finest steps; scale bytes)."""
    fine, top, _ = MX[fmt]
    v = x.float().reshape(*x.shape[:-1], -1, 32)
    # the largest magnitude's exponent, from the bits: exact for subnormal values too
    big = v.abs().amax(-1)
    s = ((big.view(torch.int32) >> 23) - 2).clamp(min=1)
    v = v.double() * torch.exp2((127 - s).double())[..., None]   # exact; fp32 could overflow
    step = fine * torch.where(v.abs() >= 4, 4.0, torch.where(v.abs() >= 2, 2.0, 1.0))
    v = (torch.round(v / step) * step).clamp(-top, top)   # round() takes halves to even
    s = torch.where(torch.isfinite(big), s, 255).to(torch.uint8)
    return torch.where(s[..., None] == 255, 0.0, v / fine).to(torch.int32), s


def _codes(x, fmt):
    """Rows [..., K] -> (packed codes [..., K bits / 8] uint8, scale bytes [..., K/32])."""
    n, s = _steps(x, fmt)
    a = n.abs()
    # whole steps to codes: every value below 4 (8) steps is its own code; then steps of 2, 4
    lo = 4 if fmt == "mxfp4" else 16
    a = torch.where(a < lo, a, torch.where(a < 2 * lo, lo // 2 + a // 2, lo + a // 4))
    bits = MX[fmt][2]
    c = (a + (n < 0) * (1 << (bits - 1))).reshape(*x.shape[:-1], x.shape[-1])
    if bits == 4:
        q = c[..., 0::2] | c[..., 1::2] << 4
    else:   # four codes fill three bytes, the first in the lowest bits
        w = c[..., 0::4] | c[..., 1::4] << 6 | c[..., 2::4] << 12 | c[..., 3::4] << 18
        q = torch.stack((w & 255, w >> 8 & 255, w >> 16), -1).reshape(*w.shape[:-1], -1)
    return q.to(torch.uint8), s


def _unpacked(q, fmt):
    """Packed codes -> one code a value, int32."""
    q = q.to(torch.int32)
    if fmt == "mxfp4":
        return torch.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1)
    w = q[..., 0::3] | q[..., 1::3] << 8 | q[..., 2::3] << 16
    return torch.stack((w & 63, w >> 6 & 63, w >> 12 & 63, w >> 18), -1).reshape(*w.shape[:-1], -1)


def _table(fmt, dtype):
    t = E2M1 if fmt == "mxfp4" else [m / 8 for m in range(16)] + [m / 4 for m in range(8, 16)] + \
        [m / 2 for m in range(8, 16)]
    return torch.tensor([*t, *(-v for v in t)], dtype=dtype, device=DEV)


def _values(q, s, fmt):
    """Codes and scales -> fp32 values [..., K]."""
    v = _table(fmt, torch.float32)[_unpacked(q, fmt)]
    scale = torch.exp2(s.float() - 127).masked_fill(s == 255, math.nan)
    return (v.view(*s.shape, 32) * scale[..., None]).view(v.shape)


# ------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _matrices(g, E, rows, K):
    """E weight matrices, normal with variance 1/K, as canonical MXFP4 planes."""
    q = torch.empty(E, rows, K // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(E, rows, K // 32, dtype=torch.uint8, device=DEV)
    for e in range(E):
        q[e], s[e] = _codes(_randn(g, rows, K) / math.sqrt(K), "mxfp4")
    return q, s


def _routing(g, c):
    """Routed and bucketed tokens: ids, offsets, perm, inv_perm and the groups' sizes."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = _randn(g, T, E)
    if c["skew"]:   # the r-th most wanted expert is offset by -log(r^skew)
        rank = torch.randperm(E, generator=g, device=DEV) + 1
        logits = logits - c["skew"] * torch.log(rank.float())
    ids = logits.topk(k, dim=1).indices.to(torch.int32)
    flat = ids.reshape(-1).long()
    perm = torch.argsort(flat, stable=True)
    sizes = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = sizes.cumsum(0)
    return offsets, perm.to(torch.int32), sizes.tolist()


def _inputs(c, seed):
    g = _gen(seed)
    op = c["op"]
    if op == "add_norm":
        T, H = c["T"], c["H"]
        return dict(
            resid=(3 * _randn(g, T, H)).to(DT[c["resid"]]),
            delta=None if c["delta"] == "none" else _randn(g, T, H, dtype=DT[c["delta"]]),
            weight=(1 + 0.2 * _randn(g, H)).to(DT[c["weight"]]))
    if op == "combine_norm":
        T, H, k, wt = c["T"], c["H"], c["k"], DT[c["weight"]]
        return dict(
            y=_randn(g, T * k, H),
            inv_perm=torch.randperm(T * k, generator=g, device=DEV).to(torch.int32),
            w=torch.softmax(_randn(g, T, k), 1),
            resid=(3 * _randn(g, T, H)).to(DT[c["resid"]]),
            post=(1 + 0.2 * _randn(g, H)).to(wt) if c["post"] else None,
            gate=None if c["gate"] == "none" else
            torch.sigmoid(_randn(g, *((T, H) if c["gate"] == "token" else (H,)))).to(wt),
            next=(1 + 0.2 * _randn(g, H)).to(wt) if c["next"] else None)
    if op == "quantise":
        x = _randn(g, c["rows"], c["K"])
        x *= torch.exp2(2 * _randn(g, c["rows"], 1))    # rows of different sizes
        return dict(x=x.to(DT[c["src"]]))
    # products: T tokens' activations (gate/up) or T*k pairs' hidden rows (down)
    up = op == "gate_up"
    rows, K = (c["T"], c["H"]) if up else (c["T"] * c["k"], c["I"])
    offsets, perm, sizes = _routing(g, c)
    slots = c["E"] - c["missing"]
    slot_map = torch.full((c["E"],), -1, dtype=torch.int32, device=DEV)
    resident = torch.randperm(c["E"], generator=g, device=DEV)[:slots]
    slot_map[resident] = torch.arange(slots, dtype=torch.int32, device=DEV)
    x = _randn(g, rows, K, dtype=torch.bfloat16)
    if not up:
        x = x * torch.nn.functional.silu(_randn(g, rows, K, dtype=torch.bfloat16))
    q, s = _codes(x, c["fmt"])
    d = dict(q=q, s=s, offsets=offsets, perm=perm, sizes=sizes, slot_map=slot_map,
             slots=slot_map.tolist())
    n, K = (c["I"], c["H"]) if up else (c["H"], c["I"])
    for name in ("gate", "up") if up else ("down",):
        d[name] = _matrices(g, slots, n, K)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = case
    if own and case["op"] in ("gate_up", "down"):
        import quantized_routed_expert_gemv_amd as moe
        H, I = case["H"], case["I"]
        pool = moe.Pool.empty("mxfp4", case["E"] - case["missing"], H, I)
        for name in ("gate", "up", "down"):
            if name in d:
                q, s = d.pop(name)
                moe.pool_pack("mxfp4", *q.shape[:2], 2 * q.shape[2], q, s,
                              pool.planes[name + "_q"], pool.planes[name + "_s"])
        d["pool"] = pool
    return d


# --------------------------------------------------------------------------------- run


def run(d):
    return (_own if own else _plain)(d, d["case"])


def _own(d, c):
    import quantized_routed_expert_gemv_amd as moe
    op = c["op"]
    if op == "add_norm":
        x, resid = moe.add_norm(d["resid"], d["weight"], delta=d["delta"], scale=c["scale"])
        return dict(x=x, resid=None if d["delta"] is None else resid)
    if op == "combine_norm":
        resid, x = moe.combine_norm(d["y"], d["inv_perm"], d["w"], d["resid"],
                                    post_weight=d["post"], gate=d["gate"], scale=c["scale"],
                                    next_weight=d["next"])
        return dict(resid=resid, x=x)
    if op == "quantise":
        q, s = moe.mx_quantize(d["x"], c["fmt"])
        return dict(s=s, values=moe.mx_dequantize(q, s, c["fmt"], d["x"].dtype))
    if op == "gate_up":
        return moe.mx_expert_gate_up(d["pool"], d["slot_map"], d["q"], d["s"], c["fmt"], c["k"],
                                     d["offsets"], d["perm"])
    return moe.mx_expert_down(d["pool"], d["slot_map"], c["T"], c["k"], d["offsets"], d["q"],
                              d["s"], c["fmt"])


EPS = 1e-6


def _norm(v, weight):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _plain(d, c):
    op = c["op"]
    if op == "add_norm":
        r = d["resid"].float()
        if d["delta"] is not None:
            r = r + c["scale"] * d["delta"].float()
        return dict(x=_norm(r, d["weight"]).bfloat16(),
                    resid=None if d["delta"] is None else r.to(d["resid"].dtype))
    if op == "combine_norm":
        rows = d["y"][d["inv_perm"].long()].view(c["T"], c["k"], c["H"])
        v = (d["w"][..., None] * rows).sum(1)
        if d["post"] is not None:
            v = _norm(v, d["post"])
        if d["gate"] is not None:
            v = v * d["gate"].float()
        r = d["resid"].float() + c["scale"] * v
        return dict(resid=r.to(d["resid"].dtype),
                    x=None if d["next"] is None else _norm(r, d["next"]).bfloat16())
    if op == "quantise":
        n, s = _steps(d["x"], c["fmt"])
        scale = torch.exp2(s.float() - 127).masked_fill(s == 255, math.nan)
        v = n * MX[c["fmt"]][0] * scale[..., None]
        return dict(s=s, values=v.reshape(d["x"].shape).to(d["x"].dtype))
    # Ragged groups: one matrix product an expert. Experts out of the pool leave zeros.
    x = _values(d["q"], d["s"], c["fmt"])
    n = c["I"] if op == "gate_up" else c["H"]
    out = torch.zeros(sum(d["sizes"]), n, device=DEV,
                      dtype=torch.bfloat16 if op == "gate_up" else torch.float32)
    at = 0
    for e, m in enumerate(d["sizes"]):
        slot = d["slots"][e]
        if m and slot >= 0:
            if op == "gate_up":
                rows = x[d["perm"][at:at + m].long() // c["k"]]
                g = rows @ _values(d["gate"][0][slot], d["gate"][1][slot], "mxfp4").T
                u = rows @ _values(d["up"][0][slot], d["up"][1][slot], "mxfp4").T
                out[at:at + m] = (g / (1 + torch.exp(-g)) * u).bfloat16()
            else:
                w = _values(d["down"][0][slot], d["down"][1][slot], "mxfp4")
                out[at:at + m] = x[at:at + m] @ w.T
        at += m
    return out


# -------------------------------------------------------------------------------- exact


def _wide(q, s, bits):
    """Packed codes and scales -> values in 64 bits, from the fields: sign, two exponent bits
    and the mantissa; exponent field 0 has no leading one."""
    q = q.long()
    parts = [q & 15, q >> 4] if bits == 4 else [
        q[..., 0::3] & 63, q[..., 0::3] >> 6 | (q[..., 1::3] & 15) << 2,
        q[..., 1::3] >> 4 | (q[..., 2::3] & 3) << 4, q[..., 2::3] >> 2]
    c = torch.stack(parts, -1).flatten(-2)
    m_bits = bits - 3
    field, m = c >> m_bits & 3, (c & ((1 << m_bits) - 1)).double() / (1 << m_bits)
    v = torch.where(field == 0, m, (1 + m) * torch.exp2(field.double() - 1))
    v = torch.where(c >> (bits - 1) == 1, -v, v)
    return v * torch.exp2(s.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    d, c, op = _inputs(case, seed), case, case["op"]
    rms = lambda v: torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS)  # noqa: E731
    if op == "add_norm":
        s = d["resid"].double()
        if d["delta"] is not None:
            s += c["scale"] * d["delta"].double()
        return dict(x=d["weight"].double() * s / rms(s), resid=None if d["delta"] is None else s)
    if op == "combine_norm":
        place = d["inv_perm"].long().view(c["T"], c["k"])
        v = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            v += d["w"][:, j, None].double() * d["y"][place[:, j]].double()
        if d["post"] is not None:
            v = v / rms(v) * d["post"].double()
        r = d["resid"].double() + c["scale"] * (v if d["gate"] is None else d["gate"].double() * v)
        return dict(resid=r, x=None if d["next"] is None else r / rms(r) * d["next"].double())
    if op == "quantise":
        # the nearest value of the format, by the borders halfway between neighbours; a value
        # on a border goes to the neighbour with the even code
        table = _table(c["fmt"], torch.float64)
        table = table[:len(table) // 2].contiguous()
        border = (table[1:] + table[:-1]) / 2
        out, scales = [], []
        for x in d["x"].split(max(1, (1 << 24) // c["K"])):
            v = x.double().view(len(x), -1, 32)
            big = v.abs().amax(-1)
            e = (torch.frexp(big).exponent - 1 - 2).clamp(min=-126)
            e = torch.where(big == 0, -126, e)
            u = v.abs() * torch.exp2(-e.double())[..., None]
            lo, hi = torch.searchsorted(border, u), torch.searchsorted(border, u, right=True)
            code = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
            w = torch.sign(v) * table[code] * torch.exp2(e.double())[..., None]
            out.append(w.view(x.shape).to(d["x"].dtype))   # exact: a code's bits fit the type
            scales.append((e + 127).to(torch.uint8))
        return dict(s=torch.cat(scales), values=torch.cat(out))
    x = _wide(d["q"], d["s"], MX[c["fmt"]][2])
    up = op == "gate_up"
    out = torch.zeros(c["T"] * c["k"], c["I"] if up else c["H"], dtype=torch.float64, device=DEV)
    ends = d["offsets"].tolist()
    for e in range(c["E"]):
        a, b, slot = ends[e], ends[e + 1], d["slots"][e]
        if a == b or slot < 0:
            continue
        m = {n: _wide(d[n][0][slot], d[n][1][slot], 4) for n in ("gate", "up", "down") if n in d}
        if up:
            t = x[torch.div(d["perm"][a:b].long(), c["k"], rounding_mode="floor")]
            gate = torch.matmul(t, m["gate"].t())
            out[a:b] = gate * torch.sigmoid(gate) * torch.matmul(t, m["up"].t())
        else:
            out[a:b] = torch.matmul(x[a:b], m["down"].t())
    return out


# --------------------------------------------------------------------------------- work


def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4, "none": 0}
    if op == "add_norm":
        n = c["T"] * c["H"]
        r, dl = size[c["resid"]], size[c["delta"]]
        return dict(bytes=n * (r + dl + (r if dl else 0) + 2) + c["H"] * size[c["weight"]],
                    flops=n * 6)
    if op == "combine_norm":
        n, w = c["T"] * c["H"], size[c["weight"]]
        gate = {"none": 0, "channel": c["H"] * w, "token": n * w}[c["gate"]]
        return dict(bytes=n * (4 * c["k"] + 2 * size[c["resid"]] + 2 * c["next"]) + gate +
                    c["T"] * c["k"] * 8 + c["H"] * w * (c["post"] + c["next"]),
                    flops=n * (2 * c["k"] + 10))
    if op == "quantise":
        # the values read, their codes and scales written; codes and scales read back, and
        # the values that they stand for written
        n = c["rows"] * c["K"]
        return dict(bytes=2 * (n * size[c["src"]] + n * MX[c["fmt"]][2] // 8 + n // 32),
                    flops=n * 6)
    up = op == "gate_up"
    E, k, T = c["E"], c["k"], c["T"]
    pairs = T * k * (E - c["missing"]) / E
    touched = (E - c["missing"]) * (1 - (1 - k / E) ** T)
    weights = touched * (2 if up else 1) * c["H"] * c["I"] * 17 / 32
    rows, K = (T, c["H"]) if up else (pairs, c["I"])
    outs = T * k * (2 * c["I"] if up else 4 * c["H"])
    return dict(bytes=weights + rows * K * (MX[c["fmt"]][2] / 8 + 1 / 32) + outs,
                flops=2 * pairs * c["H"] * c["I"] * (2 if up else 1))
