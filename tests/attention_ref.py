"""Plain 64-bit forms of the attention half of a block, on the CPU, and how far a kernel may be
from them. Written from the formulas; shares nothing with the kernels.

Half a step of a type is finfo.eps / 2 relative to the value (fp32 2^-24, fp16 2^-11, bf16 2^-8,
E4M3 2^-4), and half its smallest step below its normal range."""
import math

import torch

F32 = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(ref, dtype):
    """How far a value may move when it is rounded to dtype."""
    tiny = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25,
            E4M3: 2.0 ** -10}[dtype]
    return half_step(dtype) * ref.abs() + tiny


def rope(x, positions, freq, layout, scale, inverse=False):
    """-> (turned, tolerance before the last rounding), float64."""
    x = x.double().cpu()
    n = freq.numel()
    a = positions.double().cpu()[:, None, None] * freq.double().cpu()
    if inverse:
        a = -a
    c, s = scale * torch.cos(a), scale * torch.sin(a)
    out, tol = x.clone(), torch.zeros_like(x)
    re, im = ((slice(0, n), slice(n, 2 * n)) if layout == "half" else
              (slice(0, 2 * n, 2), slice(1, 2 * n, 2)))
    u, v = x[..., re], x[..., im]
    out[..., re], out[..., im] = u * c - v * s, u * s + v * c
    # cosine and sine: half turns are rounded to fp32 (2^-25 of a half turn: 1.6 half steps of
    # 1.0), the functions are within 2 half steps and the factor adds one: 5. The two products and
    # their sum add at most 2.
    # fp64 forms position * freq to 2^-53, and reduces it: 2^-51 of the angle in all
    t = (8 * F32 + 2.0 ** -51 * a.abs()) * abs(scale) * (u.abs() + v.abs())
    tol[..., re] = tol[..., im] = t
    return out, tol


def attend(q, keys, values, pos, scale, causal=True, window=0, keep=0, sinks=None, dtype=None,
           ok=None):
    """One sequence: q [n, Hq, D], keys and values [L, Hkv, D] (values that they stand for), pos [n],
    ok [L] False where a key has no page -> (out, tolerance), float64. dtype: the queries' type."""
    dtype = dtype or q.dtype
    q, keys, values = q.double().cpu(), keys.double().cpu(), values.double().cpu()
    n, Hq, D = q.shape
    L, Hkv = keys.shape[:2]
    G = Hq // Hkv
    j, p = torch.arange(L), pos.cpu()[:, None]
    seen = (j <= p) if causal else (j >= 0).expand(n, L)
    if window:
        seen = seen & ((j > p - window) | (j < keep))
    if ok is not None:
        seen = seen & ok.cpu()
    out, tol = torch.zeros(n, Hq, D, dtype=torch.float64), torch.zeros(n, Hq, D, dtype=torch.float64)
    h, top = half_step(dtype), 0.0
    for a in range(Hq):
        k, v = keys[:, a // G], values[:, a // G]
        for i in range(n):
            s = seen[i]
            if not s.any():
                continue
            ki, vi = k[s], v[s]
            sc = scale * (ki @ q[i, a])
            m = sc.max()
            if sinks is not None:
                m = torch.maximum(m, sinks[a].double().cpu())
            w = torch.exp(sc - m)
            tot = w.sum()
            if sinks is not None:
                tot = tot + torch.exp(sinks[a].double().cpu() - m)
            w = w / tot
            out[i, a] = w @ vi
            # a score: D exact products, D additions in fp32, times the scale; its weight: the
            # exponent's argument (below 2^6 for what counts) is rounded, exp2 adds an ulp or two
            ds = (D + 2) * F32 * abs(scale) * (ki.abs() @ q[i, a].abs()).max() + 2.0 ** -17
            # a weight is rounded to dtype; the sum of the weights has their errors once more, and
            # both sums those of len additions
            A = w @ vi.abs()
            t = (h + 2 * ds + 2 * (len(w) + 64) * F32) * A
            if dtype == torch.float16:   # weights below 2^-14 of the largest: half of 2^-24 each
                t = t + len(w) * 2.0 ** -25 * vi.abs().amax(0)
            tol[i, a] = t
    return out, tol + rounded(out, dtype)


def linear(x, w, bias, act, resid, out_dtype):
    """-> (out, tolerance), float64."""
    x, w = x.double().cpu(), w.double().cpu()
    K = x.shape[1]
    v = x @ w.T
    tol = (K + 2) * F32 * (x.abs() @ w.abs().T)    # K additions in fp32, whatever their order
    if bias is not None:
        v = v + bias.double().cpu()
        tol = tol + F32 * v.abs()
    if act != "none":
        z = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        f = {"relu": v.clamp(min=0), "silu": v * torch.sigmoid(v),
             "gelu": 0.5 * v * torch.special.erfc(-v / math.sqrt(2)),
             "gelu_tanh": v * torch.sigmoid(2 * z)}[act]
        # slopes are at most 1.13; the functions themselves are within 32 half steps of v (their
        # exponents' arguments, at most 90 where the result counts, are rounded)
        tol = 1.13 * tol + 64 * F32 * f.abs() + 2.0 ** -40
        v = f
    if resid is not None:
        v = resid.double().cpu() + v
        tol = tol + F32 * v.abs()
    return v, tol + rounded(v, out_dtype)


def near(got, ref, tol, what=""):
    got = got.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - ref).abs() / tol).nan_to_num(nan=9e9).max()):.3g} times "
                           f"the tolerance; first at {bad.nonzero()[0].tolist()}")
