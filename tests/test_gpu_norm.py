"""The norms at the block's two ends against the fp64 oracle, and the whole block in
microscaled precision.

Bounds count roundings of half a step. fp32: the sums of H squares run over at most H/256 + 16
dependent adds, and a handful of operations follow, so a value is within (H/256 + k + 24) 2^-24
of the exact one, relative to the magnitudes that were added; bf16 outputs add 2^-8.
"""
import numpy as np
import pytest

from oracle import mx

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def d(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, mag, fp32, half):
    """|got - want| <= fp32 roundings of the magnitudes `mag` + one rounding of the result."""
    tol = fp32 * 2.0 ** -24 * mag + half * (np.abs(want) + fp32 * 2.0 ** -24 * mag) + 2.0 ** -133
    bad = ~(np.abs(d(got) - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}"


# every register variant, its borders, and rows long enough to be recomputed
SIZES = [(1, 32), (3, 256), (2, 288), (5, 512), (4, 544), (300, 1024), (3, 1056), (1, 2048),
         (2, 2080), (17, 2880), (2, 4096), (1, 4128), (3, 6144), (2, 6176), (2, 8192), (2, 8224),
         (3, 20000)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("rt", [BF, F32])
@pytest.mark.parametrize("dt,wt", [(None, BF), (BF, F32), (F32, BF)])
def test_add_norm(T, H, rt, dt, wt):
    g = torch.Generator("cuda").manual_seed(H)
    r = (3 * torch.randn(T, H, generator=g, device="cuda")).to(rt)
    dl = None if dt is None else torch.randn(T, H, generator=g, device="cuda").to(dt)
    w = (1 + torch.randn(H, generator=g, device="cuda")).to(wt)
    keep = r.clone()
    x, out = qm.add_norm(r, w, 1e-5, delta=dl, scale=0.22)
    assert torch.equal(r, keep)
    want, s = mx.add_norm(d(r), d(w), float(np.float32(1e-5)), d(dl), float(np.float32(0.22)))
    mag = np.abs(d(r)) + (0 if dl is None else 0.22 * np.abs(d(dl)))
    scale = np.abs(d(w)) / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + 1e-5)
    close(x, want, mag * scale, H / 256 + 25, HALF[BF])
    if dl is None:
        assert out is r
    else:
        close(out, s, mag, 2, HALF[rt])
        # in place: the same bits
        x2, out2 = qm.add_norm(r, w, 1e-5, delta=dl, scale=0.22, resid_out=r)
        assert out2 is r and torch.equal(r, out) and torch.equal(x2, x)


@pytest.mark.parametrize("T,H,k", [(1, 32, 1), (2, 288, 3), (4, 2880, 4), (5, 1024, 8), (33, 2080, 2),
                                   (2, 4128, 5), (3, 8192, 6), (2, 8224, 7), (2, 20000, 4)])
@pytest.mark.parametrize("rt,wt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("post,gate,nxt", [(0, 0, 0), (0, 0, 1), (1, 1, 1), (1, 2, 1), (1, 0, 0),
                                           (0, 2, 1)])
def test_combine_norm(T, H, k, rt, wt, post, gate, nxt):
    g = torch.Generator("cuda").manual_seed(T * H + k)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    y, w, r = rand(T * k, H), torch.softmax(rand(T, k), 1), (3 * rand(T, H)).to(rt)
    inv = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    pw = (1 + rand(H)).to(wt) if post else None
    gt = None if not gate else rand(*((T, H) if gate == 2 else (H,))).to(wt)
    nw = (1 + rand(H)).to(wt) if nxt else None
    kw = dict(post_weight=pw, gate=gt, scale=0.5, next_weight=nw)
    out, x = qm.combine_norm(y, inv, w, r, 1e-6, **kw)
    eps = float(np.float32(1e-6))
    s, want = mx.combine_norm(d(y), inv.cpu().numpy(), d(w), d(r), eps, d(pw), d(gt), 0.5, d(nw))
    # magnitudes: |w| |y| sums through the post-norm's scale, the gate and the residual add
    mag = np.einsum("tk,tkh->th", d(w), np.abs(d(y))[inv.cpu().numpy().reshape(T, k)])
    if post:
        c = mx.combine_norm(d(y), inv.cpu().numpy(), d(w), 0 * d(r), eps)[0]
        mag = mag * np.abs(d(pw)) / np.sqrt(np.mean(c * c, axis=1, keepdims=True) + eps)
    mag = np.abs(d(r)) + 0.5 * mag * (1 if gt is None else np.abs(d(gt)))
    n = (H / 256 + k + 24) * (2 if post else 1)
    close(out, s, mag, n, HALF[rt])
    if nxt:
        scale = np.abs(d(nw)) / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
        # the mean's own error: at most the row's worst relative one
        row = np.sqrt(np.mean(mag * mag, axis=1, keepdims=True) / np.mean(s * s, axis=1, keepdims=True))
        close(x, want, mag * scale + np.abs(want) * row, 2 * n, HALF[BF])
    else:
        assert x is None
    out2, x2 = qm.combine_norm(y, inv, w, r, 1e-6, resid_out=r, **kw)
    assert out2 is r and torch.equal(r, out) and (x is None or torch.equal(x, x2))


def test_combine_norm_is_combine():
    """Without the extras and on a zero stream it gives moe_combine's bits."""
    T, H, k = 9, 736, 4
    y, w = torch.randn(T * k, H, device="cuda"), torch.rand(T, k, device="cuda")
    inv = torch.randperm(T * k, device="cuda").to(torch.int32)
    out, _ = qm.combine_norm(y, inv, w, torch.zeros(T, H, device="cuda"))
    assert torch.equal(out, qm.combine(y, inv, w))


def test_positions_outside_add_nothing():
    T, H, k = 3, 64, 2
    y, w = torch.randn(T * k, H, device="cuda"), torch.rand(T, k, device="cuda")
    r = torch.randn(T, H, device="cuda")
    inv = torch.tensor([0, -1, 6, 2, 0x7FFFFFFF, -2 ** 31], dtype=torch.int32, device="cuda")
    out, _ = qm.combine_norm(y, inv, w, r)
    want, _ = mx.combine_norm(d(y), inv.cpu().numpy(), d(w), d(r), 1e-6)
    close(out, want, np.abs(d(r)) + 2 * np.abs(d(y)).max(), 4, HALF[F32])
    y[0] = float("nan")        # a position that is not read does no harm
    out, _ = qm.combine_norm(y, torch.full_like(inv, -1), w, r)
    assert torch.equal(out, r)


@pytest.mark.parametrize("rt", [BF, F32])
def test_outputs_of_the_callers(rt):
    r, w = torch.randn(5, 96, device="cuda").to(rt), torch.ones(96, device="cuda")
    out, x = torch.empty_like(r), torch.empty(5, 96, dtype=BF, device="cuda")
    got = qm.add_norm(r, w, resid_out=out, x=x)      # without delta the stream is copied
    assert got[0] is x and got[1] is out and torch.equal(out, r)
    assert torch.equal(x, qm.add_norm(r, w)[0])
    assert torch.equal(qm.add_norm(r, w, delta=r, scale=0.0)[0], x)
    y, inv = torch.randn(5, 96, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda")
    one = torch.ones(5, 1, device="cuda")
    got = qm.combine_norm(y, inv, one, r, next_weight=w, resid_out=out, x=x)
    assert got[0] is out and got[1] is x
    want, _ = qm.combine_norm(y, inv, one, r, gate=torch.ones(5, 96, device="cuda"))
    assert torch.equal(out, want)


@pytest.mark.parametrize("H", [64, 2880, 9216])
def test_zero_and_nan_rows(H):
    r = torch.randn(4, H, device="cuda")
    r[0] = 0
    r[2, H - 1] = float("nan")
    w = torch.ones(H, device="cuda")
    x, _ = qm.add_norm(r, w)
    assert not x[0].any() and torch.isnan(x[2]).all() and torch.isfinite(x[[1, 3]]).all()


def test_no_rows_and_refusals():
    z, w = torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda")
    assert qm.add_norm(z, w)[0].shape == (0, 64)
    out, x = qm.combine_norm(z, torch.zeros(0, dtype=torch.int32, device="cuda"),
                             torch.zeros(0, 2, device="cuda"), z, next_weight=w)
    assert out.shape == x.shape == (0, 64)
    r = torch.zeros(4, 64, device="cuda")
    with pytest.raises(TypeError):
        qm.add_norm(r.half(), w)
    with pytest.raises(ValueError):
        qm.add_norm(r, w[:32])
    with pytest.raises(ValueError):
        qm.add_norm(r.t().contiguous().t(), w)
    with pytest.raises(ValueError):
        qm.add_norm(r, w, delta=r[:2])
    with pytest.raises(qm.MoeError):
        qm.add_norm(r[:, :40].contiguous(), w[:40])
    y, inv = torch.zeros(8, 64, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    k2 = torch.zeros(4, 2, device="cuda")
    with pytest.raises(TypeError):     # parameters of two types
        qm.combine_norm(y, inv, k2, r, post_weight=w, next_weight=w.bfloat16())
    with pytest.raises(ValueError):
        qm.combine_norm(y, inv, k2, r, gate=torch.zeros(2, 64, device="cuda"))
    with pytest.raises(ValueError):
        qm.combine_norm(y, inv, k2, r, x=r.bfloat16())


def test_rows_past_32_bits():
    T, H = 70000, 32768 - 32     # the stream holds more than 2^31 values
    r = torch.zeros(T, H, dtype=BF, device="cuda")
    r[-2:] = torch.randn(2, H, device="cuda").to(BF)
    w = torch.ones(H, dtype=BF, device="cuda")
    x, out = qm.add_norm(r, w, delta=r)
    xt, ot = qm.add_norm(r[-2:].contiguous(), w, delta=r[-2:].contiguous())
    assert torch.equal(x[-2:], xt) and torch.equal(out[-2:], ot) and not x[:-2].any()


# --------------------------------------------------------------------- the block as a whole


class Block:
    """Entry norm, routing, microscaled expert FFN and exit norm of one layer."""

    def __init__(self, T, H=256, I=192, E=8, k=2, fmt="mxfp6", seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.T, self.H, self.I, self.E, self.k, self.fmt = T, H, I, E, k, fmt
        self.resid, self.delta = (2 * rand(T, H)).to(BF), rand(T, H).to(BF)
        self.w_in, self.w_post, self.w_next = ((1 + 0.1 * rand(H)).to(BF) for _ in range(3))
        self.wr = (rand(E, H) / H ** 0.5).to(BF)
        # a loader's path: matrices quantised, then packed
        self.m = {n: rand(E, r, K) / K ** 0.5 for n, r, K in
                  (("gate", I, H), ("up", I, H), ("down", H, I))}
        self.planes = {}
        for n, m in self.m.items():
            self.planes[n + "_q"], self.planes[n + "_s"] = qm.mx_quantize(m.to(BF), "mxfp4")
        self.pool = qm.Pool.from_canonical("mxfp4", H, I, self.planes)
        self.slot_map = torch.arange(E, dtype=torch.int32, device="cuda")

    def __call__(self):
        x, r = qm.add_norm(self.resid, self.w_in, delta=self.delta)
        ids, w = qm.route(x, self.wr, None, self.k)
        _, off, perm, inv = qm.bucket(ids, self.E)
        xq, xs = qm.mx_quantize(x, self.fmt)
        h, y = qm.mx_expert_ffn(self.pool, self.slot_map, xq, xs, self.fmt, self.k, off, perm)
        out, nxt = qm.combine_norm(y, inv, w, r, post_weight=self.w_post, scale=0.5,
                                   next_weight=self.w_next)
        self.mid = dict(x=x, r=r, ids=ids, w=w, off=off, perm=perm, inv=inv, h=h, y=y)
        return out, nxt


@pytest.mark.parametrize("T", [1, 7, 90])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp6"])
def test_block(T, fmt):
    """Every stage against the oracle at the GPU's inputs to it."""
    b = Block(T, fmt=fmt, seed=T)
    out, nxt = b()
    m = b.mid
    # the loaded experts: the oracle's own quantisation gives the same planes
    W = {}
    for n in ("gate", "up", "down"):
        c, s = mx.quantize(d(b.m[n].to(BF)), "mxfp4")
        assert np.array_equal(b.planes[n + "_q"].cpu().numpy(), mx.pack(c, "mxfp4"))
        W[n] = mx.dequantize(mx.pack(c, "mxfp4"), s, "mxfp4")

    def rounded(v):
        c, s = mx.quantize(v, fmt)
        return mx.dequantize(mx.pack(c, fmt), s, fmt)

    xq, hq = rounded(d(m["x"])), rounded(d(m["h"]))
    perm, off = m["perm"].cpu().numpy(), m["off"].cpu().numpy()
    for e in range(b.E):
        at = slice(off[e], off[e + 1])
        gt, u = xq[perm[at] // b.k] @ W["gate"][e].T, xq[perm[at] // b.k] @ W["up"][e].T
        a = gt / (1 + np.exp(-gt)) * u
        assert (np.abs(d(m["h"])[at] - a) <= 2.0 ** -8 * np.abs(a) + 1e-5).all()
        y = hq[at] @ W["down"][e].T
        assert (np.abs(d(m["y"])[at] - y) <= 1e-5 * (1 + np.abs(y))).all()
    s, want = mx.combine_norm(d(m["y"]), m["inv"].cpu().numpy(), d(m["w"]), d(m["r"]), 1e-6,
                              d(b.w_post), None, 0.5, d(b.w_next))
    assert (np.abs(d(out) - s) <= 2.0 ** -8 * np.abs(s) + 1e-4).all()
    assert (np.abs(d(nxt) - want) <= 2.0 ** -8 * np.abs(want) + 1e-4).all()
    # and the block follows the layer that keeps its activations in bf16: the formats' own
    # error, at most half a step of 1/8 (1/2) relative to a block's values near its largest
    ref, _ = qm.layer(b.pool, b.slot_map, b.wr, None, m["x"], b.k)
    moe = qm.combine(m["y"], m["inv"], m["w"])
    rel = float((moe - ref).norm() / ref.norm())
    assert rel < (0.25 if fmt == "mxfp4" else 0.0625), rel


@pytest.mark.parametrize("T", [1, 33])
def test_block_in_a_graph(T):
    """Captured once, replayed on new inputs with eager work and synchronisation between;
    every replay equals the eager result."""
    b = Block(T)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        b()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out, nxt = b()
    for i in range(4):
        b.resid.copy_((torch.randn(T, b.H, device="cuda") * (i + 1)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), nxt.clone()
        want = b()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_streams_at_once():
    """Two blocks on two streams share nothing: each gives what it gives alone."""
    a, b = Block(40, seed=1), Block(3, seed=2)
    alone = [[t.clone() for t in p()] for p in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for p, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                got.append(p())
        torch.cuda.synchronize()
        for g, w in zip(got, alone):
            assert all(torch.equal(x, y) for x, y in zip(g, w))
