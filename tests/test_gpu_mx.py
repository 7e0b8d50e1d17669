"""Microscaled formats and the expert products on them, against the fp64 oracle.

Codes, scales and dequantised values match exactly. The products accumulate K terms in fp32:
each y is within (K/64 + 8) roundings of half a step, 2^-24 of sum |w a| each, of the exact
sum (one add per instruction's 64 or 128 terms, the terms' own sum, and the waves' partials).
h adds its own rounding to bf16 (half a step, 2^-8 of the value), the propagation of g's and
u's errors through silu(g) u, and 2^-20 of the value for the fp32 exponential and division.
"""
import numpy as np
import pytest

from oracle import mx

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FMTS = ["mxfp4", "mxfp6"]


def _quantize_check(x, fmt):
    """x: CPU tensor; compares codes and scales bit by bit."""
    q, s = qm.mx_quantize(x.cuda(), fmt)
    c, sr = mx.quantize(x.double().numpy(), fmt)
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(q.cpu().numpy(), mx.pack(c, fmt))
    return q, s


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_quantize_every_16_bit_pattern(fmt, dt):
    """Every value of the type, non-finite ones among them, as blocks of neighbours (one
    scale) and shuffled."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    g = torch.Generator().manual_seed(1)
    x = bits.view(DT[dt])
    fin = x[torch.isfinite(x)]
    fin = fin[torch.randperm(len(fin), generator=g)][:len(fin) // 32 * 32]
    _quantize_check(x.view(-1, 64), fmt)
    _quantize_check(fin.view(-1, 32), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 32), (1, 2880), (7, 96), (333, 2080), (1001, 64)])
def test_quantize_fp32(fmt, rows, K):
    g = torch.Generator().manual_seed(rows + K)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g))
    _quantize_check(x, fmt)
    # values on and next to the borders between codes, at every scale that has them exactly
    n = torch.randint(-128, 129, (rows, K), generator=g).float() / 16
    n[:, ::32] = 4.0 + torch.randint(0, 64, n[:, ::32].shape, generator=g) / 16
    e = torch.randint(-126, 120, (rows, K // 32), generator=g).repeat_interleave(32, 1)
    x = torch.ldexp(n, e)
    _quantize_check(x, fmt)
    _quantize_check(torch.nextafter(x, torch.tensor(float("inf"))), fmt)
    _quantize_check(torch.nextafter(x, torch.tensor(0.0)), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_special_blocks(fmt):
    x = torch.zeros(9, 32)
    x[0, 1] = -0.0
    x[1, 4], x[1, 5] = 2.0 ** -149, -2.0 ** -127      # subnormals
    x[2, :] = 3.4e38
    x[3, 31] = float("inf")
    x[4, 0] = float("-inf")
    x[5, 9] = float("nan")
    x[6, :] = 2.0 ** -126
    x[7, 0], x[7, 1] = 1.0, 1e-30
    q, s = _quantize_check(x, fmt)
    assert s[3:6].flatten().tolist() == [255] * 3
    v = qm.mx_dequantize(q, s, fmt, torch.float32).cpu()
    assert torch.isnan(v[3:6]).all() and torch.isfinite(v[[0, 1, 2, 6, 7, 8]]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_dequantize_every_code_and_scale(fmt, dt):
    n = 1 << mx.BITS[fmt]
    codes = np.tile(np.arange(64, dtype=np.uint8) % n, (256, 1))
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 2, 1)
    q = mx.pack(codes, fmt)
    got = qm.mx_dequantize(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), fmt, DT[dt])
    # exact in fp32 (5 digits, 2^-130 the smallest), so one rounding to the type
    want = torch.from_numpy(mx.dequantize(q, s, fmt)).float().to(DT[dt])
    assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=-1e9, posinf=1e39, neginf=-1e39),
                       torch.nan_to_num(want.float(), nan=-1e9, posinf=1e39, neginf=-1e39))
    assert torch.isnan(got[255]).all()


def test_quantize_past_32_bits():
    """More than 2^32 values: the last rows equal the same rows alone."""
    rows, K = 1 << 17, 32800
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    x.fill_(0.5)
    x[-3:] = torch.randn(3, K, device="cuda").bfloat16()
    q, s = qm.mx_quantize(x, "mxfp6")
    qt, st = qm.mx_quantize(x[-3:].contiguous(), "mxfp6")
    assert torch.equal(q[-3:], qt) and torch.equal(s[-3:], st)
    v = qm.mx_dequantize(q, s, "mxfp6")
    assert torch.equal(v[-3:], qm.mx_dequantize(qt, st, "mxfp6"))
    assert bool((v[:1000] == 0.5).all()) and bool((v[-1000:-3] == 0.5).all())


# ------------------------------------------------------------------------------ products


def _weights(g, S, rows, K):
    """Random codes and scales; canonical planes on the GPU, fp64 values here."""
    q = torch.randint(0, 256, (S, rows, K // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(118, 124, (S, rows, K // 32), generator=g, dtype=torch.uint8)
    return q, s


class Problem:
    def __init__(self, T, H, I, E, k, fmt, seed=0, missing=(), ids=None, scale_spread=4):
        g = torch.Generator().manual_seed(seed)
        self.T, self.H, self.I, self.E, self.k, self.fmt = T, H, I, E, k, fmt
        S = E + 2
        self.w = {"gate": _weights(g, S, I, H), "up": _weights(g, S, I, H),
                  "down": _weights(g, S, H, I)}
        planes = {}
        for n, (q, s) in self.w.items():
            planes[n + "_q"], planes[n + "_s"] = q, s
        self.pool = qm.Pool.from_canonical("mxfp4", H, I, planes)
        self.slots = torch.randperm(S, generator=g)[:E].to(torch.int32)
        for e in missing:
            self.slots[e] = -1
        if ids is None:
            ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
        self.ids = ids.to(torch.int32).reshape(T, k)
        self.slot_map = self.slots.cuda()
        self.counts, self.offsets, self.perm, self.inv = qm.bucket(self.ids.cuda(), E)

        def rows(n, K):
            q = torch.randint(0, 256, (n, K * mx.BITS[fmt] // 8), generator=g, dtype=torch.uint8)
            s = torch.randint(127 - scale_spread, 127 + scale_spread, (n, K // 32), generator=g,
                              dtype=torch.uint8)
            return q, s

        self.x, self.h = rows(T, H), rows(T * k, I)
        self.xd, self.hd = [t.cuda() for t in self.x], [t.cuda() for t in self.h]

    def value(self, name, slot):
        q, s = self.w[name]
        return mx.dequantize(q[slot].numpy(), s[slot].numpy(), "mxfp4")

    def buckets(self):
        off = self.offsets.cpu().numpy()
        for e in range(self.E):
            if off[e + 1] > off[e]:
                yield e, int(self.slots[e]), slice(off[e], off[e + 1])

    def gate_up(self, **kw):
        return qm.mx_expert_gate_up(self.pool, self.slot_map, *self.xd, self.fmt, self.k,
                                    self.offsets, self.perm, **kw)

    def down(self, **kw):
        return qm.mx_expert_down(self.pool, self.slot_map, self.T, self.k, self.offsets, *self.hd,
                                 self.fmt, **kw)

    def check_gate_up(self, h, experts=None):
        x = mx.dequantize(self.x[0].numpy(), self.x[1].numpy(), self.fmt)
        perm = self.perm.cpu().numpy()
        h = h.float().cpu().numpy().astype(np.float64)
        eps = (self.H / 64 + 8) * 2.0 ** -24
        for e, slot, at in self.buckets():
            if experts is not None and e not in experts:
                continue
            if slot < 0:
                assert not h[at].any(), f"expert {e}"
                continue
            r = x[perm[at] // self.k]
            wg, wu = self.value("gate", slot), self.value("up", slot)
            gt, u = r @ wg.T, r @ wu.T
            dg, du = eps * (np.abs(r) @ np.abs(wg).T), eps * (np.abs(r) @ np.abs(wu).T)
            with np.errstate(over="ignore"):
                sg = 1 / (1 + np.exp(-gt))
            a = gt * sg * u
            # |silu'| <= 1.1 everywhere; the products of both errors beside each alone
            tol = 2.0 ** -8 * np.abs(a) + 2.0 ** -20 * np.abs(a) + \
                1.1 * dg * np.abs(u) + du * np.abs(gt * sg) + 1.1 * dg * du + 2.0 ** -133
            bad = ~(np.abs(h[at] - a) <= tol)
            assert not bad.any(), f"expert {e}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}"

    def check_down(self, y, experts=None):
        h = mx.dequantize(self.h[0].numpy(), self.h[1].numpy(), self.fmt)
        y = y.cpu().numpy().astype(np.float64)
        eps = (self.I / 64 + 8) * 2.0 ** -24
        for e, slot, at in self.buckets():
            if experts is not None and e not in experts:
                continue
            if slot < 0:
                assert not y[at].any(), f"expert {e}"
                continue
            w = self.value("down", slot)
            bad = ~(np.abs(y[at] - h[at] @ w.T) <= eps * (np.abs(h[at]) @ np.abs(w).T))
            assert not bad.any(), f"expert {e}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}"


SHAPES = [
    # T, H, I, E, k, missing
    (1, 32, 32, 1, 1, ()), (1, 64, 32, 4, 2, ()), (1, 2880, 64, 8, 4, ()), (2, 96, 160, 5, 3, (1,)),
    (4, 256, 512, 8, 2, ()), (15, 224, 96, 8, 8, (0, 7)), (16, 128, 2080, 6, 2, ()),
    (17, 160, 288, 3, 2, ()), (64, 544, 320, 8, 2, (3,)), (129, 96, 128, 2, 1, ()),
    (300, 288, 224, 17, 4, (2, 16)), (777, 128, 96, 4, 3, ()),
]


@pytest.mark.parametrize("path", [qm.PATH_AUTO, qm.PATH_GEMV, qm.PATH_GROUPED])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,I,E,k,missing", SHAPES)
def test_products(T, H, I, E, k, missing, fmt, path):
    p = Problem(T, H, I, E, k, fmt, seed=T + H, missing=missing)
    p.check_gate_up(p.gate_up(path=path))
    p.check_down(p.down(path=path))


@pytest.mark.parametrize("path", [qm.PATH_GEMV, qm.PATH_GROUPED])
@pytest.mark.parametrize("fmt", FMTS)
def test_products_wide(fmt, path):
    """Many experts with few rows and one with most of them; more row groups than a tile."""
    g = torch.Generator().manual_seed(5)
    T, E, k = 600, 128, 4
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    ids[:500, 0] = 37
    p = Problem(T, 768, 352, E, k, fmt, seed=9, ids=ids)
    few = {37, 0, 1, 64, 127}
    p.check_gate_up(p.gate_up(path=path), few)
    p.check_down(p.down(path=path), few)


@pytest.mark.parametrize("path", [qm.PATH_GEMV, qm.PATH_GROUPED])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [9, 150, 450])
def test_products_long_rows(T, fmt, path):
    """Rows of more than 128 blocks, odd in number."""
    p = Problem(T, 4128, 4192, 2, 1, fmt, seed=T)
    p.check_gate_up(p.gate_up(path=path))
    p.check_down(p.down(path=path))


# Enough tiles for the taller ones: 64 rows (T = 700, 32 experts of 87 rows on average) and 128
# (T = 6500, 8 experts of 1625), for the product whose output is the wide one; short rows, rows
# whose last step is ragged, and rows of more than 128 blocks.
TALL = [(700, 160, 1056, 32, 4), (700, 2080, 160, 32, 4), (700, 4192, 1056, 32, 4),
        (700, 2080, 4192, 32, 4), (6500, 32, 1056, 8, 2), (6500, 2080, 32, 8, 2),
        (6500, 288, 1056, 8, 2), (6500, 2080, 352, 8, 2), (6500, 4192, 1056, 8, 2),
        (6500, 2080, 4192, 8, 2)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,I,E,k", TALL)
def test_products_tall(T, H, I, E, k, fmt):
    """A miss, an expert whole, a NaN block, and rows past the last bucket."""
    p = Problem(T, H, I, E, k, fmt, seed=H + I, missing=(3,))
    n = T * k
    if I == 1056:
        h = p.gate_up()
        p.check_gate_up(h, {1, 3})
        p.xd[1][5, H // 32 - 1] = 255
        h2 = p.gate_up()
        hit = ((p.perm // k) == 5) & (h.abs().sum(1) > 0)   # but for the pair that misses
        assert 1 <= int(hit.sum()) <= k
        assert torch.isnan(h2[hit]).all() and torch.equal(h2[~hit], h[~hit])
    else:
        y = p.down()
        p.check_down(y, {1, 3})
        p.hd[1][n - 1, I // 32 - 1] = 255
        y2 = p.down()
        assert torch.isnan(y2[n - 1]).all() and torch.equal(y2[:-1], y[:-1])
        p.offsets.clamp_(max=n - 9)
        y2.fill_(7)
        p.down(y=y2)
        assert bool((y2[n - 9:] == 7).all()) and torch.equal(y2[:n - 9], y[:n - 9])


@pytest.mark.parametrize("path", [qm.PATH_GEMV, qm.PATH_GROUPED])
@pytest.mark.parametrize("fmt", FMTS)
def test_scales_far_apart(fmt, path):
    """Neighbouring blocks' scales 2^-60 to 2^59: the bound is on sum |w a| all the same."""
    p = Problem(70, 288, 352, 3, 2, fmt, seed=4, scale_spread=60)
    p.check_down(p.down(path=path))


@pytest.mark.parametrize("T", [2, 90])
def test_a_stream_of_the_callers(T):
    p = Problem(T, 256, 160, 8, 2, "mxfp4")
    h, y = p.gate_up(), p.down()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    h2, y2 = p.gate_up(stream=st), p.down(stream=st)
    st.synchronize()
    assert torch.equal(h, h2) and torch.equal(y, y2)


@pytest.mark.parametrize("path", [qm.PATH_GEMV, qm.PATH_GROUPED])
def test_one_expert_twice_for_a_token(path):
    """16 tokens that name one expert in every choice: 64 rows of it on the few-token path."""
    p = Problem(16, 96, 64, 4, 4, "mxfp6", ids=torch.full((16, 4), 2))
    p.check_gate_up(p.gate_up(path=path))
    p.check_down(p.down(path=path))


@pytest.mark.parametrize("path", [qm.PATH_GEMV, qm.PATH_GROUPED])
@pytest.mark.parametrize("T", [3, 200])
def test_nan_block_stays_in_its_row(T, path):
    p = Problem(T, 160, 96, 4, 2, "mxfp4", seed=3)
    h0, y0 = p.gate_up(path=path), p.down(path=path)
    for t in (0, T - 1):
        p.xd[1][t, 4] = 255      # the last block: past the last whole 64 of K
        p.hd[1][t, 2] = 255
    h, y = p.gate_up(path=path), p.down(path=path)
    tok = (p.perm // p.k).long()
    hit = (tok == 0) | (tok == T - 1)
    assert torch.isnan(h[hit]).all() and torch.equal(h[~hit], h0[~hit])
    keep = torch.ones(len(y), dtype=torch.bool)
    keep[[0, T - 1]] = False
    assert torch.isnan(y[[0, T - 1]]).all() and torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("path", [qm.PATH_GEMV, qm.PATH_GROUPED])
@pytest.mark.parametrize("T", [4, 80])
def test_bad_slot_raises_the_flag(T, path):
    p = Problem(T, 64, 96, 4, 2, "mxfp4", ids=torch.tensor([[1, 3]]).repeat(T, 1))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p.slot_map[0] = 99          # an expert without rows
    p.slots[1] = -1
    p.slot_map[1] = -1          # a miss is no error
    p.check_gate_up(p.gate_up(err_flags=err, path=path))
    assert int(err) == 0
    p.slot_map[1] = 6           # the pool has slots 0 to 5
    p.check_gate_up(p.gate_up(err_flags=err, path=path))
    assert int(err) == 1
    err.zero_()
    p.slot_map[1] = -7
    p.check_down(p.down(err_flags=err, path=path))
    assert int(err) == 1


@pytest.mark.parametrize("path", [qm.PATH_GEMV, qm.PATH_GROUPED])
@pytest.mark.parametrize("T", [5, 100])
def test_rows_past_the_last_bucket_are_left(T, path):
    """A padded batch: the buckets end before T*k, and perm behind them holds anything."""
    p = Problem(T, 64, 96, 4, 2, "mxfp6")
    end = int(p.offsets[-1]) - 7
    p.offsets.clamp_(max=end)
    p.perm[end:] = 0x7FFFFFFF
    h = torch.full((2 * T, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    y = torch.full((2 * T, 64), 7.0, device="cuda")
    assert p.gate_up(h=h, path=path) is h and p.down(y=y, path=path) is y
    assert bool((h[end:] == 7).all()) and bool((y[end:] == 7).all())
    p.check_gate_up(h)
    p.check_down(y)


@pytest.mark.parametrize("path", [qm.PATH_GEMV, qm.PATH_GROUPED])
def test_same_call_same_bits(path):
    p = Problem(100, 768, 256, 8, 2, "mxfp6")
    h, y = p.gate_up(path=path), p.down(path=path)
    assert torch.equal(h, p.gate_up(path=path)) and torch.equal(y, p.down(path=path))


def test_y_past_32_bits():
    """y has more than 2^31 values; the buckets' first and last rows are checked."""
    T, H, I, E, k = 16500, 16416, 32, 8, 8   # k <= E
    ids = torch.zeros(T, k)
    ids[T // 2:] = 1
    p = Problem(T, H, I, E, k, "mxfp4", ids=ids)
    y = p.down()
    for path in (qm.PATH_AUTO, qm.PATH_GEMV):
        if path == qm.PATH_GEMV:
            y.zero_()
            p.down(y=y, path=path)
        h = mx.dequantize(p.h[0].numpy(), p.h[1].numpy(), "mxfp4")
        for e, slot, at in p.buckets():
            w = p.value("down", slot)
            for r in (at.start, at.stop - 1):
                want = w @ h[r]
                got = y[r].cpu().numpy().astype(np.float64)
                assert (np.abs(got - want) <= 9 * 2.0 ** -24 * (np.abs(w) @ np.abs(h[r]))).all()


def test_pool_past_32_bits():
    """Slots whose planes lie past 4 GiB."""
    H, I, S = 4096, 4096, 520          # 8 MiB of codes a matrix
    pool = qm.Pool.empty("mxfp4", S, H, I)
    assert pool.planes["gate_q"].numel() > 1 << 32
    g = torch.Generator().manual_seed(0)
    w = {n: _weights(g, 1, r, K) for n, r, K in (("gate", I, H), ("up", I, H), ("down", H, I))}
    for n, r, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
        q, s = w[n]
        nq, ns = q.numel(), s.numel()
        for slot in (0, S - 1):
            qm.pool_pack("mxfp4", 1, r, K, q.cuda(), s.cuda(),
                         pool.planes[n + "_q"][slot * nq:(slot + 1) * nq],
                         pool.planes[n + "_s"][slot * ns:(slot + 1) * ns])
    for T in (3, 40):
        xq, xs = qm.mx_quantize(torch.randn(T, H, device="cuda"), "mxfp4")
        ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
        _, off, perm, _ = qm.bucket(ids, 1)
        outs = [qm.mx_expert_gate_up(pool, torch.tensor([slot], dtype=torch.int32, device="cuda"),
                                     xq, xs, "mxfp4", 1, off, perm) for slot in (0, S - 1)]
        assert torch.equal(*outs) and bool(outs[0].any())
        outs = [qm.mx_expert_down(pool, torch.tensor([slot], dtype=torch.int32, device="cuda"), T,
                                  1, off, xq, xs, "mxfp4") for slot in (0, S - 1)]
        assert torch.equal(*outs) and bool(outs[0].any())


@pytest.mark.parametrize("T", [4, 150])
def test_ffn_is_its_three_calls(T):
    p = Problem(T, 256, 160, 8, 2, "mxfp6")
    h, y = qm.mx_expert_ffn(p.pool, p.slot_map, *p.xd, "mxfp6", p.k, p.offsets, p.perm,
                            h_fmt="mxfp4")
    h1 = p.gate_up()
    hq, hs = qm.mx_quantize(h1, "mxfp4")
    y1 = qm.mx_expert_down(p.pool, p.slot_map, T, p.k, p.offsets, hq, hs, "mxfp4")
    assert torch.equal(h, h1) and torch.equal(y, y1)


def test_outputs_of_the_callers():
    """Every output given; the flag of a slot outside the pool comes out of the fused call too."""
    T, H, I, k = 6, 96, 64, 2
    p = Problem(T, H, I, 4, k, "mxfp6", ids=torch.tensor([[0, 2]]).repeat(T, 1))
    x = torch.randn(T, H, device="cuda").bfloat16()
    new = lambda *s, dt=torch.uint8: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    q, s_ = new(T, qm.mx_row_bytes("mxfp6", H)), new(T, H // 32)
    assert qm.mx_quantize(x, "mxfp6", q=q, s=s_)[0] is q
    out = new(T, H, dt=torch.float32)
    assert qm.mx_dequantize(q, s_, "mxfp6", torch.float32, out=out) is out
    assert torch.equal(out, qm.mx_dequantize(q, s_, "mxfp6", torch.float32))
    h, y = new(T * k, I, dt=torch.bfloat16), new(T * k, H, dt=torch.float32)
    hq, hs = new(T * k, qm.mx_row_bytes("mxfp4", I)), new(T * k, I // 32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (p.pool, p.slot_map, q, s_, "mxfp6", k, p.offsets, p.perm)
    got = qm.mx_expert_ffn(*args, h_fmt="mxfp4", h=h, h_q=hq, h_s=hs, y=y, err_flags=err)
    assert got[0] is h and got[1] is y and int(err) == 0
    h1, y1 = qm.mx_expert_ffn(*args, h_fmt="mxfp4")
    assert torch.equal(h, h1) and torch.equal(y, y1)
    assert torch.equal(hq, qm.mx_quantize(h, "mxfp4")[0])
    p.slot_map[2] = 1000
    h2, y2 = qm.mx_expert_ffn(*args, h_fmt="mxfp4", err_flags=err)
    half = int(p.offsets[1])
    assert int(err) == 1 and torch.equal(y2[:half], y[:half]) and not y2[half:].any()
    assert not h2[half:].any()
    with pytest.raises(qm.MoeError):   # a row further on: codes at 8 bytes, not at 16
        qm.mx_dequantize(new(T + 1, 72)[1:], s_, "mxfp6")
    with pytest.raises(ValueError):
        qm.mx_quantize(x, "mxfp6", q=q[:, :-1])


def test_no_tokens():
    p = Problem(3, 64, 32, 4, 2, "mxfp4")
    z = torch.zeros(5, dtype=torch.int32, device="cuda")
    h, y = qm.mx_expert_ffn(p.pool, p.slot_map, p.xd[0][:0], p.xd[1][:0], "mxfp4", 2, z,
                            z[:0])
    assert h.shape == (0, 32) and y.shape == (0, 64)
    q, s = qm.mx_quantize(torch.zeros(0, 64, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0, 2)
    assert qm.mx_dequantize(q, s).shape == (0, 64)


def test_binding_refusals():
    p = Problem(3, 64, 32, 4, 2, "mxfp4")
    with pytest.raises(ValueError):
        p.pool, qm.mx_expert_gate_up(p.pool, p.slot_map, p.xd[0][:, :16], p.xd[1], "mxfp4", 2,
                                     p.offsets, p.perm)
    with pytest.raises(ValueError):   # planes of the other format
        qm.mx_expert_gate_up(p.pool, p.slot_map, *p.xd, "mxfp6", 2, p.offsets, p.perm)
    with pytest.raises(ValueError):
        qm.mx_expert_gate_up(p.pool, p.slot_map, *p.xd, "mxfp4", 2, p.offsets, p.perm[:-1])
    with pytest.raises(ValueError):
        qm.mx_expert_down(p.pool, p.slot_map, 3, 2, p.offsets[:-1], *p.hd, "mxfp4")
    with pytest.raises(ValueError):   # not contiguous
        qm.mx_quantize(torch.zeros(64, 64, device="cuda").t()[:, :32], "mxfp4")
    with pytest.raises(TypeError):
        qm.mx_expert_gate_up(p.pool, p.slot_map.long(), *p.xd, "mxfp4", 2, p.offsets, p.perm)
    q8 = qm.Pool.empty("q8_0", 4, 64, 32)
    with pytest.raises(qm.MoeError):
        qm.mx_expert_gate_up(q8, p.slot_map, *p.xd, "mxfp4", 2, p.offsets, p.perm)
    with pytest.raises(qm.MoeError):   # K not a multiple of 32
        qm.mx_quantize(torch.zeros(4, 48, device="cuda"), "mxfp4")
