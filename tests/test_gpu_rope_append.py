"""Rotary positions and the append to a paged cache, against 64-bit forms."""
import pytest

torch = pytest.importorskip("torch")
import attention_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_gemv_amd as qm
    return qm


def _plan(qm, dim, layout, scale=1.0, base=10000.0):
    i = torch.arange(dim // 2, dtype=torch.float64)
    return qm.Rope((base ** (-2 * i / dim)).to(DEV), layout, scale)


def _randn(*shape, seed=0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


# -------------------------------------------------------------------------------- rope


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("T,heads,D,dim", [(1, 1, 2, 2), (1, 40, 128, 128), (5, 3, 64, 32),
                                           (7, 2, 20, 6), (9, 5, 96, 96), (6, 1, 80, 64),
                                           (3, 2, 256, 16), (2, 3, 1024, 1024), (301, 4, 64, 64),
                                           (4, 3, 7, 4)])
def test_rope(qm, layout, dtype, T, heads, D, dim):
    x = _randn(T, heads, D, dtype=dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    plan = _plan(qm, dim, layout, 1.25)
    got = qm.rope(x, pos.to(DEV), plan)
    want, tol = ref.rope(x, pos, plan.freq, layout, 1.25)
    ref.near(got, want, tol + ref.rounded(want, dtype), "rope")
    assert torch.equal(got[..., dim:], x[..., dim:])


@pytest.mark.parametrize("pos", [0, 1, -1, 131071, (1 << 31) - 1, -(1 << 31)])
def test_rope_far_positions(qm, pos):
    x = _randn(3, 2, 64)
    p = torch.full((3,), pos, dtype=torch.int64).to(torch.int32)
    plan = _plan(qm, 64, "half", base=150000.0)
    want, tol = ref.rope(x, p, plan.freq, "half", 1.0)
    ref.near(qm.rope(x, p.to(DEV), plan), want, tol + ref.rounded(want, F32), "far")
    if pos == 0:
        assert torch.equal(qm.rope(x, p.to(DEV), plan), x)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_rope_strided_and_in_place(qm, layout, dtype, off):
    """Heads inside wider rows, at any alignment; what lies around them stays."""
    T, heads, D = 11, 3, 48
    row = _randn(T, 1000, dtype=dtype)
    view = lambda t: t[:, off:off + heads * 64].unflatten(1, (heads, 64))[..., :D]  # noqa: E731
    x = view(row)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 1000
    plan = _plan(qm, 32, layout)
    want, tol = ref.rope(x, pos, plan.freq, layout, 1.0)
    tol = tol + ref.rounded(want, dtype)
    out = torch.full_like(row, 7.0)
    qm.rope(x, pos, plan, out=view(out))
    ref.near(view(out), want, tol)
    around = torch.ones_like(row, dtype=torch.bool)
    view(around).fill_(False)
    assert (out[around] == 7).all()
    here = row.clone()
    assert qm.rope(view(here), pos, plan, out=view(here)).data_ptr() == view(here).data_ptr()
    assert torch.equal(view(here), view(out)) and torch.equal(here[around], row[around])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_inverse_is_the_gradient(qm, layout):
    """The map is linear in x: its gradient is the transposed map. Against the formula's matrix, and
    against differences, which are exact for a linear map up to rounding."""
    T, heads, D, dim, scale = 3, 2, 16, 12, 1.5
    plan = _plan(qm, dim, layout, scale)
    pos = torch.tensor([0, 5, 70000], dtype=torch.int32, device=DEV)
    g = _randn(T, heads, D, seed=3)
    grad = qm.rope(g, pos, plan, inverse=True)
    want, tol = ref.rope(g, pos, plan.freq, layout, scale, inverse=True)
    ref.near(grad, want, tol + ref.rounded(want, F32), "formula")
    for d in range(D):
        e = torch.zeros(T, heads, D, device=DEV)
        e[..., d] = 1.0
        col = qm.rope(e, pos, plan)         # derivative of every output by value d
        diff = (col.double() * g.double()).sum(-1)
        # two values of a column meet, each within 8 half steps of scale, and grad's own 10
        tol_d = 20 * ref.F32 * scale * g.double().abs().sum(-1)
        assert ((diff - grad[..., d].double()).abs() <= tol_d).all(), d


def test_rope_many_rows(qm):
    """More tokens than one launch takes."""
    T = (1 << 23) + 5
    x = torch.ones(T, 1, 2, device=DEV, dtype=BF)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    plan = qm.Rope(torch.tensor([0.5], dtype=torch.float64, device=DEV))
    got = qm.rope(x, pos, plan)
    at = torch.tensor([0, 1, (1 << 23) - 1, 1 << 23, T - 1])
    want, tol = ref.rope(x[at.to(DEV)], pos[at.to(DEV)], plan.freq, "half", 1.0)
    ref.near(got[at.to(DEV)], want, tol + ref.rounded(want, BF), "many")


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_frequencies(qm, scaling):
    dim, base, f, orig = 64, 10000.0, 8.0, 4096
    p = qm.Rope.make(dim, base, scaling=scaling, factor=f, original=orig)
    freq = p.freq.cpu()
    plain = torch.tensor([base ** (-2 * i / dim) for i in range(dim // 2)], dtype=torch.float64)
    turns = orig * plain / (2 * torch.pi)
    assert p.scale == (pytest.approx(0.1 * torch.tensor(8.0).log().item() + 1)
                       if scaling == "yarn" else 1.0)
    if scaling == "none":
        assert torch.allclose(freq, plain, rtol=1e-13)
    elif scaling == "linear":
        assert torch.allclose(freq, plain / f, rtol=1e-13)
    elif scaling == "ntk":
        assert freq[0] == 1 and torch.isclose(freq[-1], plain[-1] / f, rtol=1e-12)
    else:   # fast pairs kept, slow ones slowed, in between the ramp falls
        assert torch.allclose(freq[turns > 40], plain[turns > 40], rtol=1e-13)
        assert torch.allclose(freq[turns < 0.7], plain[turns < 0.7] / f, rtol=1e-13)
        ratio = freq / plain
        assert (ratio.diff() <= 1e-12).all() and (ratio >= 1 / f - 1e-12).all()


# ------------------------------------------------------------------------------ append


def _caches(qm, order, n_pages, page, H, D, dtype):
    """A cache whose tensors have one of several orders, and what backs them."""
    if order == "heads":       # [page, head, token, D]
        kv = qm.KvCache.empty(n_pages, page, H, D, dtype)
        kv.k.view(torch.uint8).fill_(0x11), kv.v.view(torch.uint8).fill_(0x22)
        return kv
    if order == "tokens":
        k, v = (torch.zeros(n_pages, page, H, D, device=DEV).to(dtype) for _ in range(2))
    elif order == "joined":    # keys and values of a page in one tensor
        both = torch.zeros(n_pages, 2, page, H, D, device=DEV).to(dtype)
        k, v = both[:, 0], both[:, 1]
    else:                      # rows wider than a head
        both = torch.zeros(n_pages, page, H, 2 * D + 16, device=DEV).to(dtype)
        k, v = both[..., :D], both[..., D + 16:]
    return qm.KvCache(k, v)


def _batch(qm, new, total, page, spare=2, seed=0, hints=True):
    g = torch.Generator().manual_seed(seed)
    need = [-(-t // page) for t in total]
    order = torch.randperm(sum(need) + spare, generator=g).to(torch.int32)
    table = torch.full((len(new), max(max(need), 1) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    start = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    return qm.KvBatch(start.to(DEV), torch.tensor(total, dtype=torch.int32, device=DEV),
                      table.to(DEV), max(new) if hints else 0, max(total) if hints else 0), \
        sum(need) + spare, table


CASES = [   # new tokens, keys after them
    ([1], [1]), ([1, 1, 1], [7, 1, 40]), ([5, 1, 0, 9], [5, 33, 12, 30]), ([130], [200]),
    ([0, 3, 0], [4, 3, 0]),
]


@pytest.mark.parametrize("new,total", CASES)
@pytest.mark.parametrize("page", [1, 5, 16])
@pytest.mark.parametrize("order,dtype,cache,layout,dim", [
    ("heads", BF, BF, "half", 32), ("tokens", FP, FP, "interleaved", 32),
    ("joined", BF, E4, "half", 16), ("wide", F32, BF, "interleaved", 6), ("tokens", BF, FP, None, 0),
    ("heads", FP, E4, None, 0)])
def test_append(qm, new, total, page, order, dtype, cache, layout, dim):
    Hkv, G, D, pad = 3, 2, 32, 3
    batch, n_pages, table = _batch(qm, new, total, page)
    kv = _caches(qm, order, n_pages, page, Hkv, D, cache)
    T = sum(new)
    row = _randn(T + pad, (G + 2) * Hkv * D, dtype=dtype).unflatten(1, ((G + 2) * Hkv, D))
    q, k, v = row[:, :G * Hkv], row[:, G * Hkv:(G + 1) * Hkv], row[:, (G + 1) * Hkv:]
    plan = None if layout is None else _plan(qm, dim, layout, 1.1)
    before = kv.k.clone(), kv.v.clone()
    q_out = torch.full_like(q, 5.0)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = qm.kv_append(kv, batch, k, v, rope=plan, q=q, q_out=q_out, err_flags=flags)
    assert got is q_out and flags.item() == 0
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(new, total)]).to(torch.int32)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).long()

    def turned(x):
        if plan is None:
            return x.double().cpu(), torch.zeros(x.shape, dtype=torch.float64)
        return ref.rope(x, pos, plan.freq, layout, 1.1)

    want, tol = turned(q[:T])
    ref.near(q_out[:T], want, tol + ref.rounded(want, dtype), "q")
    assert (q_out[T:] == 5).all()
    touched = torch.zeros(n_pages, page, dtype=torch.bool)
    place = table[seq, pos.long() // page].long(), pos.long() % page
    touched[place] = True
    for x, plane, old in ((k, kv.k, before[0]), (v, kv.v, before[1])):
        want, tol = turned(x[:T]) if x is k else (x[:T].double().cpu(), 0.0)
        if cache == E4:
            want = want.clamp(-448, 448)
        plane, old = plane.float().cpu(), old.float().cpu()
        ref.near(plane[place], want, tol + ref.rounded(want, cache) * (1 + 2.0 ** -20), "cache")
        assert torch.equal(plane[~touched], old[~touched])


def test_append_codes_bit_by_bit(qm):
    """Every fp16 value into an 8-bit cache: the nearest code, saturated; a head's scale divides."""
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(FP).view(-1, 2, 16).to(DEV)
    T = x.shape[0]
    scales = torch.tensor([1.0, 0.37], device=DEV)
    kv = qm.KvCache(*(torch.zeros(T // 16, 16, 2, 16, device=DEV).to(E4) for _ in range(2)),
                    scales, torch.ones(2, device=DEV))
    table = torch.arange(T // 16, dtype=torch.int32, device=DEV)[None]
    batch = qm.KvBatch(torch.tensor([0, T], dtype=torch.int32, device=DEV),
                       torch.tensor([T], dtype=torch.int32, device=DEV), table)
    qm.kv_append(kv, batch, x, x)
    for plane, s in ((kv.k, scales), (kv.v, torch.ones(2, device=DEV))):
        want = (x.float() / s[:, None]).clamp(-448, 448).to(E4).view(torch.uint8)
        got = plane.reshape(T, 2, 16).view(torch.uint8)
        nan = x.isnan()
        assert torch.equal(got[~nan], want[~nan])
        assert plane.reshape(T, 2, 16).float().isnan()[nan].all()


def test_append_positions_and_in_place_queries(qm):
    """Turned by given positions; queries in place; the cache's places stay the sequence's."""
    batch, n_pages, table = _batch(qm, [4, 2], [9, 2], 4)
    kv = _caches(qm, "tokens", n_pages, 4, 2, 16, BF)
    x = _randn(6, 6, 16, dtype=BF)
    pos = torch.tensor([100, 3, -7, 5000, 0, 1 << 30], dtype=torch.int32, device=DEV)
    plan = _plan(qm, 16, "half")
    q = x[:, :2].clone()
    assert qm.kv_append(kv, batch, x[:, 2:4], x[:, 4:], rope=plan, positions=pos, q=q,
                        q_out=q) is q
    assert torch.equal(q, qm.rope(x[:, :2], pos, plan))
    at = torch.tensor([5, 6, 7, 8, 0, 1])
    place = table[torch.tensor([0, 0, 0, 0, 1, 1]), at // 4].long(), at % 4
    assert torch.equal(kv.k.cpu()[place], qm.rope(x[:, 2:4], pos, plan).cpu())
    assert torch.equal(kv.v.cpu()[place], x[:, 4:].cpu())


def test_append_bad_places_are_left_out(qm):
    """Pages outside the cache, positions below zero and past the table: flagged, not followed;
    the other tokens go in."""
    page = 4
    kv = _caches(qm, "tokens", 3, page, 1, 16, BF)
    table = torch.tensor([[0, 7], [-2, 1], [2, -1]], dtype=torch.int32, device=DEV)
    # sequence 0: positions 2..5 (4, 5 on page 7 of 3); 1: 3..4 (3 on page -2); 2: -1..1
    batch = qm.KvBatch(torch.tensor([0, 4, 6, 9], dtype=torch.int32, device=DEV),
                       torch.tensor([6, 5, 2], dtype=torch.int32, device=DEV), table)
    x = _randn(9, 1, 16, dtype=BF)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    qm.kv_append(kv, batch, x, x, err_flags=flags)
    assert flags.item() == 1
    want = torch.zeros(3, page, 1, 16, dtype=BF)
    for t, (p, r) in {0: (0, 2), 1: (0, 3), 5: (1, 0), 7: (2, 0), 8: (2, 1)}.items():
        want[p, r] = x[t].cpu()
    assert torch.equal(kv.k.cpu(), want) and torch.equal(kv.v.cpu(), want)
    # past the table
    flags.zero_()
    batch = qm.KvBatch(torch.tensor([0, 2], dtype=torch.int32, device=DEV),
                       torch.tensor([9], dtype=torch.int32, device=DEV), table[2:])
    kv.k.zero_()
    qm.kv_append(kv, batch, x[:2], x[:2], err_flags=flags)
    assert flags.item() == 1 and not kv.k.any()


def test_append_many_sequences(qm):
    """More sequences than the search probes at once, some without new tokens."""
    g = torch.Generator().manual_seed(5)
    new = torch.randint(0, 3, (5000,), generator=g).tolist()
    total = [n + int(torch.randint(0, 9, (), generator=g)) for n in new]
    batch, n_pages, table = _batch(qm, new, total, 4)
    kv = _caches(qm, "tokens", n_pages, 4, 1, 16, BF)
    x = _randn(sum(new), 1, 16, dtype=BF)
    qm.kv_append(kv, batch, x, x)
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(new, total)])
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).long()
    assert torch.equal(kv.k.cpu()[table[seq, pos // 4].long(), pos % 4], x.cpu())


def test_append_far_pages(qm):
    """Places past 2^32 elements of a plane."""
    n_pages = (1 << 32) // (64 * 2 * 64) + 3
    k, v = (torch.zeros(n_pages, 64, 2, 64, dtype=E4, device=DEV) for _ in range(2))
    kv = qm.KvCache(k, v)
    batch = qm.KvBatch(torch.tensor([0, 2], dtype=torch.int32, device=DEV),
                       torch.tensor([65], dtype=torch.int32, device=DEV),
                       torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=DEV))
    x = torch.full((2, 2, 64), 3.0, dtype=BF, device=DEV)
    qm.kv_append(kv, batch, x, x)
    assert (kv.k[n_pages - 1, 63].float() == 3).all() and (kv.v[n_pages - 2, 0].float() == 3).all()
    assert int(kv.k.view(torch.uint8)[:4].any()) == 0
    assert not kv.k.view(torch.uint8)[n_pages - 1, :63].any()
