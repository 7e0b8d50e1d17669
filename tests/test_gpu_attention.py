"""Attention over a paged cache, against the 64-bit form."""
import pytest

torch = pytest.importorskip("torch")
import attention_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_gemv_amd as qm
    return qm


class Setup:
    """A batch over a cache. Everything out of sight (page tails, spare pages, padding) is NaN."""

    def __init__(self, qm, new, total, page, Hq, Hkv, D, dtype=BF, cache=None, seed=0, pad=2,
                 order="tokens", hints=True, spare=2):
        cache = cache or dtype
        g = torch.Generator().manual_seed(seed)
        need = [-(-t // page) for t in total]
        perm = torch.randperm(sum(need) + spare, generator=g).to(torch.int32)
        self.table = torch.full((len(new), max(need) + 1), -1, dtype=torch.int32)
        n_pages = sum(need) + spare
        shape = (n_pages, page, Hkv, D)
        k, v = torch.full(shape, float("nan")), torch.full(shape, float("nan"))
        at = 0
        self.scales = None
        if cache == E4:
            self.scales = [0.5 + torch.rand(Hkv, generator=g), 0.25 + torch.rand(Hkv, generator=g)]
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
            t = torch.arange(total[b])
            rows = self.table[b, t // page].long(), t % page
            k[rows] = torch.randn(total[b], Hkv, D, generator=g)
            v[rows] = torch.randn(total[b], Hkv, D, generator=g)
        self.k, self.v = k.to(cache).to(DEV), v.to(cache).to(DEV)
        if order == "heads":
            self.k, self.v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (self.k, self.v))
        self.new, self.total, self.page, self.Hkv, self.D, self.dtype = new, total, page, Hkv, D, dtype
        self.kv = qm.KvCache(self.k, self.v, *([s.to(DEV) for s in self.scales] if self.scales else []))
        self.start = [0]
        for n in new:
            self.start.append(self.start[-1] + n)
        self.batch = qm.KvBatch(torch.tensor(self.start, dtype=torch.int32, device=DEV),
                                torch.tensor(total, dtype=torch.int32, device=DEV),
                                self.table.to(DEV), max(new) if hints else 0,
                                max(total) if hints else 0)
        T = self.start[-1]
        self.q = (1.5 * torch.randn(T + pad, Hq, D, generator=g)).to(dtype)
        self.q[T:] = float("nan")
        self.q = self.q.to(DEV)
        self.T, self.Hq, self.g = T, Hq, g

    def rows(self, b, plane):
        t = torch.arange(self.total[b])
        page = self.table[b, t // self.page].long()
        x = (self.k, self.v)[plane].float().cpu()[page.clamp(min=0), t % self.page].double()
        return x * self.scales[plane].double()[:, None] if self.scales else x

    def check(self, out, scale=None, ok=None, **kw):
        scale = self.D ** -0.5 if scale is None else scale
        for b, n in enumerate(self.new):
            if not n:
                continue
            pos = torch.arange(self.total[b] - n, self.total[b])
            rows = slice(self.start[b], self.start[b + 1])
            want, tol = ref.attend(self.q[rows].cpu(), self.rows(b, 0), self.rows(b, 1), pos, scale,
                                   ok=None if ok is None else ok[b], **kw)
            ref.near(out[rows], want, tol, f"sequence {b}")


def _run(qm, s, **kw):
    out = torch.full_like(s.q, 3.0)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert qm.attend(s.q, s.kv, s.batch, out=out, err_flags=flags, **kw) is out
    assert (out[s.T:] == 3).all(), "padding rows"
    return out, flags.item()


BATCHES = {
    "token": ([1], [1]),
    "tokens": ([1, 1, 1], [33, 1, 300]),
    "chunk": ([70], [70]),
    "later": ([37], [201]),
    "ragged": ([1, 40, 0, 5, 129], [77, 64, 9, 5, 331]),
}


@pytest.mark.parametrize("shape", BATCHES)
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 64), (6, 2, 128), (3, 3, 16), (16, 1, 80), (7, 1, 256),
                                      (40, 2, 64), (5, 5, 96)])
@pytest.mark.parametrize("dtype,cache,page", [(BF, BF, 16), (FP, FP, 5), (BF, E4, 32), (FP, E4, 1),
                                              (BF, BF, 64)])
def test_attend(qm, shape, Hq, Hkv, D, dtype, cache, page):
    s = Setup(qm, *BATCHES[shape], page, Hq, Hkv, D, dtype, cache,
              order="heads" if page > 8 else "tokens")
    out, flags = _run(qm, s)
    assert flags == 0
    s.check(out)


@pytest.mark.parametrize("shape", BATCHES)
@pytest.mark.parametrize("window,keep", [(1, 0), (8, 0), (33, 4), (128, 40), (500, 4), (64, 1000)])
@pytest.mark.parametrize("sinks", [False, True])
def test_windows(qm, shape, window, keep, sinks):
    """The evicted pages of a window are not read: their entries are taken away."""
    s = Setup(qm, *BATCHES[shape], 8, 8, 2, 64)
    table = s.table.clone()
    for b, (n, t) in enumerate(zip(s.new, s.total)):
        for p in range(table.shape[1]):
            if keep <= p * 8 and p * 8 + 8 <= t - n + 1 - window:
                table[b, p] = -1
    s.batch = qm.KvBatch(s.batch.q_start, s.batch.seq_len, table.to(DEV), max(s.new), max(s.total))
    sink = torch.linspace(-3, 4, 8).to(DEV) if sinks else None
    out, flags = _run(qm, s, window=window, keep_first=keep, sinks=sink)
    assert flags == 0
    s.check(out, window=window, keep=keep, sinks=sink)


@pytest.mark.parametrize("new,total", [([1], [40000]), ([3], [9001]), ([1, 1], [20000, 3]),
                                       ([200], [6000])])
@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("hints", [True, False])
def test_long_contexts_are_split(qm, new, total, cache, hints):
    s = Setup(qm, new, total, 16, 4, 1, 64, BF, cache, hints=hints)
    if hints and len(new) == 1 and new[0] < 4:
        assert qm.attend_scratch_bytes(s.kv, s.batch, s.T + 2, 4) > 0
    sink = torch.tensor([0.0, 2.0, -1.0, float("-inf")], device=DEV)
    out, flags = _run(qm, s, sinks=sink)
    assert flags == 0
    s.check(out, sinks=sink)
    again, _ = _run(qm, s, sinks=sink)
    assert torch.equal(out, again)


@pytest.mark.parametrize("new,total", [([1], [50]), ([40, 3], [40, 90]), ([150], [150])])
def test_not_causal(qm, new, total):
    s = Setup(qm, new, total, 16, 6, 2, 64)
    out, flags = _run(qm, s, causal=False)
    assert flags == 0
    s.check(out, causal=False)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0, 1e-30])
@pytest.mark.parametrize("new,total", [([1], [90]), ([140], [180])])
def test_scales(qm, scale, new, total):
    s = Setup(qm, new, total, 16, 4, 2, 32)
    out, _ = _run(qm, s, scale=scale)
    s.check(out, scale=scale)


@pytest.mark.parametrize("new,total", [([1], [70]), ([60], [100]), ([200, 1], [200, 3])])
def test_large_scores(qm, new, total):
    """Scores that rise by thousands along the keys, past what an exponential holds."""
    s = Setup(qm, new, total, 16, 4, 1, 64)
    ramp = torch.arange(s.k.shape[1], device=DEV).view(1, -1, 1, 1) * 4.0
    s.k.copy_((s.k.float() * ramp).to(BF))
    out, _ = _run(qm, s)
    s.check(out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("plane", ["k", "v"])
@pytest.mark.parametrize("new,total,at", [([40], [40], 17), ([40], [100], 80), ([200], [260], 130),
                                          ([3], [64], 62)])
def test_later_tokens_do_not_reach_earlier_ones(qm, bad, plane, new, total, at):
    """An infinity or NaN among one token's keys or values: the tokens before it are as they were."""
    s = Setup(qm, new, total, 16, 8, 2, 64)
    clean, _ = _run(qm, s)
    t = getattr(s, plane)
    t[s.table[0, at // 16].long(), at % 16, 1, 5] = bad
    out, _ = _run(qm, s)
    before = at - (total[0] - new[0])
    assert torch.equal(out[:max(before, 0), :], clean[:max(before, 0), :])
    assert torch.equal(out[:, :4], clean[:, :4])        # the other KV head's
    hit = out[max(before, 0):s.T, 4:].float()
    if plane == "v":
        others = [d for d in range(64) if d != 5]
        assert torch.equal(hit[..., others], clean[max(before, 0):s.T, 4:].float()[..., others])
        assert (hit[..., 5].isnan() if bad != bad else hit[..., 5] == bad).all()
    elif bad != bad:
        assert hit.isnan().all()


@pytest.mark.parametrize("window,keep", [(16, 0), (16, 4)])
@pytest.mark.parametrize("new", [1, 30, 140])
def test_values_before_the_window_do_not_reach_it(qm, window, keep, new):
    total = 300
    s = Setup(qm, [new], [total], 16, 4, 1, 64)
    clean, _ = _run(qm, s, window=window, keep_first=keep)
    gone = torch.arange(keep, total - new - window + 1)
    rows = s.table[0, gone // 16].long().to(DEV), (gone % 16).to(DEV)
    s.k[rows], s.v[rows] = float("nan"), float("inf")
    out, flags = _run(qm, s, window=window, keep_first=keep)
    assert flags == 0 and torch.equal(out, clean)


def test_rows_that_see_nothing(qm):
    """Lengths of zero, or below the new tokens': zeros, with and without sinks."""
    s = Setup(qm, [3, 4, 1], [3, 4, 1], 16, 4, 2, 64)
    s.batch = qm.KvBatch(s.batch.q_start, torch.tensor([0, 2, 1], dtype=torch.int32, device=DEV),
                         s.batch.page_table)
    for sinks in (None, torch.ones(4, device=DEV)):
        out, flags = _run(qm, s, sinks=sinks)
        assert flags == 1                           # positions below zero
        assert not out[:5].any() and not out[:3].isnan().any()
        assert out[5:8].abs().amax((1, 2)).bool().all()


@pytest.mark.parametrize("new,total", [([1], [80]), ([20], [80]), ([200], [300])])
@pytest.mark.parametrize("page", [5, 16])
def test_bad_pages_are_left_out(qm, new, total, page):
    s = Setup(qm, new, total, page, 4, 2, 64)
    table = s.table.clone()
    table[0, 1], table[0, 3] = 1 << 30, -5
    s.batch = qm.KvBatch(s.batch.q_start, s.batch.seq_len, table.to(DEV))
    out, flags = _run(qm, s)
    assert flags == 1
    key = torch.arange(total[0])
    s.check(out, ok=[(key // page != 1) & (key // page != 3)])


def test_longer_than_the_table(qm):
    s = Setup(qm, [2], [40], 8, 4, 2, 64)
    s.batch = qm.KvBatch(s.batch.q_start, s.batch.seq_len, s.table[:, :3].contiguous().to(DEV))
    out, flags = _run(qm, s)
    assert flags == 1
    s.check(out, ok=[torch.arange(40) < 24])


def test_malformed_batches_stay_inside(qm):
    """Row numbers that fall, go below zero or past T: what comes out is unspecified, but nothing
    outside the rows is touched."""
    s = Setup(qm, [5, 5, 5], [20, 30, 40], 8, 4, 2, 64, pad=0)
    for start in ([0, 12, 4, 15], [-7, 5, 10, 15], [0, 5, 10, 99], [0, 5, 99, 3]):
        s.batch = qm.KvBatch(torch.tensor(start, dtype=torch.int32, device=DEV), s.batch.seq_len,
                             s.batch.page_table)
        big = torch.full((s.T + 8, 4, 64), 3.0, dtype=BF, device=DEV)
        qm.attend(s.q, s.kv, s.batch, out=big[4:4 + s.T])
        assert (big[:4] == 3).all() and (big[4 + s.T:] == 3).all()


@pytest.mark.parametrize("new,total", [([1, 1], [90, 20]), ([150], [190])])
def test_strided_queries_and_outputs(qm, new, total):
    s = Setup(qm, new, total, 16, 4, 2, 64)
    plain, _ = _run(qm, s)
    row = torch.zeros(s.q.shape[0], 8, 72, dtype=BF, device=DEV)
    row[:, 1:5, 8:] = s.q
    out = torch.full((4, s.q.shape[0], 64), 3.0, dtype=BF, device=DEV)    # heads first
    qm.attend(row[:, 1:5, 8:], s.kv, s.batch, out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), plain)


def test_far_pages(qm):
    """Keys and values past 2^32 elements of their planes."""
    D, page = 64, 64
    n_pages = (1 << 32) // (page * D) + 4
    k, v = (torch.zeros(n_pages, page, 1, D, dtype=E4, device=DEV) for _ in range(2))
    s = Setup(qm, [1, 70], [100, 130], page, 2, 1, D, BF, E4, spare=0)
    far = (n_pages - s.k.shape[0] + s.table).to(torch.int32)
    k[n_pages - s.k.shape[0]:], v[n_pages - s.k.shape[0]:] = s.k, s.v
    near, _ = _run(qm, s)
    s.kv = qm.KvCache(k, v, s.kv.k_scale, s.kv.v_scale)
    s.batch = qm.KvBatch(s.batch.q_start, s.batch.seq_len, far.to(DEV), 70, 130)
    out, _ = _run(qm, s)
    assert torch.equal(out, near)


def test_many_sequences(qm):
    """More sequences than the search probes at once; a shared page table row of shared pages."""
    g = torch.Generator().manual_seed(2)
    new = torch.randint(0, 3, (300,), generator=g).tolist()
    total = [n + int(torch.randint(1, 40, (), generator=g)) for n in new]
    s = Setup(qm, new, total, 8, 4, 2, 32)
    out, flags = _run(qm, s)
    assert flags == 0
    s.check(out)


def test_mixed_hints_do_not_change_what_is_seen(qm):
    """Wrong hints pick another launch, never another result than the tolerance allows."""
    s = Setup(qm, [1, 150, 1], [500, 150, 90], 16, 8, 2, 64)
    for max_q, max_len in ((0, 0), (1, 1), (150, 500), (1 << 20, 1 << 20), (1, 500)):
        s.batch = qm.KvBatch(s.batch.q_start, s.batch.seq_len, s.batch.page_table, max_q, max_len)
        out, _ = _run(qm, s)
        s.check(out)
