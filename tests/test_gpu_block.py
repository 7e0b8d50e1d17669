"""The attention half of a block and the layer behind it, run as they are used: entry norm, QKV
product, append, attention, output product into the residual stream, norm, experts."""
import pytest

torch = pytest.importorskip("torch")
import attention_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
H, HQ, HKV, D, I, E, K, PAGE = 512, 8, 2, 64, 352, 8, 2, 16
HEADS = HQ + 2 * HKV


class Weights:
    def __init__(self, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.norm1, self.norm2 = 1 + 0.2 * rand(H), 1 + 0.2 * rand(H)
        self.wqkv, self.bqkv = (rand(HEADS * D, H) / H ** 0.5).to(BF), rand(HEADS * D)
        self.wo, self.sinks = (rand(H, HQ * D) / (HQ * D) ** 0.5).to(BF), rand(HQ)
        self.wr = (rand(E, H) / H ** 0.5).to(BF)
        planes = {}
        for n, r, c in (("gate", I, H), ("up", I, H), ("down", H, I)):
            planes[n + "_q"], planes[n + "_s"] = qm.mx_quantize(rand(E, r, c) / c ** 0.5)
        self.pool = qm.Pool.from_canonical("mxfp4", H, I, planes)
        self.slots = torch.arange(E, dtype=torch.int32, device="cuda")
        self.rope = qm.Rope.make(D, base=1e4, scaling="yarn", factor=4.0, original=64)


class Step:
    """Sequences with `new` tokens each behind `past` cached ones; room for 8 more tokens."""

    def __init__(self, weights, new, past, cache=BF, window=0, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.w, self.new, self.past, self.window = weights, new, past, window
        self.T, n_seq = sum(new), len(new)
        most = max(n + p for n, p in zip(new, past)) + 8
        need = -(-most // PAGE)
        table = torch.randperm(n_seq * need, generator=g, device="cuda").to(torch.int32)
        scale = [0.5 + torch.rand(HKV, generator=g, device="cuda") for _ in range(2)] \
            if cache == E4 else [None, None]
        self.cache = qm.KvCache.empty(n_seq * need, PAGE, HKV, D, cache, *scale)
        for t in (self.cache.k, self.cache.v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(cache))
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.start, self.table = start, table.view(n_seq, need)
        self.seq_len = torch.tensor([n + p for n, p in zip(new, past)], **i32)
        self.batch = qm.KvBatch(torch.tensor(start, **i32), self.seq_len, self.table, max(new), most)
        self.resid = torch.randn(self.T, H, generator=g, device="cuda").to(BF)

    def __call__(self, stream=None):
        """-> every stage's result."""
        w, st = self.w, dict(stream=stream)
        x, _ = qm.add_norm(self.resid, w.norm1, **st)
        row = qm.linear(x, w.wqkv, bias=w.bqkv, **st)
        q, k, v = row.view(self.T, HEADS, D).split([HQ, HKV, HKV], 1)
        turned = qm.kv_append(self.cache, self.batch, k, v, w.rope, q=q, **st)
        a = qm.attend(turned, self.cache, self.batch, window=self.window,
                      keep_first=4 if self.window else 0, sinks=w.sinks, **st)
        r = qm.linear(a.view(self.T, HQ * D), w.wo, resid=self.resid, **st)
        x2, _ = qm.add_norm(r, w.norm2, **st)
        y, _ = qm.layer(w.pool, w.slots, w.wr, None, x2, K, **st)
        return dict(x=x, row=row, q=turned, a=a, r=r, x2=x2, y=y)

    def planes(self):
        return [self.cache.k.clone().view(torch.uint8), self.cache.v.clone().view(torch.uint8)]


@pytest.fixture(scope="module")
def weights():
    return Weights()


SHAPES = {"token": ([1], [40]), "tokens": ([1, 1, 1, 1], [0, 17, 300, 1000]),
          "prompt": ([150], [0]), "mixed": ([1, 60, 1, 9], [90, 16, 700, 0])}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cache,window", [(BF, 0), (E4, 0), (BF, 33)])
def test_stages(weights, shape, cache, window):
    """Each stage against the 64-bit form of what the stage before it left."""
    s, w = Step(weights, *SHAPES[shape], cache, window), weights
    before = s.planes()
    m = s()
    torch.cuda.synchronize()
    want, tol = ref.linear(m["x"], w.wqkv, w.bqkv, "none", None, BF)
    ref.near(m["row"], want, tol, "qkv")
    q, k, v = m["row"].cpu().view(s.T, HEADS, D).split([HQ, HKV, HKV], 1)
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(s.new, s.past)])
    freq, f = w.rope.freq.cpu(), w.rope.scale
    want, tol = ref.rope(q, pos, freq, "half", f)
    ref.near(m["q"], want, tol + ref.rounded(want.abs() + tol, BF), "queries")
    turned, tol_k = ref.rope(k, pos, freq, "half", f)
    seq = torch.repeat_interleave(torch.arange(len(s.new)), torch.tensor(s.new))
    place = s.table.cpu()[seq, pos // PAGE].long(), pos % PAGE
    planes = []
    for plane, scale, rows, t in ((s.cache.k, s.cache.k_scale, turned, tol_k),
                                  (s.cache.v, s.cache.v_scale, v.double(), torch.zeros(v.shape))):
        one = torch.ones(HKV, 1, dtype=torch.float64) if scale is None else \
            scale.double().cpu()[:, None]
        code = rows / one
        # of an 8-bit cache the reciprocal of the scale and the product with it are rounded to fp32
        t = t / one + (4 * ref.F32 * code.abs() if scale is not None else 0)
        ref.near(plane.float()[tuple(i.to("cuda") for i in place)], code,
                 t + ref.rounded(code.abs() + t, cache), "cache")
        planes.append(plane.float().cpu().double() * one)
    keep = torch.ones(s.cache.n_pages, PAGE, dtype=torch.bool)
    keep[place] = False
    for a, b in zip(before, s.planes()):   # nothing else was written
        same = (a == b).flatten(2).all(-1).cpu()
        assert same[keep].all()
    for b, n in enumerate(s.new):
        t = torch.arange(s.past[b] + n)
        at = s.table.cpu()[b, t // PAGE].long(), t % PAGE
        rows = slice(s.start[b], s.start[b + 1])
        want, tol = ref.attend(m["q"][rows], planes[0][at], planes[1][at], t[-n:], D ** -0.5,
                               window=window, keep=4 if window else 0, sinks=w.sinks)
        ref.near(m["a"][rows], want, tol, f"attention of sequence {b}")
    want, tol = ref.linear(m["a"].view(s.T, -1), w.wo, None, "none", s.resid, BF)
    ref.near(m["r"], want, tol, "output product")
    again, _ = qm.layer(w.pool, w.slots, w.wr, None, qm.add_norm(m["r"], w.norm2)[0], K)
    assert torch.equal(again, m["y"])


def _same(s, got, planes, stream=None):
    """The eager block gives the same bits, in its results and in the cache."""
    want = s(stream)
    torch.cuda.synchronize()
    for n in got:
        assert torch.equal(got[n], want[n]), n
    for a, b in zip(planes, s.planes()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cache", [BF, E4])
def test_in_a_graph(weights, shape, cache):
    """Captured once; each replay is the next step: lengths and inputs move between replays, with
    eager work and synchronisation, and every replay equals the eager run."""
    s = Step(weights, *SHAPES[shape], cache)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = s()
    for i in range(5):
        s.resid.copy_((torch.randn(s.T, H, device="cuda") * (i + 1)).to(BF))
        s.seq_len.add_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _same(s, {n: t.clone() for n, t in out.items()}, s.planes())


def test_two_graphs_take_turns(weights):
    """Two captured steps, replayed in turn and at once on two streams, share nothing."""
    steps = [Step(weights, *SHAPES["tokens"], seed=1), Step(weights, *SHAPES["mixed"], seed=2)]
    streams = [torch.cuda.Stream() for _ in steps]
    graphs, outs = [], []
    for s, st in zip(steps, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            s()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(s())
        graphs.append(g)
    for _ in range(3):
        for s in steps:
            s.seq_len.add_(1)
            s.resid.mul_(-1)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, out in zip(steps, outs):
            _same(s, {n: t.clone() for n, t in out.items()}, s.planes())


def test_on_a_named_stream(weights):
    """On a stream that the calls name, twice and at once with another on the current stream."""
    a, b = Step(weights, *SHAPES["mixed"], seed=3), Step(weights, *SHAPES["tokens"], E4, seed=4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [a(side), b()]
    torch.cuda.synchronize()
    planes = [s.planes() for s in (a, b)]
    _same(a, got[0], planes[0])
    _same(b, got[1], planes[1], side)


def test_chunks_and_tokens_agree(weights):
    """A prompt in one step, and the same in chunks: keys and values come out bit by bit, whatever
    the launch; attention within its tolerance (tokens of a chunk see the same cache)."""
    whole = Step(weights, [48], [0], seed=5)
    m = whole()
    want = [p[whole.table[0].long()].clone() for p in (whole.cache.k, whole.cache.v)]
    x = m["row"].view(48, HEADS, D)
    out = []
    i32 = dict(dtype=torch.int32, device="cuda")
    for lo, hi in ((0, 5), (5, 6), (6, 48)):
        batch = qm.KvBatch(torch.tensor([0, hi - lo], **i32), torch.tensor([hi], **i32),
                           whole.table, hi - lo, hi)
        q, k, v = x[lo:hi].split([HQ, HKV, HKV], 1)
        cache = whole.cache if lo else qm.KvCache.empty(whole.cache.n_pages, PAGE, HKV, D)
        if not lo:
            cache.k.fill_(float("nan"))
            cache.v.fill_(float("nan"))
            whole.cache = cache
        turned = qm.kv_append(cache, batch, k, v, weights.rope, q=q)
        assert torch.equal(turned, m["q"][lo:hi])
        out.append(qm.attend(turned, cache, batch, sinks=weights.sinks))
    got = [p[whole.table[0].long()] for p in (whole.cache.k, whole.cache.v)]
    for a, b in zip(got, want):
        a, b = a.reshape(-1, HKV, D)[:48], b.reshape(-1, HKV, D)[:48]
        assert torch.equal(a, b)
    rows = [p.reshape(-1, HKV, D)[:48] for p in want]
    y, tol = ref.attend(m["q"], *rows, torch.arange(48), D ** -0.5, sinks=weights.sinks)
    ref.near(torch.cat(out), y, tol, "in chunks")
    ref.near(m["a"], y, tol, "at once")
