"""Batches of more sequences than one launch takes, and rows on either side of where the launch
changes."""
import pytest

torch = pytest.importorskip("torch")
import attention_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_gemv_amd as qm
    return qm


def _shared(qm, new, total, Hkv, D, page, capacity, hints, seed=0):
    """Sequences that all read the same pages, through one row of a page table."""
    g = torch.Generator().manual_seed(seed)
    n = capacity // page
    k, v = (torch.randn(n, page, Hkv, D, generator=g).to(BF) for _ in range(2))
    order = torch.randperm(n, generator=g).to(torch.int32)
    table = order.to(DEV)[None].expand(len(new), n)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32)
    batch = qm.KvBatch(start.to(DEV), total.to(torch.int32).to(DEV), table,
                       int(new.max()) if hints else 0, int(total.max()) if hints else 0)
    rows = [t[order.long()].reshape(capacity, Hkv, D) for t in (k, v)]
    return qm.KvCache(k.to(DEV), v.to(DEV)), batch, rows


@pytest.mark.parametrize("chunks", [False, True])
def test_many_sequences(qm, chunks):
    """70000 sequences; with chunks some of them have more than a row tile of new tokens. Each row
    sees one of few lengths of the shared keys: the rows of one length are checked together."""
    B, Hkv, G, D, capacity = 70000, 1, 2, 16, 64
    b = torch.arange(B)
    new, total = torch.ones(B, dtype=torch.int64), 1 + b * 7 % capacity
    if chunks:
        new[1000::17000], total[1000::17000] = 50, 61
    cache, batch, (k, v) = _shared(qm, new, total, Hkv, D, 16, capacity, False)
    T = int(new.sum())
    q = torch.randn(T, G, D, generator=torch.Generator().manual_seed(1)).to(BF)
    got = qm.attend(q.to(DEV), cache, batch)
    seq = torch.repeat_interleave(b, new)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    pos = total[seq] - new[seq] + torch.arange(T) - start[seq]
    for p in range(capacity):
        rows = (pos == p).nonzero().flatten()
        rows = torch.cat([rows[:6], rows[-6:]])
        if len(rows):
            want, tol = ref.attend(q[rows], k, v, pos[rows], D ** -0.5)
            ref.near(got.cpu()[rows], want, tol, f"at {p}")
    # and all of them, against a sum over the keys in fp64
    s = torch.einsum("tgd,kd->tgk", q.double(), k[:, 0].double()) * D ** -0.5
    w = s.masked_fill(torch.arange(capacity) > pos[:, None, None], -torch.inf).softmax(-1)
    want = w @ v[:, 0].double()
    # as in the reference, with sums of D products' magnitudes below 64: a score's error is below
    # 18 2^-24 D^-1/2 64 + 2^-17 < 2^-15
    tol = (2.0 ** -8 + 2 * 2.0 ** -15 + 256 * ref.F32) * (w @ v[:, 0].double().abs())
    ref.near(got, want, tol + ref.rounded(want, BF), "all")


@pytest.mark.parametrize("hints", [False, True])
def test_many_split_sequences(qm, hints):
    """Few sequences with long contexts, tokens and chunks together: split ones meet again."""
    new, total = torch.tensor([1, 40, 1, 33, 2]), torch.tensor([9000, 9001, 3, 33, 8192])
    Hkv, G, D = 2, 4, 64
    cache, batch, (k, v) = _shared(qm, new, total, Hkv, D, 16, 9008, hints)
    q = torch.randn(int(new.sum()), Hkv * G, D, generator=torch.Generator().manual_seed(1)).to(BF)
    got = qm.attend(q.to(DEV), cache, batch, window=0)
    at = 0
    for n, t in zip(new.tolist(), total.tolist()):
        pick = sorted({0, n // 2, n - 1})
        rows = torch.tensor([at + i for i in pick])
        want, tol = ref.attend(q[rows], k[:t], v[:t], torch.tensor([t - n + i for i in pick]), D ** -0.5)
        ref.near(got.cpu()[rows], want, tol, f"{n} of {t}")
        at += n


@pytest.mark.parametrize("B", [2, 63, 64, 65, 129])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_of_many_sequences(qm, B, causal):
    """Chunks of one to three tiles and single tokens, sequences without new tokens among them, many of
    the same length, on either side of the number of sequences that a wave orders by length."""
    b = torch.arange(B)
    new = torch.tensor([40, 1, 0, 70, 33, 1, 9])[b % 7]
    total = torch.tensor([80, 71, 200, 200, 33])[b % 5].maximum(new)
    Hkv, G, D = 2, 4, 32
    cache, batch, (k, v) = _shared(qm, new, total, Hkv, D, 16, 208, False, seed=B)
    T = int(new.sum())
    q = torch.randn(T + 3, Hkv * G, D, generator=torch.Generator().manual_seed(1)).to(BF)
    out = torch.full_like(q, 3.0).to(DEV)
    qm.attend(q.to(DEV), cache, batch, causal=causal, out=out)
    assert (out[T:] == 3).all()
    out, at = out.cpu(), 0
    for n, t in zip(new.tolist(), total.tolist()):
        pick = sorted({0, 16, 31, 32, n - 1} & set(range(n)))
        if pick:
            rows = torch.tensor([at + i for i in pick])
            want, tol = ref.attend(q[rows], k[:t], v[:t], torch.tensor([t - n + i for i in pick]),
                                   D ** -0.5, causal=causal)
            ref.near(out[rows], want, tol, f"{n} of {t}")
        at += n


@pytest.mark.parametrize("T", [255, 257, 2047, 2048, 2049, 2055])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_where_the_launch_changes(qm, T, dtype):
    """Rotation and append of as many tokens as the small launch takes, and of one more; many heads,
    so that a token's pairs are over several workgroups."""
    Hkv, G, D, page = 40, 2, 64, 16
    g = torch.Generator().manual_seed(T)
    row = torch.randn(T, Hkv * (G + 2), D, generator=g).to(dtype).to(DEV)
    q, k, v = row.split([Hkv * G, Hkv, Hkv], 1)
    plan = qm.Rope.make(D)
    pos = torch.arange(T) + 5
    want, tol = ref.rope(row[:, :Hkv * (G + 1)], pos, plan.freq, "half", 1.0)
    tol = tol + ref.rounded(want, dtype)
    ref.near(qm.rope(row, (pos.to(torch.int32)).to(DEV), plan)[:, :Hkv * (G + 1)], want, tol, "rope")
    n = -(-(T + 5) // page)
    cache = qm.KvCache(*(torch.full((n, page, Hkv, D), 7.0, device=DEV, dtype=BF) for _ in range(2)))
    batch = qm.KvBatch(torch.tensor([0, T], dtype=torch.int32, device=DEV),
                       torch.tensor([T + 5], dtype=torch.int32, device=DEV),
                       torch.arange(n, dtype=torch.int32, device=DEV)[None])
    got = qm.kv_append(cache, batch, k, v, plan, q=q)
    ref.near(got, want[:, :Hkv * G], tol[:, :Hkv * G], "queries")
    keys, values = (t.reshape(n * page, Hkv, D) for t in (cache.k, cache.v))
    wk = want[:, Hkv * G:]
    _, t0 = ref.rope(k, pos, plan.freq, "half", 1.0)
    ref.near(keys[5:5 + T], wk, t0 + ref.rounded(wk.abs() + t0, BF), "keys")
    assert torch.equal(values[5:5 + T], v.to(BF))
    for t in (keys, values):
        assert (t[:5] == 7).all() and (t[5 + T:] == 7).all()
