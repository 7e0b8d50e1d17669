"""Splits of some sequences beside others: where their sums meet, against the 64-bit form."""
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


class Shared:
    """Sequences that all read the same pages, through one row of a page table."""

    def __init__(self, qm, new, total, Hkv, G, D, dtype=BF, cache=None, page=16, hints=True):
        g = torch.Generator().manual_seed(len(new))
        n = -(-max(total) // page)
        planes = [torch.randn(n, page, Hkv, D, generator=g).to(cache or dtype) for _ in range(2)]
        scales = [0.5 + torch.rand(Hkv, generator=g) for _ in range(2)] if cache == E4 else [None] * 2
        order = torch.randperm(n, generator=g).to(torch.int32)
        self.rows = [p.float()[order.long()].reshape(n * page, Hkv, D).double() *
                     (1 if s is None else s.double()[:, None]) for p, s in zip(planes, scales)]
        self.kv = qm.KvCache(*(p.to(DEV) for p in planes),
                             *(None if s is None else s.to(DEV) for s in scales))
        self.start = [0]
        for i in new:
            self.start.append(self.start[-1] + i)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.batch = qm.KvBatch(torch.tensor(self.start, **i32), torch.tensor(total, **i32),
                                order.to(DEV)[None].expand(len(new), n),
                                max(new) if hints else 0, max(total) if hints else 0)
        self.new, self.total, self.D = new, total, D
        self.q = torch.randn(self.start[-1] + 2, Hkv * G, D, generator=g).to(dtype)

    def check(self, out, window=0, keep=0, sinks=None):
        for b, (n, t) in enumerate(zip(self.new, self.total)):
            pick = sorted({0, 1, n // 2, n - 1} & set(range(n)))
            if not pick:
                continue
            at = torch.tensor([self.start[b] + i for i in pick])
            want, tol = ref.attend(self.q[at], self.rows[0][:t], self.rows[1][:t],
                                   torch.tensor([t - n + i for i in pick]), self.D ** -0.5,
                                   window=window, keep=keep, sinks=sinks)
            ref.near(out[at], want, tol, f"sequence {b}: {n} of {t}")


def run(qm, s, **kw):
    """In scratch memory of just the size that is asked for: nothing behind it is touched, and nothing
    that stood in it before reaches a row."""
    need = qm.attend_scratch_bytes(s.kv, s.batch, *s.q.shape[:2], kw.get("window", 0),
                                   kw.get("keep_first", 0))
    memory = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)     # NaN as floats
    out = torch.full_like(s.q, 3.0).to(DEV)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    qm.attend(s.q.to(DEV), s.kv, s.batch, out=out, scratch=memory[:need], err_flags=flags, **kw)
    assert flags.item() == any(t < n for n, t in zip(s.new, s.total))    # positions below zero
    assert (memory[need:] == 0xFF).all() and (out[s.start[-1]:] == 3).all()
    return out, need


# one split of the chunks' tiles and many of the tokens; splits of both; of the chunks alone
@pytest.mark.parametrize("hints", [True, False])
@pytest.mark.parametrize("new,total,Hkv,G,D", [([8200, 1, 3], [8300, 16384, 9000], 1, 8, 64),
                                               ([1, 0, 8200], [16384, 70, 8200], 1, 8, 32),
                                               ([1, 40, 4, 33, 0, 5], [9000, 9001, 3, 33, 8, 8192], 2, 8, 64),
                                               ([40, 1, 2], [9000, 6000, 33], 3, 5, 128),
                                               ([300, 1, 200], [5000, 5001, 4000], 2, 8, 256),
                                               ([40] + [1] * 40, [9000] + [50 * i + 1 for i in range(40)],
                                                12, 2, 32)])
def test_tokens_beside_chunks(qm, new, total, Hkv, G, D, hints):
    s = Shared(qm, new, total, Hkv, G, D, hints=hints)
    sinks = torch.linspace(-2, 3, Hkv * G, device=DEV)
    out, need = run(qm, s, sinks=sinks)
    assert need > 0
    s.check(out, sinks=sinks)
    assert torch.equal(run(qm, s, sinks=sinks)[0], out)


@pytest.mark.parametrize("where", [0, 5000, 8990])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_odd_values_beside_chunks(qm, where, bad):
    """A value that some rows do not see, in splits of both kinds: the others are as they were."""
    s = Shared(qm, [40, 1, 2], [9000, 8000, 4000], 1, 8, 64)
    clean, _ = run(qm, s)
    page = s.batch.page_table[0, where // 16].item()
    s.kv.v[page, where % 16, 0, 7] = bad
    out, _ = run(qm, s)
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(s.new, s.total)])
    sees = pos >= where
    other = [d for d in range(64) if d != 7]
    assert torch.equal(out[:43][~sees], clean[:43][~sees])
    assert torch.equal(out[:43][..., other], clean[:43][..., other])
    hit = out[:43][sees][..., 7].float()
    assert (hit.isnan() if bad != bad else hit == bad).all()


def test_malformed_batches_stay_inside(qm):
    """Row numbers that fall or go past T, in a batch whose splits meet."""
    s = Shared(qm, [40, 1, 33, 2], [9000, 8000, 4000, 2000], 2, 8, 64)
    T = s.start[-1]
    for start in ([0, 40, 20, 74, 76], [0, 40, 41, 99, 3], [-5, 40, 41, 70, 1 << 30], [7, 7, 50, 50, 60]):
        s.batch = qm.KvBatch(torch.tensor(start, dtype=torch.int32, device=DEV), s.batch.seq_len,
                             s.batch.page_table, 40, 9000)
        need = qm.attend_scratch_bytes(s.kv, s.batch, T, 16)
        memory = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
        big = torch.full((T + 8, 16, 64), 3.0, dtype=BF, device=DEV)
        qm.attend(s.q[:T].to(DEV), s.kv, s.batch, out=big[4:4 + T], scratch=memory[:need])
        assert (big[:4] == 3).all() and (big[4 + T:] == 3).all() and (memory[need:] == 0xFF).all()


@pytest.mark.parametrize("new,total,Hkv,G,D", [([1, 1, 1], [3000, 1, 700], 1, 33, 64),
                                               ([40, 1, 0, 2], [900, 20000, 5, 77], 2, 64, 128),
                                               ([1] * 70 + [9], [31 * i + 1 for i in range(71)], 1, 48, 32)])
def test_groups_of_more_than_few_rows(qm, new, total, Hkv, G, D):
    """Tokens and chunks of more query heads a KV head than the kernel for few rows takes."""
    s = Shared(qm, new, total, Hkv, G, D)
    s.check(run(qm, s)[0])
