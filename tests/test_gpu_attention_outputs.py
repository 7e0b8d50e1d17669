"""Rotation, append and attention of rows that overlap or are expanded, against the 64-bit forms."""
import pytest

torch = pytest.importorskip("torch")
import attention_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
VIEWS = [((8, 37, 64), (100, 1, 1)), ((8, 1, 64), (1, 1, 1)), ((8, 4, 64), (1, 64, 1)),
         ((8, 4, 64), (0, 1, 1)), ((8, 4, 64), (0, 64, 1)), ((4, 8, 64), (64, 256, 1))]


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_gemv_amd as qm
    return qm


@pytest.mark.parametrize("shape,strides", VIEWS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_overlapping_rows_turn(qm, shape, strides, dtype):
    T, n, D = shape
    g = torch.Generator().manual_seed(0)
    x = torch.randn(1 << 12, generator=g).to(dtype).to(DEV).as_strided(shape, strides)
    pos = torch.arange(T) * 1000 + 3
    plan = qm.Rope.make(D)
    want, tol = ref.rope(x, pos, plan.freq, "half", 1.0)
    tol = tol + ref.rounded(want, dtype)
    got = qm.rope(x, pos.to(torch.int32).to(DEV), plan)
    ref.near(got, want, tol, "rope")
    kv = qm.KvCache(*(torch.zeros(2, 16, 1, D, dtype=BF, device=DEV) for _ in range(2)))
    i32 = dict(dtype=torch.int32, device=DEV)
    batch = qm.KvBatch(torch.tensor([0, T], **i32), torch.tensor([T], **i32),
                       torch.arange(2, **i32)[None])
    new = torch.zeros(T, 1, D, dtype=dtype, device=DEV)
    got = qm.kv_append(kv, batch, new, new, plan, pos.to(torch.int32).to(DEV), q=x)
    ref.near(got, want, tol, "queries")


@pytest.mark.parametrize("T", [1, 40])
def test_expanded_queries_attend(qm, T):
    """One query a token, for every head of a group."""
    Hkv, G, D, L = 1, 8, 64, 90
    g = torch.Generator().manual_seed(1)
    q = torch.randn(T, 1, D, generator=g).to(BF)
    k, v = (torch.randn(6, 16, Hkv, D, generator=g).to(BF) for _ in range(2))
    i32 = dict(dtype=torch.int32, device=DEV)
    batch = qm.KvBatch(torch.tensor([0, T], **i32), torch.tensor([L], **i32),
                       torch.arange(6, **i32)[None], T, L)
    got = qm.attend(q.to(DEV).expand(T, G, D), qm.KvCache(k.to(DEV), v.to(DEV)), batch)
    want, tol = ref.attend(q.expand(T, G, D), k.flatten(0, 1)[:L], v.flatten(0, 1)[:L],
                           torch.arange(L - T, L), D ** -0.5)
    ref.near(got, want, tol, "attention")
