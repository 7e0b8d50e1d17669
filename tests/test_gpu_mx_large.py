"""Microscaled calls at sizes past one launch or past 32 bits of an index."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def repeated(first, last, rows):
    t = torch.empty(rows, first.shape[1], dtype=first.dtype, device="cuda")
    n = rows - len(last)
    t[:n].view(-1, *first.shape).copy_(first.expand(n // len(first), *first.shape))
    t[n:] = last
    return t


def rows_like(t, first, last):
    """Row i of t equals first[i % len(first)], and its last rows equal `last`."""
    n, m = len(t) - len(last), len(first)
    assert n % m == 0 and torch.equal(t[n:], last)
    step = max(m, (1 << 28) // t.shape[1] // m * m)
    for i in range(0, n, step):
        part = t[i:min(i + step, n)].view(-1, *first.shape)
        assert torch.equal(part, first.expand_as(part)), f"rows {i} on"


# a launch has fewer than 2^32 threads, of 8 values (MXFP4 codes, fp32 values) or of 16, and
# takes 2^34 values
@pytest.mark.parametrize("fmt,log_values,dt", [("mxfp4", 35, F32), ("mxfp6", 34, BF)])
def test_more_values_than_a_launch(fmt, log_values, dt):
    K = 1 << 15
    rows = (1 << (log_values - 15)) + 3
    g = torch.Generator("cuda").manual_seed(1)
    first, last = (torch.randn(n, K, generator=g, device="cuda").to(BF) for n in (64, 3))
    x = repeated(first, last, rows)
    q, s = qm.mx_quantize(x, fmt)
    del x
    torch.cuda.empty_cache()
    f, l = qm.mx_quantize(first, fmt), qm.mx_quantize(last, fmt)
    rows_like(q, f[0], l[0])
    rows_like(s, f[1], l[1])
    v = qm.mx_dequantize(q, s, fmt, dt)
    rows_like(v, qm.mx_dequantize(*f, fmt, dt), qm.mx_dequantize(*l, fmt, dt))


def test_more_tiles_than_a_launch():
    """66 row tiles by 2^18 of 256 columns, of 256 threads each, pass 2^32 threads."""
    H, I, T = 1 << 26, 32, 64
    g = torch.Generator("cuda").manual_seed(2)
    rand = lambda a, b, *s: torch.randint(a, b, s, generator=g, dtype=torch.uint8, device="cuda")  # noqa: E731
    pool = qm.Pool.empty("mxfp4", 1, H, I)
    qm.pool_pack("mxfp4", 1, H, I, rand(0, 256, H, I // 2), rand(118, 124, H, 1),
                 pool.planes["down_q"], pool.planes["down_s"])
    sm = torch.zeros(T, dtype=torch.int32, device="cuda")
    ids = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    off = qm.bucket(ids, T)[1]
    hq, hs = rand(0, 256, T, I // 2), rand(123, 131, T, 1)
    y = qm.mx_expert_down(pool, sm, T, 1, off, hq, hs, "mxfp4", path=qm.PATH_GROUPED)
    # one block a row: its sum is exact, so both schedules give the same
    few = qm.mx_expert_down(pool, sm, T, 1, off, hq, hs, "mxfp4", path=qm.PATH_GEMV)
    assert bool(y[:, -32:].any(1).all()) and torch.equal(y, few)


def test_a_miss_of_many_rows():
    """An expert outside the pool whose rows hold 2^31 values and more in 16 columns."""
    T, H, I = (1 << 27) + 5, 32, 32
    pool = qm.Pool.empty("mxfp4", 1, H, I)
    sm = torch.full((1,), qm.SLOT_MISS, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    perm = torch.arange(T, dtype=torch.int32, device="cuda")
    q = torch.zeros(T, I // 2, dtype=torch.uint8, device="cuda")
    s = torch.full((T, 1), 127, dtype=torch.uint8, device="cuda")
    h = torch.full((T, I), 7, dtype=BF, device="cuda")
    qm.mx_expert_gate_up(pool, sm, q, s, "mxfp4", 1, off, perm, h=h, path=qm.PATH_GEMV)
    assert not h.any()
    del h, perm
    y = torch.full((T, H), 7, dtype=F32, device="cuda")
    qm.mx_expert_down(pool, sm, T, 1, off, q, s, "mxfp4", y=y, path=qm.PATH_GEMV)
    assert not y.any()
