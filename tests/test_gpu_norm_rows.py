"""Row lengths and row counts of the norms that need more care than a small shape shows."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
import quantized_routed_expert_gemv_amd as qm  # noqa: E402
import test_gpu_norm as against_oracle  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


# rows of 12289 to 16384 values, which have a variant of their own, and the borders next to it
@pytest.mark.parametrize("T,H", [(3, 12288), (2, 12320), (3, 14336), (2, 16384), (1, 16416)])
@pytest.mark.parametrize("rt", [BF, F32])
@pytest.mark.parametrize("exit", [False, True])
def test_wide_rows(T, H, rt, exit):
    if exit:
        against_oracle.test_combine_norm(T, H, 4, rt, F32, 1, 2, 1)
        against_oracle.test_combine_norm(T, H, 3, rt, BF, 0, 1, 1)
    else:
        against_oracle.test_add_norm(T, H, rt, BF, F32)
        against_oracle.test_add_norm(T, H, rt, None, BF)


def signs(n, every, dt=BF):
    """Ones, every `every`-th of them negative: each partial sum of their squares is a whole
    number, so the mean is 1 but for the last sums' roundings."""
    v = torch.ones(n, dtype=dt, device="cuda")
    v[::every] = -1
    return v


def test_long_sums_keep_their_digits():
    """2^30 squares of 25: a thread's share, 2^20 of them, passes 2^24, where fp32 adds of 25
    lose a digit each. The mean is 25, so x is the row's signs exactly."""
    H = 1 << 30
    r, w = signs(H, 3).view(1, H), signs(H, 5)
    x, out = qm.add_norm(r, w, delta=r, scale=4.0)
    assert torch.equal(out, 5 * r)
    assert torch.equal(x.view(-1), r.view(-1) * w)
    y, one = 5 * signs(H, 3, F32).view(1, H), torch.ones(1, 1, device="cuda")
    inv = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, x = qm.combine_norm(y, inv, one, torch.zeros_like(r), post_weight=5 * w, next_weight=w)
    assert torch.equal(out.view(-1), 5 * r.view(-1) * w)
    assert torch.equal(x, r)


@pytest.mark.parametrize("exit", [False, True])
def test_the_longest_row(exit):
    """H = 2^31 - 32: the column behind a thread's last one does not fit 31 bits."""
    H = (1 << 31) - 32
    w, r = signs(H, 5), signs(H, 3).view(1, H)
    if not exit:
        x, out = qm.add_norm(r, w, delta=r, scale=2.0)
        assert torch.equal(out, 3 * r)          # 1 + 2 * 1: the same row, three times as far
        del out
    else:
        one = torch.ones(1, 1, device="cuda")
        y = signs(H, 7, F32).view(1, H)
        inv = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = signs(H, 7) * w + r.view(-1)     # y has a mean square of 1, too
        out, x = qm.combine_norm(y, inv, one, r, eps=0.0, post_weight=w, next_weight=w)
        del y, one
        assert torch.equal(out.view(-1), want)
        # 0 or +-2: x = s / rms(s) w, rms^2 = 4 times the share of columns that are not zero
        hit = want != 0
        scale = (4 * hit.sum().double() / H).rsqrt().float()
        del hit
        want = (want.float() * scale * w).view(1, H)
        # 2^-8 for the rounding to bf16; each thread's sum of whole numbers is exact below 2^24,
        # the 1024 threads' has 21 adds of half a step
        assert bool(((x.float() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs()).all())
        return
    assert torch.equal(x.view(-1), r.view(-1) * w)


# more rows than one launch may have threads for, 2^32: 64 threads a row up to H = 1024, 1024
# from H = 8224 on
MANY = [((1 << 26) + 3, 32), ((1 << 22) + 3, 8224)]


def rows_like(t, first, last):
    """Row i of t equals first[i % len(first)], and its last rows equal `last`."""
    n, m = len(t) - len(last), len(first)
    assert n % m == 0 and torch.equal(t[n:], last)
    step = max(m, (1 << 28) // t.shape[1] // m * m)
    for i in range(0, n, step):
        part = t[i:min(i + step, n)].view(-1, *first.shape)
        assert torch.equal(part, first.expand_as(part)), f"rows {i} on"


def repeated(first, last, T):
    t = torch.empty(T, first.shape[1], dtype=first.dtype, device="cuda")
    n = T - len(last)
    t[:n].view(-1, *first.shape).copy_(first.expand(n // len(first), *first.shape))
    t[n:] = last
    return t


@pytest.mark.parametrize("T,H", MANY)
def test_more_rows_than_a_launch(T, H):
    g = torch.Generator("cuda").manual_seed(H)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    first, last, w = rand(64, H).to(BF), rand(3, H).to(BF), rand(H).to(BF)
    r = repeated(first, last, T)
    x, out = qm.add_norm(r, w, delta=r, scale=0.5, resid_out=r)
    want = [qm.add_norm(v, w, delta=v, scale=0.5) for v in (first, last)]
    rows_like(x, want[0][0], want[1][0])
    rows_like(out, want[0][1], want[1][1])


def test_more_rows_than_a_launch_at_the_exit():
    T, H = (1 << 26) + 3, 32
    g = torch.Generator("cuda").manual_seed(7)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    first, last, w = rand(64, H), rand(3, H), rand(H)
    y, r = repeated(first, last, T), repeated(first.to(BF), last.to(BF), T)
    tw = torch.full((T, 1), 0.5, device="cuda")
    inv = torch.arange(T, dtype=torch.int32, device="cuda")
    out, x = qm.combine_norm(y, inv, tw, r, post_weight=w, gate=r.float(), next_weight=w)
    want = [qm.combine_norm(v, inv[:len(v)], tw[:len(v)], v.to(BF), post_weight=w,
                            gate=v.to(BF).float(), next_weight=w) for v in (first, last)]
    rows_like(out, want[0][0], want[1][0])
    rows_like(x, want[0][1], want[1][1])
