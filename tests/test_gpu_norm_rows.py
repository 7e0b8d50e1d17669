"""Row lengths and row counts of the norms that need more care than a small shape shows."""
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
