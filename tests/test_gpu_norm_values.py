"""Values of the norms' inputs that need more care than ordinary ones."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
BITS = {BF: torch.int16, F32: torch.int32}


@pytest.mark.parametrize("rt", [BF, F32])
@pytest.mark.parametrize("H", [64, 2880, 20000])
@pytest.mark.parametrize("scale", [1.0, 0.0, float("inf"), float("nan")])
def test_without_delta_the_stream_stays(scale, H, rt):
    """No delta: s is resid, whatever the scale, bit by bit (a zero's sign too)."""
    r, w = torch.randn(3, H, device="cuda").to(rt), torch.ones(H, device="cuda")
    r[0, ::3] = -0.0
    r[1] = 0
    x, out = qm.add_norm(r, w, scale=scale, resid_out=torch.empty_like(r))
    assert torch.equal(out.view(BITS[rt]), r.view(BITS[rt]))
    want = r.float()
    want = want * torch.rsqrt(want.square().mean(1, keepdim=True) + 1e-6)
    # 2^-8 for bf16; the mean's roundings (H / 256 + 16 adds) and a few more in both sides
    tol = (2.0 ** -8 + 2 * (H / 256 + 24) * 2.0 ** -24) * want.abs()
    assert bool(((x.float() - want).abs() <= tol).all())
