"""Dense products at sizes on either side of each change of tile, with last tiles that are partly
filled and depths that end inside a step."""
import pytest

torch = pytest.importorskip("torch")
import attention_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32

# by the number of tiles: 256 of 16 x 16, 257; 256 of 16 x 32; 16 rows and wide; 32 x 32; 64 x 32;
# 64 x 64 up to 256, up to 400, more; 128 x 128; 768 of 128 x 256 and more
SIZES = [(16, 4096), (17, 2040), (16, 4097), (32, 4090), (16, 8192), (16, 8193), (1, 20003),
         (9, 30000), (33, 4000), (130, 1500), (250, 1024), (100, 4000), (64, 8190), (200, 3900),
         (1024, 1000), (333, 3000), (1280, 1270), (500, 4000), (1100, 4000), (1300, 4000),
         (129, 40001), (4097, 6000), (12300, 2050)]


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_gemv_amd as qm
    return qm


@pytest.mark.parametrize("K", [8, 72, 520])
@pytest.mark.parametrize("M,N", SIZES)
def test_whole_numbers_are_exact(qm, M, N, K):
    """Sums below 2^24: nothing may be off. Bias, relu and a residual in place, at places that no
    four values wide store fits; what lies beside the outputs stays."""
    g = torch.Generator().manual_seed(M + N + K)
    x = torch.randint(-4, 5, (M, K), generator=g).to(BF)
    w = torch.randint(-4, 5, (N, K), generator=g).to(BF)
    b = torch.randint(-9, 10, (N,), generator=g).float()
    r = torch.randint(-99, 100, (M, N + 5), generator=g).float()
    got = r.to(DEV)
    qm.linear(x.to(DEV), w.to(DEV), bias=b.to(DEV), act="relu", resid=got[:, 3:3 + N],
              out=got[:, 3:3 + N])
    r[:, 3:3 + N] += (x.float() @ w.float().T + b).clamp(min=0)
    assert torch.equal(got.cpu(), r)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,N", SIZES)
def test_values(qm, M, N, dtype):
    K = 200
    g = torch.Generator().manual_seed(M + N)
    x = torch.randn(M, K, generator=g).to(dtype)
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(dtype)
    b = torch.randn(N, generator=g).to(dtype)
    got = qm.linear(x.to(DEV), w.to(DEV), bias=b.to(DEV), act="silu")
    want, tol = ref.linear(x, w, b, "silu", None, dtype)
    ref.near(got, want, tol, "tiles")
