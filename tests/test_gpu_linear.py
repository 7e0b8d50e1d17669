"""Dense products with bias, activation and residual, against the 64-bit form."""
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


def _randn(*shape, seed=0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


SIZES = [(1, 1, 8), (1, 16, 64), (3, 17, 72), (4, 320, 2880), (16, 100, 512), (17, 64, 64),
         (31, 33, 200), (64, 128, 256), (65, 130, 136), (128, 256, 128), (200, 300, 1000),
         (333, 257, 264), (513, 520, 96), (130, 1, 64), (1, 5000, 40)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bias,act,resid,out", [
    (None, "none", None, F32), (BF, "silu", None, BF), (F32, "none", F32, F32),
    (FP, "gelu", BF, BF), (None, "gelu_tanh", FP, FP), (F32, "relu", None, FP)])
def test_linear(qm, M, N, K, dtype, bias, act, resid, out):
    x, w = _randn(M, K, dtype=dtype), _randn(N, K, seed=1, dtype=dtype)
    w = (w.float() / K ** 0.5).to(dtype)
    b = None if bias is None else _randn(N, seed=2, dtype=bias)
    r = None if resid is None else _randn(M, N, seed=3, dtype=resid)
    got = qm.linear(x, w, bias=b, act=act, resid=r, out_dtype=out)
    assert got.dtype == out and got.shape == (M, N)
    want, tol = ref.linear(x, w, b, act, r, out)
    ref.near(got, want, tol, "linear")


@pytest.mark.parametrize("M,N,K", SIZES + [(1000, 700, 2880), (2048, 1024, 512)])
def test_whole_numbers_are_exact(qm, M, N, K):
    """Small whole numbers: every sum fits fp32, so nothing may be off at all."""
    g = torch.Generator().manual_seed(M + N + K)
    x = torch.randint(-4, 5, (M, K), generator=g).to(BF).to(DEV)
    w = torch.randint(-4, 5, (N, K), generator=g).to(BF).to(DEV)
    r = torch.randint(-99, 99, (M, N), generator=g).float().to(DEV)
    got = qm.linear(x, w, resid=r)
    assert torch.equal(got.cpu(), x.float().cpu() @ w.float().cpu().T + r.cpu())


@pytest.mark.parametrize("M,N,K", [(5, 40, 64), (100, 200, 96), (300, 520, 128)])
def test_strided_rows(qm, M, N, K):
    """Rows inside wider ones, outputs at odd places; what lies around stays. A residual in place."""
    X, W = _randn(M, K + 24, dtype=BF), _randn(N, K + 8, seed=1, dtype=BF)
    x, w = X[:, 16:16 + K], W[:, :K]
    for dtype in (F32, BF):
        wide = torch.full((M, N + 7), 5.0, device=DEV, dtype=dtype)
        got = qm.linear(x, w, out=wide[:, 3:3 + N])
        want, tol = ref.linear(x, w, None, "none", None, dtype)
        ref.near(got, want, tol)
        assert (wide[:, :3] == 5).all() and (wide[:, 3 + N:] == 5).all()
        r = _randn(M, N + 7, seed=4, dtype=dtype)
        want, tol = ref.linear(x, w, None, "relu", r[:, 1:1 + N], dtype)
        edge = r[:, [0] + list(range(N + 1, N + 7))].clone()
        qm.linear(x, w, act="relu", resid=r[:, 1:1 + N], out=r[:, 1:1 + N])
        ref.near(r[:, 1:1 + N], want, tol)
        assert torch.equal(r[:, [0] + list(range(N + 1, N + 7))], edge)
    same = qm.linear(x[:1].expand(M, K), w)          # one row over and over
    assert torch.equal(same, same[:1].expand(M, N))


@pytest.mark.parametrize("M,N", [(0, 5), (5, 0), (3, 4), (200, 300)])
def test_empty_sizes(qm, M, N):
    """Nothing to sum: the bias and the residual are left."""
    x, w = torch.empty(M, 0, dtype=BF, device=DEV), torch.empty(N, 0, dtype=BF, device=DEV)
    b, r = _randn(N), _randn(M, N, seed=1)
    assert torch.equal(qm.linear(x, w, bias=b, resid=r), r + b)


@pytest.mark.parametrize("M", [2, 40, 300])
def test_infinities_and_nan_stay_in_their_rows(qm, M):
    x, w = _randn(M, 128, dtype=BF), _randn(200, 128, seed=1, dtype=BF)
    clean = qm.linear(x, w, out_dtype=F32)
    x[1, 3], w[7, 100] = float("nan"), float("inf")
    got = qm.linear(x, w, out_dtype=F32)
    assert got[1].isnan().all()
    rows, cols = [i for i in range(M) if i != 1], [i for i in range(200) if i != 7]
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
    assert not got[rows, 7].isfinite().any()


def test_far_outputs_and_rows(qm):
    """Outputs past 2^32 values, and rows of x past 2^32."""
    M, N, K = 70000, 62000, 8
    g = torch.Generator().manual_seed(0)
    x = torch.randint(-4, 5, (M, K), generator=g).to(BF).to(DEV)
    w = torch.randint(-4, 5, (N, K), generator=g).to(BF).to(DEV)
    got = qm.linear(x, w)
    at = torch.tensor([0, 1, 34636, 69273, 69999], device=DEV)
    assert torch.equal(got[at].float(), x[at].float() @ w.float().T)
    del got
    wide = torch.empty(70000, 62000, dtype=BF, device=DEV)
    wide[:, :K] = x
    assert torch.equal(qm.linear(wide[:, :K], w[:64])[at].float(), x[at].float() @ w[:64].float().T)


def test_repeats_bit_by_bit(qm):
    for M, N, K in ((4, 5120, 2880), (333, 2880, 4096)):
        x, w = _randn(M, K, dtype=BF), _randn(N, K, seed=1, dtype=BF)
        a = qm.linear(x, w)
        assert all(torch.equal(a, qm.linear(x, w)) for _ in range(5))
