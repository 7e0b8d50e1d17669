"""Scores that are far apart."""
import pytest

torch = pytest.importorskip("torch")
import attention_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_gemv_amd as qm
    return qm


def _batch(qm, T, L, page, max_len):
    i32 = dict(dtype=torch.int32, device=DEV)
    return qm.KvBatch(torch.tensor([0, T], **i32), torch.tensor([L], **i32),
                      torch.arange(-(-L // page), **i32)[None], T, max_len)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("first", [0, 1, 2])
def test_scores_a_step_of_fp32_apart(qm, T, dtype, first):
    """Scores past 2^27 (of powers of two), where neighbouring fp32 numbers are 16 apart: the higher of
    two keys has nearly all of the weight, whichever comes first."""
    L, D, page = 256, 64, 16
    scale = 11.090355                # times log2(e) in fp32: 16
    k = torch.zeros(L // page, page, 1, D, device=DEV)
    v = torch.zeros(L // page, page, 1, D, device=DEV)
    for j, extra in ((0, first), (128, first + 1)):
        k[j // page, j % page, 0, 0] = 2048.0
        k[j // page, j % page, 0, 1] = float(extra)
        v[j // page, j % page, 0, :] = 1.0 + j
    q = torch.zeros(T, 2, D, dtype=dtype, device=DEV)
    q[..., 0], q[..., 1] = 4096.0, 1.0
    out = qm.attend(q, qm.KvCache(k.to(dtype), v.to(dtype)), _batch(qm, T, L, page, 1), scale=scale)
    # the lower key's weight is 2^-16 of the higher one's
    want = torch.full(out.shape, 129.0 - 128.0 / (1 + 2 ** 16), dtype=torch.float64)
    ref.near(out, want, 2 * ref.half_step(dtype) * want, "scores")
