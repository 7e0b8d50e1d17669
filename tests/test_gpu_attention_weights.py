"""Softmax weights far below the row's largest, and scores that are far apart."""
import math

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


def _batch(qm, T, L, page, max_len):
    i32 = dict(dtype=torch.int32, device=DEV)
    return qm.KvBatch(torch.tensor([0, T], **i32), torch.tensor([L], **i32),
                      torch.arange(-(-L // page), **i32)[None], T, max_len)


@pytest.mark.parametrize("T", [1, 40])                # the kernels for few and for many rows
@pytest.mark.parametrize("top", [13.0, 16.0, 18.0, 20.0])
@pytest.mark.parametrize("dtype,cache", [(FP, FP), (FP, E4), (BF, BF)])
@pytest.mark.parametrize("split", [False, True])
def test_small_weights_of_many_keys(qm, T, top, dtype, cache, split):
    """Four keys that stand 18 to 28 binary orders above 131068 others, whose weights are together far
    from nothing: values of 1 (others) beside 0 (the four), and of 1 everywhere."""
    L, D, page, G, low = 131072, 64, 64, 4, 0.25
    k = torch.zeros(L // page, page, 1, D, device=DEV)
    v = torch.ones(L // page, page, 1, D, device=DEV)
    k[..., 0] = low
    high = [0, 32, 64, 96]           # each wave that shares out the keys has one of them first
    for j in high:
        k[j // page, j % page, 0, 0] = top
        v[j // page, j % page, 0, :32] = 0.0
    q = torch.zeros(T, G, D, dtype=dtype, device=DEV)
    q[..., 0] = 1.0
    out = qm.attend(q, qm.KvCache(k.to(cache), v.to(cache)), _batch(qm, T, L, page, L if split else 1),
                    scale=1.0).double().cpu()
    n = torch.arange(L - T, L, dtype=torch.float64) + 1 - len(high)
    share = n * math.exp(low) / (n * math.exp(low) + len(high) * math.exp(top))
    want = torch.ones(T, G, D, dtype=torch.float64)
    want[..., :32] = share[:, None, None]
    # a weight is rounded to the type: half a step, and of fp16 half of the smallest step, 2^-25, of
    # weights whose largest is above 2^6. Scores: two roundings of a number below 2^5, and exp2's; the
    # sums, L additions of the weights' sum in fp32 each.
    tol = (ref.half_step(dtype) + 2 * 2.0 ** -17 + 2 * (L + 64) * ref.F32) * want
    if dtype == FP:
        tol = tol + L * 2.0 ** -25 / 2 ** 6
    ref.near(out, want, tol + ref.rounded(want, dtype), "weights")


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
