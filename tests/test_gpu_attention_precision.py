"""What rounding the softmax weights costs, against the 64-bit form: tokens whose weights have more bits
than the type."""
import pytest

torch = pytest.importorskip("torch")
import attention_ref as ref  # noqa: E402
from test_gpu_attention_parts import BF, E4, FP, Shared, run  # noqa: E402

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_gemv_amd as qm
    return qm


@pytest.mark.parametrize("new,total", [([1] * 40, [1 + i % 20 for i in range(40)]), ([1] * 8, [100, 333] * 4),
                                       ([3, 1, 2], [9, 7000, 2]), ([1] * 6 + [90], [2, 3, 4, 5, 900, 33, 90])])
@pytest.mark.parametrize("Hkv,G,D", [(2, 8, 64), (1, 3, 128), (1, 8, 256)])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
def test_few_rows_weights_have_more_bits(qm, new, total, Hkv, G, D, dtype, cache):
    """Sequences of up to 32 rows, alone and beside a chunk, in few keys and in split ones."""
    s = Shared(qm, new, total, Hkv, G, D, dtype, cache)
    out, _ = run(qm, s)
    for b, (n, t) in enumerate(zip(new, total)):
        if n * G > 32:
            continue
        rows = slice(s.start[b], s.start[b + 1])
        args = (torch.arange(t - n, t), D ** -0.5)
        k, v = s.rows[0][:t], s.rows[1][:t]
        want, tol = ref.attend(s.q[rows], k, v, *args, dtype=F32)        # all but the weights' rounding
        size, _ = ref.attend(s.q[rows], k, v.abs(), *args, dtype=F32)    # sum of weight times |value|
        # bf16: what is left of a weight is at most 1.25 2^-6 of it, and rounded by 2^-8 of that; fp16: a
        # quarter, by 2^-11, and by 2^-25 where the row's largest weight is above 2^6
        if dtype == BF:
            tol = tol + 1.25 * 2.0 ** -14 * size
        else:
            tol = tol + 2.0 ** -13 * size + t * 2.0 ** -31 * v.abs().amax((0, 2)).repeat_interleave(G)[:, None]
        ref.near(out[rows], want, tol + ref.rounded(want.abs() + tol, dtype), f"sequence {b}: {n} of {t}")


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new,total,G", [([1, 2], [70, 200], 8), ([1, 60], [9000, 70], 4)])
def test_infinite_values_stay_infinite(qm, bad, dtype, new, total, G):
    """A value that every row of its block sees, in both operands of its weight."""
    s = Shared(qm, new, total, 1, G, 64, dtype)
    clean, _ = run(qm, s)
    s.kv.v[s.batch.page_table[0, 0].item(), 5, 0, 9] = bad
    out, _ = run(qm, s)
    T = s.start[-1]
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(new, total)])
    others = [d for d in range(64) if d != 9]
    assert torch.equal(out[:T][..., others], clean[:T][..., others])
    hit = out[:T][pos >= 5][..., 9].float()
    assert (hit.isnan() if bad != bad else hit == bad).all()


@pytest.mark.parametrize("new,total", [([40], [40]), ([90, 50], [90, 52]), ([300, 33], [300, 400]), ([64], [3000])])
@pytest.mark.parametrize("Hkv,G,D", [(2, 1, 64), (1, 4, 128), (1, 2, 256)])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4)])
def test_many_rows_weights_sum_to_one(qm, new, total, Hkv, G, D, dtype, cache):
    """Rounded weights over the sum of the same rounded weights: what a weight's rounding moves is its
    value's distance from the row's output, which is little where few keys have most of the weight."""
    s = Shared(qm, new, total, Hkv, G, D, dtype, cache)
    out, _ = run(qm, s)
    h = ref.half_step(dtype)
    for b, (n, t) in enumerate(zip(new, total)):
        if n * G <= 32:
            continue
        pick = sorted({*range(12), 31, 32, n // 2, n - 1})
        rows = torch.tensor([s.start[b] + i for i in pick])
        pos = torch.tensor([t - n + i for i in pick])
        k, v = s.rows[0][:t], s.rows[1][:t]
        want, tol = ref.attend(s.q[rows], k, v, pos, D ** -0.5, dtype=F32)    # all but the weights' rounding
        for j in range(Hkv * G):
            x = s.q[rows, j].double() @ k[:, j // G].T * D ** -0.5
            w = x.masked_fill(torch.arange(t) > pos[:, None], -torch.inf).softmax(-1)
            away = (v[None, :, j // G] - want[:, None, j]).abs()
            tol[:, j] += h * (1 + 2 * h) * (w[..., None] * away).sum(1)
            if dtype == FP:      # and 2^-25 where the row's largest weight is above 2^6
                tol[:, j] += t * 2.0 ** -31 * away.amax(1)
        ref.near(out[rows], want, tol + ref.rounded(want.abs() + tol, dtype), f"sequence {b}: {n} of {t}")
