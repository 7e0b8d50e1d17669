"""Windows over 8-bit caches, and windows whose keys are split, against the 64-bit form; a page table row
that all sequences share."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_attention_parts import BF, DEV, E4, FP, Shared, run  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_gemv_amd as qm
    return qm


@pytest.mark.parametrize("new,total", [([1], [331]), ([40], [201]), ([1, 40, 0, 5, 129], [77, 64, 9, 5, 331])])
@pytest.mark.parametrize("window,keep", [(1, 0), (33, 4), (128, 40), (100, 1000)])
@pytest.mark.parametrize("dtype,Hkv,G,D,page", [(BF, 2, 4, 64, 16), (FP, 1, 8, 128, 5), (BF, 2, 2, 80, 8)])
def test_windows_of_8_bit_caches(qm, new, total, window, keep, dtype, Hkv, G, D, page):
    s = Shared(qm, new, total, Hkv, G, D, dtype, E4, page)
    sinks = torch.linspace(-3, 2, Hkv * G, device=DEV)
    out, _ = run(qm, s, window=window, keep_first=keep, sinks=sinks)
    s.check(out, window=window, keep=keep, sinks=sinks)


# tokens alone; chunks; both, with splits of the one kind or of both
@pytest.mark.parametrize("new,total", [([1], [9000]), ([1, 3, 1], [9000, 3, 5000]), ([60], [6000]),
                                       ([40, 1, 60, 2], [5000, 9000, 700, 300]), ([300, 1], [2000, 8000])])
@pytest.mark.parametrize("window,keep", [(2048, 4), (4000, 0), (600, 700), (1000, 1 << 20)])
@pytest.mark.parametrize("dtype,cache,page", [(BF, BF, 16), (FP, FP, 8), (BF, E4, 32), (BF, BF, 5)])
def test_windows_whose_keys_are_split(qm, new, total, window, keep, dtype, cache, page):
    """The window's keys and the kept ones before them are shared out together."""
    s = Shared(qm, new, total, 1, 8, 64, dtype, cache, page)
    sinks = torch.linspace(-3, 4, 8, device=DEV)
    out, need = run(qm, s, window=window, keep_first=keep, sinks=sinks)
    assert need > 0
    s.check(out, window=window, keep=keep, sinks=sinks)


@pytest.mark.parametrize("hints", [True, False])
def test_many_sequences_on_shared_pages(qm, hints):
    """More sequences than the search probes at once, all through one row of the page table."""
    g = torch.Generator().manual_seed(2)
    new = torch.randint(0, 3, (300,), generator=g).tolist()
    total = [n + int(torch.randint(1, 40, (), generator=g)) for n in new]
    s = Shared(qm, new, total, 2, 2, 32, page=8, hints=hints)
    s.check(run(qm, s)[0])
