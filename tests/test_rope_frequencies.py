"""Frequencies of contexts scaled by parts (YaRN), against the definition written out, without a GPU."""
import math

import pytest

torch = pytest.importorskip("torch")
import quantized_routed_expert_gemv_amd as qm  # noqa: E402


@pytest.fixture(autouse=True)
def host_tensors(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)


@pytest.mark.parametrize("dim,base,factor,original,fast,slow", [(64, 150000.0, 32.0, 4096, 32.0, 1.0),
                                                                (128, 10000.0, 4.0, 32768, 32.0, 1.0),
                                                                (96, 1e6, 8.0, 2048, 16.0, 2.0),
                                                                (64, 10000.0, 4.0, 64, 32.0, 1.0),
                                                                (4, 10000.0, 2.0, 4096, 32.0, 1.0)])
@pytest.mark.parametrize("whole", [True, False])
def test_ramp(dim, base, factor, original, fast, slow, whole):
    """The ramp runs over the pairs between those that turn `fast` and `slow` times over the original
    context: pair i turns original * base^(-2i/dim) / (2 pi) times. Its ends are whole pairs, or not."""
    p = qm.Rope.make(dim, base, scaling="yarn", factor=factor, original=original, beta_fast=fast,
                     beta_slow=slow, device="cpu", **({} if whole else {"whole_pairs": False}))
    ends = [dim / 2 * math.log(original / (2 * math.pi * b), base) for b in (fast, slow)]
    lo, hi = (math.floor(ends[0]), math.ceil(ends[1])) if whole else ends
    lo, hi = max(lo, 0), min(hi, dim - 1)
    want = []
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        want.append(f / factor * r + f * (1 - r))
    assert p.freq.tolist() == pytest.approx(want, rel=1e-12)
    assert p.scale == pytest.approx(0.1 * math.log(factor) + 1)


def test_unrounded_ends_are_other_frequencies():
    a, b = (qm.Rope.make(64, 150000.0, scaling="yarn", factor=32.0, whole_pairs=w, device="cpu").freq
            for w in (True, False))
    assert not torch.equal(a, b)
    assert torch.equal(a[:8], b[:8]) and torch.equal(a[18:], b[18:])      # ends 8.09 and 17.40
