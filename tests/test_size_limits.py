"""Sizes that do not fit the C calls' 32-bit arguments: ctypes would pass their low 32 bits, and
the call would work on a part of the tensor. Tensors without memory stand in for the large ones."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

BIG = (1 << 32) + 64
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
POOL = SimpleNamespace(H=64, I=32, planes={"gate_q": torch.empty(1, device="meta")},
                       struct=qm.PoolStruct(qm.MXFP4, 4, 64, 32))


def empty(*shape, dt=F32):
    return torch.empty(shape, dtype=dt, device="meta")


def norm(T, H):
    return qm.add_norm(empty(T, H), empty(H))


def exit_norm(T, H):
    return qm.combine_norm(empty(T, H), empty(T, dt=I32), empty(T, 1), empty(T, H))


def planes(n, K):
    return empty(n, K // 2, dt=U8), empty(n, K // 32, dt=U8)


OFF, SM = empty(5, dt=I32), empty(4, dt=I32)
CALLS = {
    "quantise, long row": lambda: qm.mx_quantize(empty(BIG, dt=BF)),
    "quantise, rows": lambda: qm.mx_quantize(empty(BIG, 32, dt=BF)),
    "quantise, rows of two dimensions": lambda: qm.mx_quantize(empty(1 << 16, BIG >> 16, 32, dt=BF)),
    "dequantise, long row": lambda: qm.mx_dequantize(*planes(1, BIG)),
    "dequantise, rows": lambda: qm.mx_dequantize(*planes(BIG, 32)),
    "norm, long row": lambda: norm(1, BIG),
    "norm, rows": lambda: norm(BIG, 32),
    "exit norm, long row": lambda: exit_norm(1, BIG),
    "exit norm, rows": lambda: exit_norm(BIG, 32),
    "gate/up": lambda: qm.mx_expert_gate_up(POOL, SM, *planes(BIG, 64), "mxfp4", 1, OFF,
                                            empty(BIG, dt=I32)),
    "down": lambda: qm.mx_expert_down(POOL, SM, BIG, 1, OFF, *planes(BIG, 32), "mxfp4"),
    "ffn": lambda: qm.mx_expert_ffn(POOL, SM, *planes(BIG, 64), "mxfp4", 1, OFF, empty(BIG, dt=I32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_sizes_past_32_bits_are_refused(monkeypatch, name):
    launched = []
    monkeypatch.setattr(qm, "_tensor", lambda *a: None)     # they are no device tensors
    monkeypatch.setattr(qm, "_run", lambda *a: launched.append(a))
    with pytest.raises(ValueError, match=r"limit 2\^31"):
        CALLS[name]()
    assert not launched


def test_row_bytes_past_32_bits():
    with pytest.raises(ValueError):
        qm.mx_row_bytes("mxfp4", BIG)
    assert qm.mx_row_bytes("mxfp6", (1 << 31) - 32) == ((1 << 31) - 32) // 4 * 3


def test_the_largest_eps_is_taken():
    """eps is finite and not negative: fp32's largest number is one, what is past it is not.
    No rows, so nothing is launched."""
    import ctypes
    import os
    lib = ctypes.CDLL(os.path.join(os.path.dirname(qm.__file__), "libmoe.so"))
    f32, ptr = ctypes.c_float, ctypes.c_void_p

    def add_norm(eps):
        return lib.moe_add_norm(ptr(), 1, ptr(), 1, f32(1.0), ptr(), 1, f32(eps), 0, 64, ptr(), ptr(),
                                ptr())

    assert [add_norm(e) for e in (0.0, 3.402e38, float.fromhex("0x1.fffffep127"))] == [0, 0, 0]
    assert [add_norm(e) for e in (-1e-45, 3.41e38, float("inf"), float("nan"))] == [1, 1, 1, 1]
