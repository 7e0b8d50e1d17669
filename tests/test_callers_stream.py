"""Buffers that a call allocates itself, when its caller names a stream: each has to be taken
while that stream is current. The allocator keeps memory by stream, so a buffer of another
stream can still be in use there when this one writes it, and a temporary goes back to that
other stream's work as soon as the call returns. Shown here without a GPU: the launch is left
out and every allocation noted with the stream that was current."""
import contextlib
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
from torch.utils._python_dispatch import TorchDispatchMode  # noqa: E402

import quantized_routed_expert_gemv_amd as qm  # noqa: E402

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
T, H, I, E, K = 6, 96, 64, 4, 2
ALLOCATE = {torch.ops.aten.empty, torch.ops.aten.empty_like, torch.ops.aten.new_empty}


class Allocations(TorchDispatchMode):
    """Notes the stream that is current at each allocation."""

    def __init__(self):
        super().__init__()
        self.current, self.seen = None, []

    @contextlib.contextmanager
    def stream(self, st):
        self.current, before = st, self.current
        try:
            yield
        finally:
            self.current = before

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if func.overloadpacket in ALLOCATE:
            self.seen.append(self.current)
        return func(*args, **(kwargs or {}))


def _zeros(*shape, dt=F32):
    return torch.zeros(shape, dtype=dt)


@pytest.fixture
def notes(monkeypatch):
    notes = Allocations()
    monkeypatch.setattr(torch.cuda, "stream", notes.stream)
    monkeypatch.setattr(qm, "_run", lambda *a: None)
    monkeypatch.setattr(qm, "_tensor", lambda *a: None)
    return notes


POOL = SimpleNamespace(H=H, I=I, planes={"gate_q": torch.zeros(1)},
                       struct=qm.PoolStruct(qm.MXFP4, E, H, I))
SM, OFF, PERM = _zeros(E, dt=I32), _zeros(E + 1, dt=I32), _zeros(T * K, dt=I32)
X4 = _zeros(T, H // 2, dt=U8), _zeros(T, H // 32, dt=U8)
H4 = _zeros(T * K, I // 2, dt=U8), _zeros(T * K, I // 32, dt=U8)
CALLS = {   # call -> buffers that it allocates
    "quantize": (2, lambda st: qm.mx_quantize(_zeros(T, H, dt=BF), stream=st)),
    "dequantize": (1, lambda st: qm.mx_dequantize(*X4, stream=st)),
    "gate_up": (1, lambda st: qm.mx_expert_gate_up(POOL, SM, *X4, "mxfp4", K, OFF, PERM, stream=st)),
    "down": (1, lambda st: qm.mx_expert_down(POOL, SM, T, K, OFF, *H4, "mxfp4", stream=st)),
    "ffn": (4, lambda st: qm.mx_expert_ffn(POOL, SM, *X4, "mxfp4", K, OFF, PERM, stream=st)),
    "add_norm": (2, lambda st: qm.add_norm(_zeros(T, H), _zeros(H), delta=_zeros(T, H), stream=st)),
    "combine_norm": (2, lambda st: qm.combine_norm(_zeros(T * K, H), PERM, _zeros(T, K), _zeros(T, H),
                                                   next_weight=_zeros(H), stream=st)),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_belong_to_the_given_stream(notes, name):
    n, call = CALLS[name]
    side = object()
    with notes:
        call(side)
    mine = [st for st in notes.seen if st is side]
    assert len(mine) == n, notes.seen


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one(notes, name):
    with notes:
        CALLS[name][1](None)
    assert notes.seen and all(st is None for st in notes.seen)


def test_a_stream_of_another_device_is_refused():
    like = SimpleNamespace(device=torch.device("cuda", 0), get_device=lambda: 0)
    launched = []
    with pytest.raises(ValueError, match="stream: on cuda:1"):
        qm._run(lambda *a: launched.append(a) or 0, like,
                SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=16))
    assert not launched
