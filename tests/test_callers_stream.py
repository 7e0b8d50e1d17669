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


# --------------------------------------------------------------- the layer and its stages

X, WR = _zeros(T, H, dt=BF), _zeros(E, H, dt=BF)
IDS, COUNTS = _zeros(T, K, dt=I32), _zeros(E, dt=I32)
PLANES = {n + p: torch.zeros(E, 16 * 3, c, dtype=U8) for n in ("gate", "up", "down")
          for p, c in (("_q", 16), ("_s", 1))}
LAYER_CALLS = {
    "route": (3, lambda st: qm.route(X, WR, None, K, stream=st)),
    "bucket": (5, lambda st: qm.bucket(IDS, E, stream=st)),
    "expert_ffn": (2, lambda st: qm.expert_ffn(POOL, SM, X, K, OFF, PERM, stream=st)),
    "expert_gate_up": (1, lambda st: qm.expert_gate_up(POOL, SM, X, K, OFF, PERM, stream=st)),
    "expert_down": (1, lambda st: qm.expert_down(POOL, SM, T, K, OFF, _zeros(T * K, I, dt=BF),
                                                 stream=st)),
    "combine": (1, lambda st: qm.combine(_zeros(T * K, H), PERM, _zeros(T, K), stream=st)),
    "miss_list": (3, lambda st: qm.miss_list(SM, OFF, PERM, K, stream=st)),
    "stage_plan": (3, lambda st: qm.stage_plan(COUNTS, SM, 0, 1, stream=st)),
    "layer": (2, lambda st: qm.layer(POOL, SM, WR, None, X, K, stream=st)),
    "layer_noalloc": (1, lambda st: qm.layer_noalloc(POOL, SM, WR, None, X, K, stream=st)),
    "from_canonical": (6, lambda st: qm.Pool.from_canonical("mxfp4", 32, 48, PLANES, "cpu", st)),
}


@pytest.fixture
def layer_notes(notes, monkeypatch):
    monkeypatch.setattr(qm, "_need", lambda *a: None)
    monkeypatch.setattr(qm, "route_scratch_bytes", lambda *a: 512)
    monkeypatch.setattr(qm, "bucket_scratch_bytes", lambda *a: 512)
    for fn in ("_pool_pack", "_route", "_bucket", "_ffn", "_gate_up", "_down", "_combine",
               "_miss_list", "_stage_plan", "_layer", "_layer_noalloc"):
        monkeypatch.setattr(qm, fn, lambda *a: 0)
    monkeypatch.setattr(qm, "_stream", lambda *a: None)
    return notes


@pytest.mark.parametrize("name", LAYER_CALLS)
def test_layer_buffers_belong_to_the_given_stream(layer_notes, name):
    n, call = LAYER_CALLS[name]
    side = object()
    with layer_notes:
        call(side)
    assert layer_notes.seen == [side] * len(layer_notes.seen) and len(layer_notes.seen) >= n


def test_miss_count_is_read_behind_the_kernel(layer_notes, monkeypatch):
    read = []
    item = torch.Tensor.item
    monkeypatch.setattr(torch.Tensor, "item", lambda t: read.append(layer_notes.current) or 0)
    side = object()
    with layer_notes:
        qm.miss_list(SM, OFF, PERM, K, stream=side)
    monkeypatch.setattr(torch.Tensor, "item", item)
    assert read == [side]
