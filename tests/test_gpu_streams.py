"""Calls on a stream that their caller names, while the current stream has work of its own: the
buffers that a call makes must not be memory that the current stream still uses, nor go back to
it while the call's stream uses them."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
T, H, I, E, K = 500, 512, 352, 8, 2


def busy(stream):
    """Some tens of milliseconds of work on a stream."""
    with torch.cuda.stream(stream):
        a = torch.ones(8192, 8192, dtype=BF, device="cuda")
        for _ in range(30):
            b = a @ a
        return a, b


class Args:
    def __init__(self):
        g = torch.Generator("cuda").manual_seed(0)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.planes = planes = {}
        for n, r, c in (("gate", I, H), ("up", I, H), ("down", H, I)):
            planes[n + "_q"], planes[n + "_s"] = qm.mx_quantize(rand(E, r, c) / c ** 0.5)
        self.pool = qm.Pool.from_canonical("mxfp4", H, I, planes)
        self.sm = torch.arange(E, dtype=torch.int32, device="cuda")
        self.x, self.w = rand(T, H).to(BF), rand(H)
        self.x4 = qm.mx_quantize(self.x)
        self.h4 = qm.mx_quantize(rand(T * K, I))
        self.ids = torch.argsort(rand(T, E), 1)[:, :K].to(torch.int32).contiguous()
        _, self.off, self.perm, self.inv = qm.bucket(self.ids, E)
        self.part = torch.where(self.sm % 3 == 0, qm.SLOT_MISS, self.sm).to(torch.int32)
        self.wr = (rand(E, H) / H ** 0.5).to(BF)
        self.y, self.tw = rand(T * K, H), rand(T, K)


CALLS = {   # call -> (result, the shape and type of a buffer that it makes)
    "quantize": (lambda a, st: qm.mx_quantize(a.x, stream=st), (T, H // 2), U8),
    "dequantize": (lambda a, st: qm.mx_dequantize(*a.x4, stream=st), (T, H), BF),
    "gate_up": (lambda a, st: qm.mx_expert_gate_up(a.pool, a.sm, *a.x4, "mxfp4", K, a.off, a.perm,
                                                   stream=st), (T * K, I), BF),
    "down": (lambda a, st: qm.mx_expert_down(a.pool, a.sm, T, K, a.off, *a.h4, "mxfp4", stream=st),
             (T * K, H), F32),
    "ffn": (lambda a, st: qm.mx_expert_ffn(a.pool, a.sm, *a.x4, "mxfp4", K, a.off, a.perm,
                                           stream=st), (T * K, I // 2), U8),
    "add_norm": (lambda a, st: qm.add_norm(a.x, a.w, delta=a.x, stream=st), (T, H), BF),
    "combine_norm": (lambda a, st: qm.combine_norm(a.y, a.inv, a.tw, a.x, next_weight=a.w,
                                                   stream=st), (T, H), BF),
    "route": (lambda a, st: qm.route(a.x, a.wr, None, K, stream=st), (T, K), F32),
    "bucket": (lambda a, st: qm.bucket(a.ids, E, stream=st), (T * K,), torch.int32),
    "miss_list": (lambda a, st: qm.miss_list(a.part, a.off, a.perm, K, stream=st), (T * K,),
                  torch.int32),
    "expert_ffn": (lambda a, st: qm.expert_ffn(a.pool, a.sm, a.x, K, a.off, a.perm, stream=st),
                   (T * K, H), F32),
    "layer": (lambda a, st: qm.layer(a.pool, a.sm, a.wr, None, a.x, K, stream=st)[0], (T, H), F32),
    "from_canonical": (lambda a, st: tuple(qm.Pool.from_canonical("mxfp4", H, I, a.planes,
                                                                  stream=st).planes.values()),
                       (E, I, H // 2), U8),
}


@pytest.fixture(scope="module")
def args():
    return Args()


def tensors(r):
    return list(r) if isinstance(r, tuple) else [r]


@pytest.mark.parametrize("name", CALLS)
def test_buffers_do_not_return_early(args, name):
    """The named stream lags behind: what the current stream allocates and fills after the call
    is not what the call still writes and reads."""
    call, shape, dt = CALLS[name]
    want = tensors(call(args, None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    keep = busy(side)
    got = tensors(call(args, side))
    fill = [torch.full(shape, 85, dtype=dt, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((f == 85).all()) for f in fill)
    del keep


@pytest.mark.parametrize("name", CALLS)
def test_buffers_are_not_in_use(args, name):
    """The current stream lags behind: memory that it has freed, but not yet finished with, is
    not what the call writes."""
    call, shape, dt = CALLS[name]
    want = tensors(call(args, None))
    torch.cuda.synchronize()
    keep = busy(torch.cuda.current_stream())
    late = [torch.full(shape, 85, dtype=dt, device="cuda") for _ in range(16)]
    copies = [t.clone() for t in late]
    del late
    side = torch.cuda.Stream()
    got = tensors(call(args, side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((f == 85).all()) for f in copies)
    del keep
