"""Rotation, append, attention and products on a stream that their caller names, while the current
stream has work of its own: the buffers that a call makes must not be memory that the current
stream still uses, nor go back to it while the call's stream uses them."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
T, HQ, HKV, D, LONG = 4, 8, 2, 64, 20000


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
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
        n = LONG // 16
        self.cache = qm.KvCache(rand(n, 16, HKV, D), rand(n, 16, HKV, D))
        i32 = dict(dtype=torch.int32, device="cuda")
        self.batch = qm.KvBatch(torch.tensor([0, T], **i32), torch.tensor([LONG], **i32),
                                torch.randperm(n, generator=g, device="cuda").to(torch.int32)[None])
        self.q, self.k = rand(T, HQ, D), rand(T, HKV, D)
        self.pos, self.plan = torch.arange(T, **i32), qm.Rope.make(D)
        self.x, self.w, self.r = rand(333, 512), rand(400, 512), rand(333, 400)
        self.scratch = qm.attend_scratch_bytes(self.cache, self.batch, T, HQ)
        assert self.scratch   # such a call is split, and makes its scratch


CALLS = {   # call -> (result, the shape and type of a buffer that it makes)
    "rope": (lambda a, st: qm.rope(a.q, a.pos, a.plan, stream=st), lambda a: (T, HQ, D), BF),
    "append": (lambda a, st: qm.kv_append(a.cache, a.batch, a.k, a.k, a.plan, q=a.q, stream=st),
               lambda a: (T, HQ, D), BF),
    "attend": (lambda a, st: qm.attend(a.q, a.cache, a.batch, stream=st), lambda a: (T, HQ, D), BF),
    "scratch": (lambda a, st: qm.attend(a.q, a.cache, a.batch, stream=st), lambda a: (a.scratch,), U8),
    "linear": (lambda a, st: qm.linear(a.x, a.w, resid=a.r, act="silu", stream=st),
               lambda a: (333, 400), BF),
}


@pytest.fixture(scope="module")
def args():
    return Args()


@pytest.mark.parametrize("name", CALLS)
def test_buffers_do_not_return_early(args, name):
    """The named stream lags behind: what the current stream allocates and fills after the call
    is not what the call still writes and reads."""
    call, shape, dt = CALLS[name]
    want = call(args, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    keep = busy(side)
    got = call(args, side)
    fill = [torch.full(shape(args), 85, dtype=dt, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((f == 85).all()) for f in fill)
    del keep


@pytest.mark.parametrize("name", CALLS)
def test_buffers_are_not_in_use(args, name):
    """The current stream lags behind: memory that it has freed, but not yet finished with, is
    not what the call writes."""
    call, shape, dt = CALLS[name]
    want = call(args, None)
    torch.cuda.synchronize()
    keep = busy(torch.cuda.current_stream())
    late = [torch.full(shape(args), 85, dtype=dt, device="cuda") for _ in range(16)]
    copies = [t.clone() for t in late]
    del late
    side = torch.cuda.Stream()
    got = call(args, side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((f == 85).all()) for f in copies)
    del keep
