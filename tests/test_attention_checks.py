"""Refusals of the rotary, cache, attention and dense-product calls: on the host, before any launch,
without a GPU. The binding's checks of tensors, too."""
import pytest

torch = pytest.importorskip("torch")
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

lib = qm._lib
OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE, ODD = 0x10000, 0x10004        # never dereferenced
OUT = 0x30000
BF, FP, F32, E4 = 1, 2, 3, 4


def said():
    return lib.moe_last_error().decode()


def heads(p=FAKE, token=512, head=64):
    return qm.HeadsStruct(p, token, head)


def plan(freq=FAKE, dim=64, layout=0, scale=1.0):
    return qm.RopeStruct(freq, dim, layout, scale)


def cache(type=BF, n_pages=4, page_size=16, n_heads=2, D=64, k=FAKE, strides=(2048, 128, 64), v=FAKE,
          k_scale=None, v_scale=None):
    return qm.KvCacheStruct(type, n_pages, page_size, n_heads, D, k, *strides, v, 2048, 128, 64,
                            k_scale, v_scale)


def batch(n_seq=2, T=3, q_start=FAKE, seq_len=FAKE, table=FAKE, max_pages=4, stride=4, max_q=2,
          max_len=9):
    return qm.KvBatchStruct(n_seq, T, q_start, seq_len, table, max_pages, stride, max_q, max_len)


def rope(p=None, x=None, type=BF, T=3, n=8, D=64, pos=FAKE, inv=0, out=None):
    return lib.moe_rope(p or plan(), x or heads(), type, T, n, D, pos, inv, out or heads(0x20000), None)


def test_rope():
    assert rope(T=0) == OK
    assert rope(type=4) == UNSUPPORTED and rope(type=0) == UNSUPPORTED
    assert rope(p=plan(layout=2)) == UNSUPPORTED
    for p in (plan(dim=0), plan(dim=3), plan(dim=66), plan(dim=-2), plan(freq=None),
              plan(freq=ODD)):
        assert rope(p=p) == INVALID, (p.dim, p.freq)
    for kw in (dict(T=-1), dict(n=0), dict(D=1), dict(D=1026), dict(n=1 << 23, D=64),
               dict(T=1 << 28, n=8), dict(pos=None), dict(pos=0x10002),
               dict(x=heads(None)), dict(x=heads(0x10001)), dict(x=heads(token=-8)),
               dict(x=heads(head=-1)), dict(x=heads(token=1 << 32)), dict(out=heads(None)),
               dict(out=heads(FAKE, 513))):
        assert rope(**kw) == INVALID, kw
        assert said()
    assert lib.moe_rope(None, heads(), BF, 3, 8, 64, FAKE, 0, heads(), None) == INVALID
    assert lib.moe_rope(plan(), None, BF, 3, 8, 64, FAKE, 0, heads(), None) == INVALID
    assert rope(x=heads(token=512), out=heads(token=1024)) == INVALID
    assert "other strides" in said()


BAD_CACHES = [dict(n_pages=0), dict(page_size=0), dict(n_heads=0), dict(D=0), dict(D=24),
              dict(D=272), dict(k=None), dict(v=None), dict(k=ODD), dict(strides=(2048, 128, 60)),
              dict(strides=(-2048, 128, 64)), dict(strides=(2048, 1 << 32, 64)),
              dict(k_scale=FAKE), dict(type=E4, strides=(2048, 128, 72)),
              dict(type=E4, v_scale=0x10002)]
BAD_BATCHES = [dict(n_seq=-1), dict(n_seq=1 << 24), dict(T=-1), dict(T=(1 << 29) + 1), dict(max_pages=0),
               dict(max_pages=1 << 27), dict(stride=-1), dict(stride=1 << 32), dict(max_q=-1),
               dict(max_len=-1), dict(q_start=None), dict(seq_len=None), dict(table=None),
               dict(table=0x10002)]


def append(c=None, b=None, k=None, v=None, type=BF, r=None, pos=None, q=None, n_q=4, q_out=None,
           err=None):
    return lib.moe_kv_append(c or cache(), b or batch(), k or heads(), v or heads(), type, r, pos, q,
                             n_q, q_out, err, None)


def attend(c=None, b=None, q=None, type=BF, n_q=4, scale=1.0, causal=1, window=0, keep=0, sinks=None,
           out=None, scratch=None, size=0, err=None):
    return lib.moe_attend(c or cache(), b or batch(), q or heads(), type, n_q, scale, causal, window,
                          keep, sinks, out or heads(OUT), scratch, size, err, None)


def test_caches_and_batches():
    for call in (append, attend):
        for kw in BAD_CACHES:
            assert call(c=cache(**kw)) == INVALID, (call, kw)
        for t in (0, 3, 5):
            assert call(c=cache(type=t)) == UNSUPPORTED
        for kw in BAD_BATCHES:
            assert call(b=batch(**kw)) == INVALID, (call, kw)
        assert call(b=batch(T=0)) == OK and call(b=batch(n_seq=0)) == OK
        assert call(err=0x10001) == INVALID
    assert lib.moe_kv_append(None, batch(), heads(), heads(), BF, None, None, None, 0, None, None,
                             None) == INVALID
    assert lib.moe_attend(cache(), None, heads(), BF, 4, 1.0, 1, 0, 0, None, heads(), None, 0, None,
                          None) == INVALID


def test_append():
    assert append(type=4) == UNSUPPORTED
    for kw in (dict(q=heads()), dict(q_out=heads()), dict(q=heads(), q_out=heads(), n_q=0),
               dict(k=heads(None)), dict(v=heads(0x10001)), dict(k=heads(token=-1)),
               dict(r=plan(dim=66)), dict(r=plan(freq=None)), dict(pos=0x10002),
               dict(q=heads(), q_out=heads(token=1024)), dict(q=heads(), q_out=heads(None))):
        assert append(**kw) == INVALID, kw
    assert append(r=plan(layout=-1)) == UNSUPPORTED


def test_attend():
    assert attend(type=F32) == UNSUPPORTED and attend(type=FP) == UNSUPPORTED
    for kw in (dict(n_q=3), dict(n_q=0), dict(window=-1), dict(keep=-1), dict(window=4, causal=0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q=heads(None)),
               dict(q=heads(0x10008)), dict(q=heads(head=60)), dict(out=heads(token=-8)),
               dict(sinks=0x10002)):
        assert attend(**kw) == INVALID, kw
    assert attend(out=heads()) == INVALID and "out is q" in said()
    # a grid's dimension holds fewer than 2^24 workgroups of 256 threads
    for call in (append, attend):
        assert call(c=cache(n_heads=1 << 24, D=16), b=batch(T=1)) == INVALID and "heads" in said()
    long = batch(n_seq=1, T=1, max_pages=4096, max_len=60000)
    need = lib.moe_attend_scratch_bytes(cache(), long, 4, 0, 0)
    assert need > 0 and need % (4 * 66 * 4) == 0           # whole splits of 4 rows
    assert attend(b=long) == INVALID and "scratch" in said()
    assert attend(b=long, scratch=FAKE, size=need - 1) == INVALID
    assert attend(b=long, scratch=ODD, size=need) == INVALID
    assert lib.moe_attend_scratch_bytes(cache(), batch(T=0), 4, 0, 0) == 0
    assert lib.moe_attend_scratch_bytes(cache(D=7), long, 4, 0, 0) == 0


def linear(x=FAKE, xs=64, w=FAKE, ws=64, type=BF, M=4, N=32, K=64, bias=None, bt=0, act=0, resid=None,
           rs=32, out=OUT, ot=BF, os=32):
    return lib.moe_linear(x, xs, w, ws, type, M, N, K, bias, bt, act, resid, rs, out, ot, os, None)


def test_linear():
    for kw in (dict(type=F32), dict(type=0), dict(ot=4), dict(ot=0), dict(bias=FAKE, bt=0),
               dict(act=5), dict(act=-1)):
        assert linear(**kw) == UNSUPPORTED, kw
    for kw in (dict(M=-1), dict(N=-1), dict(K=-8), dict(K=60), dict(M=1 << 30), dict(N=1 << 30),
               dict(K=1 << 30), dict(M=1 << 21, N=1 << 20), dict(x=None), dict(w=None), dict(x=ODD),
               dict(w=ODD), dict(xs=-8), dict(ws=60), dict(xs=1 << 39), dict(out=None),
               dict(out=0x10001), dict(ot=F32, out=0x10002), dict(resid=0x10001),
               dict(bias=0x10002, bt=F32), dict(os=31), dict(os=1 << 39), dict(resid=FAKE, rs=-1),
               dict(resid=FAKE, rs=1 << 39), dict(resid=OUT, rs=64, os=32), dict(out=FAKE, w=0x20000),
               dict(out=FAKE, x=0x20000)):
        assert linear(**kw) == INVALID, kw
        assert said()
    assert linear(M=0) == OK and linear(N=0) == OK


# ------------------------------------------------------------------------- the binding




@pytest.fixture
def on_device(monkeypatch):
    """CPU tensors pass for device tensors, and no call leaves the binding."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    calls = []
    monkeypatch.setattr(qm, "_run", lambda fn, like, stream, *a: calls.append((fn, a)))
    return calls


def z(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt)


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="device"):
        qm.linear(z(2, 8), z(4, 8))
    with pytest.raises(ValueError, match="device"):
        qm.KvCache(z(1, 16, 2, 64), z(1, 16, 2, 64))
    with pytest.raises(ValueError):
        qm.Rope(torch.zeros(4, dtype=torch.float64))


def test_binding(on_device):
    i32 = torch.int32
    p = qm.Rope(z(32, dt=torch.float64))
    kv = qm.KvCache(z(4, 16, 2, 64), z(4, 16, 2, 64))
    b = qm.KvBatch(z(3, dt=i32), z(2, dt=i32), z(2, 4, dt=i32), 1, 9)
    x = z(5, 4, 64)
    for bad, call in (
            (TypeError, lambda: qm.Rope(z(32))),
            (ValueError, lambda: qm.Rope(z(32, dt=torch.float64), "quarter")),
            (TypeError, lambda: qm.KvCache(z(4, 16, 2, 64, dt=torch.float32), z(4, 16, 2, 64))),
            (TypeError, lambda: qm.KvCache(z(4, 16, 2, 64), z(4, 16, 2, 64, dt=torch.float16))),
            (ValueError, lambda: qm.KvCache(z(4, 16, 2, 64), z(4, 16, 2, 32))),
            (ValueError, lambda: qm.KvCache(z(4, 16, 2), z(4, 16, 2))),
            (ValueError, lambda: qm.KvCache(z(4, 16, 64, 2).transpose(2, 3), z(4, 16, 2, 64))),
            (ValueError, lambda: qm.KvCache(z(4, 16, 2, 64), z(4, 16, 2, 64),
                                            z(3, dt=torch.float32))),
            (ValueError, lambda: qm.KvBatch(z(2, dt=i32), z(2, dt=i32), z(2, 4, dt=i32))),
            (TypeError, lambda: qm.KvBatch(z(3, dt=torch.int64), z(2, dt=i32), z(2, 4, dt=i32))),
            (ValueError, lambda: qm.KvBatch(z(3, dt=i32), z(2, dt=i32), z(3, 4, dt=i32))),
            (ValueError, lambda: qm.KvBatch(z(3, dt=i32), z(2, dt=i32), z(8, dt=i32))),
            (ValueError, lambda: qm.rope(z(5, 64), z(5, dt=i32), p)),
            (TypeError, lambda: qm.rope(x, z(5, dt=torch.int64), p)),
            (ValueError, lambda: qm.rope(x, z(4, dt=i32), p)),
            (ValueError, lambda: qm.rope(x, z(5, dt=i32), p, out=z(5, 4, 32))),
            (TypeError, lambda: qm.rope(x, z(5, dt=i32), p, out=z(5, 4, 64, dt=torch.float16))),
            (ValueError, lambda: qm.kv_append(kv, b, x, x)),
            (ValueError, lambda: qm.kv_append(kv, b, x[:, :2], x[:4, :2])),
            (TypeError, lambda: qm.kv_append(kv, b, x[:, :2], x[:, :2].half())),
            (ValueError, lambda: qm.kv_append(kv, b, x[:, :2], x[:, :2], q_out=x)),
            (ValueError, lambda: qm.kv_append(kv, b, x[:, :2], x[:, :2], q=x[:4])),
            (ValueError, lambda: qm.kv_append(kv, b, x[:, :2], x[:, :2], err_flags=z(0, dt=i32))),
            (TypeError, lambda: qm.attend(x.float(), kv, b)),
            (ValueError, lambda: qm.attend(z(5, 4, 32), kv, b)),
            (ValueError, lambda: qm.attend(x[0], kv, b)),
            (ValueError, lambda: qm.attend(x, kv, b, sinks=z(3, dt=torch.float32))),
            (TypeError, lambda: qm.attend(x, kv, b, sinks=z(4))),
            (TypeError, lambda: qm.attend(x, kv, b, scratch=z(4))),
            (ValueError, lambda: qm.attend(x, kv, b, out=z(5, 4, 128)[..., ::2])),
            (ValueError, lambda: qm.linear(z(5, 8), z(4, 16))),
            (TypeError, lambda: qm.linear(z(5, 8), z(4, 8).half())),
            (TypeError, lambda: qm.linear(z(5, 8).float(), z(4, 8).float())),
            (ValueError, lambda: qm.linear(z(5, 8), z(4, 8), bias=z(5))),
            (ValueError, lambda: qm.linear(z(5, 8), z(4, 8), act="tanh")),
            (TypeError, lambda: qm.linear(z(5, 8), z(4, 8), resid=z(5, 4), out_dtype=torch.float32)),
            (ValueError, lambda: qm.linear(z(5, 8), z(4, 8), out_dtype=torch.int32)),
            (ValueError, lambda: qm.linear(z(5, 8), z(4, 8), out=z(4, 5).T)),
            (ValueError, lambda: qm.Rope.make(7)),
            (ValueError, lambda: qm.Rope.make(8, scaling="cubic")),
            (ValueError, lambda: qm.Rope.make(2, scaling="ntk"))):
        with pytest.raises(bad):
            call()
    assert not on_device
    qm.rope(x, z(5, dt=i32), p)
    qm.kv_append(kv, b, x[:, :2], x[:, 2:], rope=p, q=x)
    qm.attend(x, kv, b)
    qm.linear(z(5, 8), z(4, 8))
    assert len(on_device) == 4


def test_sizes_past_31_bits_are_refused(on_device):
    big = torch.empty(1, dtype=torch.bfloat16).expand(1 << 31, 1, 64, 64)[..., 0]
    with pytest.raises(ValueError):
        qm.rope(big, z(1, dt=torch.int32), qm.Rope(z(8, dt=torch.float64)))
    row = torch.empty(8, dtype=torch.bfloat16).expand(1 << 31, 8)
    with pytest.raises(ValueError, match="limit"):
        qm.linear(row, z(4, 8))
    with pytest.raises(ValueError, match="limit"):
        qm.linear(z(4, 8), row)


def test_buffers_belong_to_the_given_stream(monkeypatch):
    """What a call allocates is taken while its stream is current."""
    import contextlib
    seen, current = [], [None]

    @contextlib.contextmanager
    def stream(st):
        current[0], before = st, current[0]
        try:
            yield
        finally:
            current[0] = before

    new_empty, empty_like = torch.Tensor.new_empty, torch.empty_like
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.Tensor, "new_empty",
                        lambda t, *a, **k: (seen.append(current[0]), new_empty(t, *a, **k))[1])
    monkeypatch.setattr(torch, "empty_like",
                        lambda t, *a, **k: (seen.append(current[0]), empty_like(t, *a, **k))[1])
    monkeypatch.setattr(qm, "_run", lambda *a: None)
    i32, side = torch.int32, object()
    p = qm.Rope(z(32, dt=torch.float64))
    kv = qm.KvCache(z(4096, 16, 2, 64), z(4096, 16, 2, 64))
    b = qm.KvBatch(z(2, dt=i32), z(1, dt=i32), z(1, 4096, dt=i32), 1, 60000)
    x = z(1, 4, 64)
    for n, call in ((1, lambda: qm.rope(x, z(1, dt=i32), p, stream=side)),
                    (1, lambda: qm.kv_append(kv, b, x[:, :2], x[:, 2:], q=x, stream=side)),
                    (2, lambda: qm.attend(x, kv, b, stream=side)),       # out and scratch
                    (1, lambda: qm.linear(z(5, 8), z(4, 8), stream=side))):
        seen.clear()
        call()
        assert seen == [side] * n
