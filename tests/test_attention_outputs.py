"""What the rotary, append and attention calls allocate for rows of any strides, without a GPU."""
import pytest

torch = pytest.importorskip("torch")
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

# (tokens, heads, values), strides: rows that overlap, that are expanded, that come heads first
VIEWS = [((8, 37, 64), (100, 1, 1)), ((8, 1, 64), (1, 1, 1)), ((8, 2, 64), (2, 1, 1)),
         ((8, 4, 64), (1, 64, 1)), ((200, 4, 64), (1, 64, 1)), ((8, 4, 64), (0, 0, 1)),
         ((8, 4, 64), (64, 0, 1)), ((8, 4, 64), (0, 1, 1)), ((4, 8, 64), (64, 256, 1)),
         ((1, 1, 64), (7, 3, 1)), ((3, 5, 64), (700, 80, 1)), ((0, 100, 64), (0, 1, 1))]


@pytest.fixture
def passed(monkeypatch):
    """CPU tensors pass for device tensors, and no call leaves the binding."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(qm, "_run", lambda *a: None)


def _dense_and_apart(out, shape):
    assert out.shape == shape and out.stride(-1) == 1
    at = sum(torch.arange(n).view([-1 if j == i else 1 for j in range(3)]) * out.stride(i)
             for i, n in enumerate(shape))
    assert at.unique().numel() == out.numel()


@pytest.mark.parametrize("shape,strides", VIEWS)
def test_new_outputs_are_dense(passed, shape, strides):
    T, n, D = shape
    i32 = dict(dtype=torch.int32)
    x = torch.zeros(1 << 14, dtype=torch.bfloat16).as_strided(shape, strides)
    plan = qm.Rope(torch.zeros(32, dtype=torch.float64))
    _dense_and_apart(qm.rope(x, torch.zeros(T, **i32), plan), shape)
    kv = qm.KvCache(*(torch.zeros(4, 16, 1, D, dtype=x.dtype) for _ in range(2)))
    b = qm.KvBatch(torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1, 4, **i32))
    new = torch.zeros(T, 1, D, dtype=x.dtype)
    _dense_and_apart(qm.kv_append(kv, b, new, new, plan, q=x), shape)
    _dense_and_apart(qm.attend(x, kv, b), shape)


def test_new_outputs_of_ordinary_rows_keep_their_order(passed):
    x = torch.zeros(4, 8, 64, dtype=torch.bfloat16).transpose(0, 1)     # heads first
    out = qm.rope(x, torch.zeros(8, dtype=torch.int32), qm.Rope(torch.zeros(32, dtype=torch.float64)))
    assert out.stride() == x.stride()


def test_descriptions_keep_their_tensors(passed):
    """Calls read the addresses that were taken from the tensors: another tensor in a tensor's place would
    leave them on memory that was given back."""
    i32 = dict(dtype=torch.int32)
    plan = qm.Rope(torch.zeros(32, dtype=torch.float64))
    kv = qm.KvCache(*(torch.zeros(4, 16, 1, 64, dtype=torch.float8_e4m3fn) for _ in range(2)),
                    torch.ones(1), torch.ones(1))
    b = qm.KvBatch(torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1, 4, **i32), 1, 9)
    for of, names in ((plan, ("freq", "layout", "scale", "index", "struct")),
                      (kv, ("k", "v", "k_scale", "v_scale", "n_pages", "page_size", "n_heads", "D",
                            "index", "struct")),
                      (b, ("q_start", "seq_len", "page_table", "n_seq", "max_q", "max_len", "index"))):
        for name in names:
            before = getattr(of, name)
            with pytest.raises(AttributeError, match=name):
                setattr(of, name, before)
            with pytest.raises(AttributeError, match=name):
                delattr(of, name)
            assert getattr(of, name) is before
        of.note = "a caller's own"
        of.note = "again"
        assert of.note == "again"


# ---------------------------------------------------------------------- rows that are written

FAKE, OUT = 0x10000, 0x8000000        # never dereferenced


def _refused(status):
    assert status == 1
    return "overlap" in qm._lib.moe_last_error().decode()


@pytest.mark.parametrize("T,n", [(1, 1), (1, 5), (4, 1), (2, 3), (3, 2), (4, 5), (7, 3)])
def test_overlapping_outputs_are_refused(T, n):
    """Every pair of strides up to a few rows: refused where two rows share a place, and only there. (A
    call that is not refused for that is stopped by the next check, of missing positions.)"""
    D = 4
    plan = qm.RopeStruct(FAKE, 4, 0, 1.0)
    x = qm.HeadsStruct(FAKE, 64, 8)
    for token in range(0, 40):
        for head in range(0, 40):
            places = {t * token + h * head + d for t in range(T) for h in range(n) for d in range(D)}
            st = qm._lib.moe_rope(plan, x, 1, T, n, D, None, 0, qm.HeadsStruct(OUT, token, head), None)
            assert _refused(st) == (len(places) < T * n * D), (token, head)


def test_overlapping_outputs_of_other_calls():
    lib, D = qm._lib, 64
    rows = lambda p, *st: qm.HeadsStruct(p, *st)  # noqa: E731
    batch = qm.KvBatchStruct(2, 3, FAKE, FAKE, FAKE, 4, 4, 2, 9)

    def cache(k_head, v_head):
        return qm.KvCacheStruct(1, 4, 16, 2, D, FAKE, 2048, 128, k_head, FAKE, 2048, 128, v_head, None, None)

    def append(q_out, c=cache(64, 64)):
        q = None if q_out is None else rows(FAKE, 256, 64)
        return lib.moe_kv_append(c, batch, rows(FAKE, 0, 0), rows(FAKE, 0, 0), 1, None, FAKE + 2, q, 4,
                                 q_out, None, None)

    assert _refused(append(rows(OUT, 256, 32))) and _refused(append(rows(OUT, 192, 64)))
    assert _refused(append(rows(OUT, 0, 64)))
    assert _refused(append(None, cache(0, 64))) and _refused(append(None, cache(64, 48)))
    assert not _refused(append(rows(OUT, 256, 64))) and not _refused(append(rows(OUT, 64, 192)))

    def attend(out):
        return lib.moe_attend(cache(64, 0), batch, rows(FAKE, 0, 0), 1, 4, 1.0, 1, 0, 0, FAKE + 2, out, None,
                              0, None, None)

    assert _refused(attend(rows(OUT, 256, 0))) and _refused(attend(rows(OUT, 192, 64)))
    assert not _refused(attend(rows(OUT, 256, 64)))


def test_many_interleaved_rows_are_looked_through():
    """Rows of heads between rows of tokens, as many as a call takes."""
    plan, x = qm.RopeStruct(FAKE, 2, 0, 1.0), qm.HeadsStruct(FAKE, 64, 8)
    n = 1 << 15
    for token, head, meet in ((2 * n + 2, 2 * n, False), (6 * n + 3, 6 * n, False), (2 * n + 1, 2 * n, True),
                              (4 * n, 6 * n, True)):
        st = qm._lib.moe_rope(plan, x, 1, n, n, 2, None, 0, qm.HeadsStruct(OUT, token, head), None)
        assert _refused(st) == meet, (token, head)
