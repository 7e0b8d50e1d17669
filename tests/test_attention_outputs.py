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
