"""How much scratch memory attention asks for, on the host, without a GPU."""
import itertools

import pytest

pytest.importorskip("torch")
import quantized_routed_expert_gemv_amd as qm  # noqa: E402

lib = qm._lib
FAKE = 0x10000        # never dereferenced
BF = 1


def need(new, keys, Hkv, G, D, page=16, hints=True, window=0):
    cache = qm.KvCacheStruct(BF, 1 << 14, page, Hkv, D, FAKE, Hkv * D * page, Hkv * D, D, FAKE,
                             Hkv * D * page, Hkv * D, D, None, None)
    batch = qm.KvBatchStruct(len(new), sum(new), FAKE, FAKE, FAKE, -(-keys // page), -(-keys // page),
                             max(new) if hints else 0, keys if hints else 0)
    return lib.moe_attend_scratch_bytes(cache, batch, Hkv * G, window, 0)


# Sums and statistics of a row of a split: D + 2 floats.
# Splits of the sequences with few rows: at most 1024 places of up to 32 rows. Of those with many: at
# most 1024 tiles of 128 rows.
def few_limit(D):
    return 1024 * 32 * (D + 2) * 4


def many_limit(D):
    return 1024 * 128 * (D + 2) * 4


@pytest.mark.parametrize("hints", [True, False])
@pytest.mark.parametrize("new,keys,Hkv,G,D", [([8192, 1], 32768, 8, 4, 128), ([8192, 1], 131072, 4, 8, 128),
                                              ([8192, 1], 16384, 4, 8, 128), ([8192, 1], 131072, 8, 8, 128),
                                              ([16384, 1], 131072, 1, 64, 128), ([8192, 1], 131072, 1, 32, 128),
                                              ([16384, 1], 131072, 1, 128, 256),
                                              ([512, 1] * 8, 8704, 4, 8, 128),
                                              ([8192] + [1] * 63, 131072, 8, 1, 64)])
def test_tokens_beside_a_chunk(new, keys, Hkv, G, D, hints):
    """Only the sequences with few rows are split beside a long chunk, and only their rows need room."""
    assert need(new, keys, Hkv, G, D, hints=hints) <= few_limit(D)


def test_whole_range():
    for new, keys, Hkv, G, D, hints in itertools.product(
            ([1], [5], [33], [700], [20000], [1] * 300, [4, 1], [40, 1], [300, 1, 1], [5000, 2],
             [70, 60, 50, 1], [100000, 1, 900]), (1, 300, 9000, 200000), (1, 2, 8, 12),
            (1, 3, 8, 16, 32, 33, 128), (64, 128, 256), (True, False)):
        got = need(new, max(keys, *new), Hkv, G, D, hints=hints)
        assert got <= few_limit(D) + many_limit(D), (new[:4], keys, Hkv, G, D, hints)


@pytest.mark.parametrize("G", [33, 64, 128])
def test_groups_of_more_than_few_rows(G):
    """Then no sequence has few rows, and beside a chunk whose tiles fill the launch nothing is split."""
    for new in ([16384, 1], [16384, 3, 700]):
        assert need(new, 131072, 1, 32, 128) > 0
        assert need(new, 131072, 1, G, 128) == 0
