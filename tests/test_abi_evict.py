"""Refusals of the eviction calls: every bad argument is found on the host, with its status code, before the device is
touched (no GPU needed)."""
import ctypes
import math

import pytest

P = 4096          # a 16-byte aligned non-null address, never dereferenced
INVALID, SHAPE, ALIGN, SMALL = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from deepseek_sparse_attention_indexer_gb300 import _build, _lib
    return _lib.load(_build.build())


def refusals(fn, names, good, table):
    for code, bads in table.items():
        for bad in bads:
            assert set(bad) <= set(names)
            assert fn(*[bad.get(n, g) for n, g in zip(names, good)]) == code, (bad, code)


WEIGHTS_BAD = {
    INVALID: [{n: None} for n in ("q", "cache", "idx", "lse", "acc")]
    + [{"rows": 0}, {"N": 0}, {"scale": 0.0}, {"scale": -1.0}, {"scale": math.nan}, {"scale": math.inf}, {"format": 3},
       {"format": -1}, {"format": 0, "scales": P}, {"format": 1, "scales": None}, {"format": 2, "scales": None},
       {"accumulate": 2}, {"accumulate": -1}],
    SHAPE: [{"top_k": 0}, {"top_k": 2049}, {"rows": 1 << 26}, {"page": 48}, {"page": 8}, {"pages": 1 << 26}],
    ALIGN: [{"q": P + 2}, {"cache": P + 16}],
}


def test_key_weights_prefill_refusals(lib):
    names = ("q", "cache", "scales", "format", "table", "page", "pages", "idx", "lse", "rows", "N", "top_k", "scale", "acc",
             "accumulate", "ws", "bytes", "stream")
    good = (P, P, P, 2, P, 64, 8, P, P, 4, 256, 64, 0.0625, P, 0, P, 1 << 20, None)
    refusals(lib.mla_key_weights_prefill, names, good, WEIGHTS_BAD)
    refusals(lib.mla_key_weights_prefill, names, good,
             {INVALID: [{"ws": None}, {"pages": 0}], ALIGN: [{"ws": P + 16}], SMALL: [{"bytes": 256 * 8 - 1}]})
    size = lib.mla_key_weights_workspace_size
    assert size(2, 4, 256, 64) == size(0, 4096, 256, 64) == size(1, 4096, 256, 64) == 2048
    assert size(2, 4096, 256, 64) >= 256 * (8 + 640 + 4)                  # the rows expanded
    assert size(3, 4, 256, 64) == size(-1, 4, 256, 64) == size(0, 0, 256, 64) == size(0, 4, 0, 64) == size(0, 4, 256, 2049) == 0


def test_key_weights_decode_refusals(lib):
    names = ("q", "cache", "scales", "format", "kv_len", "table", "stride", "page", "pages", "idx", "lse", "rows", "N", "top_k",
             "scale", "acc", "accumulate", "stream")
    good = (P, P, P, 1, P, P, 4, 64, 8, P, P, 4, 256, 64, 0.0625, P, 1, None)
    refusals(lib.mla_key_weights_decode, names, good, WEIGHTS_BAD)
    refusals(lib.mla_key_weights_decode, names, good,
             {INVALID: [{"kv_len": None}, {"stride": 0}, {"N": 257}],
              SHAPE: [{"rows": 1 << 20, "N": 1 << 12, "table": None}]})


def test_evict_plan_refusals(lib):
    names = ("acc", "pos", "kv_len", "B", "Nmax", "keep", "recent", "sink", "src", "dst", "left", "stream")
    good = (P, P, P, 4, 256, 100, 50, 50, P, 2 * P, P, None)
    refusals(lib.dsa_cache_evict_plan, names, good, {
        INVALID: [{n: None} for n in ("acc", "pos", "kv_len", "src", "dst", "left")]
        + [{"dst": P}, {"B": 0}, {"Nmax": 1}, {"keep": 0}, {"keep": 256}, {"recent": -1}, {"sink": -1}, {"recent": 51},
           {"recent": (1 << 31) - 1, "sink": (1 << 31) - 1}],
        SHAPE: [{"B": 1 << 24}, {"B": 1 << 28, "Nmax": 2, "keep": 1, "recent": 0, "sink": 0}],
    })


def test_move_rows_refusals(lib):
    def call(ptrs=(P, P), sizes=(4, 1152), kinds=(0, 1), **bad):
        n = bad.pop("count", len(ptrs))
        a = dict(src=P, dst=P, B=2, moves=4, Nmax=64, count=n, tensors=(ctypes.c_void_p * len(ptrs))(*ptrs),
                 row_bytes=(ctypes.c_int * len(sizes))(*sizes), paged=(ctypes.c_int * len(kinds))(*kinds), table=P, stride=4,
                 page=16, pages=8, stream=None)
        a.update(bad)
        return lib.dsa_cache_move_rows(*a.values())

    for bad in ({"src": None}, {"dst": None}, {"tensors": None}, {"row_bytes": None}, {"paged": None}, {"B": 0}, {"moves": 0},
                {"Nmax": 0}, {"count": 0}, {"table": None}, {"Nmax": 65}, {"stride": 0}, {"pages": 0}, {"ptrs": (P, 0)},
                {"sizes": (4, 0)}, {"sizes": (-4, 4)}, {"kinds": (0, 2)}):
        assert call(**bad) == INVALID, bad
    for bad in ({"B": 65536}, {"page": 24}, {"moves": 1 << 30}, {"Nmax": 1 << 30, "page": 65536, "stride": 1 << 14, "pages": 1 << 15},
                {"ptrs": (P,) * 9, "sizes": (4,) * 9, "kinds": (0,) * 9}, {"sizes": (4, (1 << 20) + 4)},
                {"sizes": ((1 << 31) - 4, 4)}):
        assert call(**bad) == SHAPE, bad
    for bad in ({"sizes": (4, 6)}, {"ptrs": (P + 2, P)}):
        assert call(**bad) == ALIGN, bad
