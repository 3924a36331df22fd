"""Refusals of the 8-bit cache calls and of the indexer's input pass: every bad argument is found on
the host, with its status code, before the device is touched (no GPU needed)."""
import math

import pytest

P = 4096          # a 16-byte aligned non-null address, never dereferenced
INVALID, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from deepseek_sparse_attention_indexer_gb300 import _build, _lib
    return _lib.load(_build.build())


def call(fn, names, good, **bad):
    """fn with the good arguments, some of them replaced."""
    assert set(bad) <= set(names)
    return fn(*[bad.get(n, g) for n, g in zip(names, good)])


def refusals(fn, names, good, table):
    for code, bads in table.items():
        for bad in bads:
            assert call(fn, names, good, **bad) == code, (bad, code)


WRITE = ("kv_a", "kv_a_stride", "norm_w", "eps", "cos_sin", "max_pos", "interleave", "pos", "slots", "R", "cache",
         "cache_scale", "cache_rows", "stream")
WRITE_OK = (P, 576, P, 1e-6, P, 4096, 1, P, P, 8, P, P, 1024, None)


def test_write_refusals(lib):
    refusals(lib.mla_cache_write_q8, WRITE, WRITE_OK, {
        INVALID: [{n: None} for n in ("kv_a", "norm_w", "cos_sin", "pos", "slots", "cache", "cache_scale")]
        + [{"R": 0}, {"R": -1}, {"max_pos": 0}, {"cache_rows": 0}, {"kv_a_stride": 568}, {"eps": -1e-6},
           {"eps": math.inf}, {"eps": math.nan}, {"interleave": 2}, {"interleave": -1}],
        SHAPE: [{"cache_rows": 1 << 31}],
        ALIGN: [{"kv_a": P + 2}, {"norm_w": P + 4}, {"cos_sin": P + 8}, {"cache": P + 16}, {"kv_a_stride": 580}],
    })


def test_read_refusals(lib):
    names = ("cache", "cache_scale", "cache_rows", "slots", "R", "out", "stream")
    refusals(lib.mla_cache_read_q8, names, (P, P, 1024, P, 8, P, None), {
        INVALID: [{n: None} for n in ("cache", "cache_scale", "slots", "out")] + [{"R": 0}, {"cache_rows": 0}],
        SHAPE: [{"cache_rows": 1 << 31}],
        ALIGN: [{"cache": P + 16}, {"out": P + 2}],
    })
    names = ("cache", "cache_scale", "kv_len", "block_table", "bt_stride", "page_size", "num_pages", "B", "Nmax", "out",
             "stream")
    refusals(lib.mla_cache_read_q8_paged, names, (P, P, P, P, 4, 64, 8, 2, 256, P, None), {
        INVALID: [{n: None} for n in ("cache", "cache_scale", "kv_len", "block_table", "out")]
        + [{"B": 0}, {"Nmax": 0}, {"Nmax": 257}, {"bt_stride": 0}, {"num_pages": 0}],
        SHAPE: [{"page_size": 8}, {"page_size": 48}, {"page_size": 1 << 17}, {"num_pages": 1 << 25},
                {"B": 1 << 24, "Nmax": 256}, {"B": 1 << 30}],
        ALIGN: [{"cache": P + 16}, {"out": P + 2}],
    })


ATTN_BAD = {
    INVALID: [{n: None} for n in ("q", "cache", "cache_scale", "idx", "out")]
    + [{"rows": 0}, {"N": 0}, {"scale": 0.0}, {"scale": -1.0}, {"scale": math.nan}, {"scale": math.inf},
       {"out_dtype": 2}, {"out_dtype": -1}],
    SHAPE: [{"top_k": 0}, {"top_k": 2049}, {"rows": 1 << 26}],
    ALIGN: [{"q": P + 2}, {"cache": P + 16}, {"out": P + 4}],
}


def test_prefill_refusals(lib):
    names = ("q", "cache", "cache_scale", "idx", "rows", "N", "top_k", "scale", "out", "out_dtype", "lse", "ws", "bytes",
             "stream")
    refusals(lib.mla_sparse_attn_prefill_q8, names, (P, P, P, P, 4, 256, 64, 0.0625, P, 0, None, None, 0, None), ATTN_BAD)
    names = ("q", "cache", "cache_scale", "table", "page", "pages", "idx", "rows", "N", "top_k", "scale", "out",
             "out_dtype", "lse", "ws", "bytes", "stream")
    good = (P, P, P, P, 64, 8, P, 4, 256, 64, 0.0625, P, 0, None, None, 0, None)
    refusals(lib.mla_sparse_attn_prefill_q8_paged, names, good, ATTN_BAD)
    refusals(lib.mla_sparse_attn_prefill_q8_paged, names, good,
             {INVALID: [{"table": None}, {"pages": 0}, {"page": 0}], SHAPE: [{"page": 48}, {"page": 8}, {"pages": 1 << 26}]})


def test_decode_refusals(lib):
    names = ("q", "cache", "cache_scale", "kv_len", "idx", "rows", "N", "top_k", "scale", "out", "out_dtype", "lse", "ws",
             "bytes", "stream")
    good = (P, P, P, P, P, 4, 256, 64, 0.0625, P, 0, None, P, 1 << 24, None)
    more = {INVALID: [{"kv_len": None}], ALIGN: [{"ws": P + 8}]}
    refusals(lib.mla_sparse_attn_decode_q8, names, good, ATTN_BAD)
    refusals(lib.mla_sparse_attn_decode_q8, names, good, more)
    refusals(lib.mla_sparse_attn_decode_q8, names, good, {SHAPE: [{"rows": 1 << 20, "N": 1 << 12}]})
    names = ("q", "cache", "cache_scale", "kv_len", "table", "stride", "page", "pages", "idx", "rows", "N", "top_k",
             "scale", "out", "out_dtype", "lse", "ws", "bytes", "stream")
    good = (P, P, P, P, P, 4, 64, 8, P, 4, 256, 64, 0.0625, P, 0, None, P, 1 << 24, None)
    refusals(lib.mla_sparse_attn_decode_q8_paged, names, good, ATTN_BAD)
    refusals(lib.mla_sparse_attn_decode_q8_paged, names, good, more)
    refusals(lib.mla_sparse_attn_decode_q8_paged, names, good,
             {INVALID: [{"table": None}, {"stride": 0}, {"N": 257}, {"pages": 0}], SHAPE: [{"page": 100}]})
    for B, top_k in ((0, 64), (-1, 64), (4, 0), (4, 2049)):
        assert lib.mla_sparse_attn_q8_workspace_size(B, top_k) == 0


def test_norm_rope_refusals(lib):
    names = ("q", "q_stride", "k", "k_stride", "norm", "q_w", "q_b", "k_w", "k_b", "eps", "cos_sin", "max_pos",
             "interleave", "pos", "slots", "R", "q_out", "k_cache", "cache_rows", "stream")
    good = (P, 4096, P, 128, 1, None, None, P, P, 1e-6, P, 4096, 1, P, P, 8, 2 * P, P, 1024, None)
    refusals(lib.dsa_indexer_norm_rope, names, good, {
        INVALID: [{n: None} for n in ("q", "k", "cos_sin", "pos", "slots", "q_out", "k_cache")]
        + [{"q_b": P}, {"k_w": None}, {"R": 0}, {"max_pos": 0}, {"cache_rows": 0}, {"q_stride": 4088}, {"k_stride": 120},
           {"eps": -1.0}, {"eps": math.nan}, {"norm": 2}, {"norm": -1}, {"interleave": 3},
           {"q_out": P, "q_stride": 8192}],
        SHAPE: [{"cache_rows": 1 << 31}, {"R": 1 << 27}],
        ALIGN: [{"q": P + 2}, {"k": P + 2}, {"cos_sin": P + 4}, {"q_out": P + 2}, {"k_cache": P + 8}, {"k_w": P + 4},
                {"k_b": P + 4}, {"q_w": P + 4}, {"q_w": P, "q_b": P + 4}, {"q_stride": 4100}, {"k_stride": 132}],
    })
