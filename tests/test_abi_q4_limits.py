"""Workspaces of the 4-bit prefill: what is refused on the host, and what is not (no GPU needed)."""
import pytest

P = 4096          # a 32-byte aligned non-null address, never dereferenced
ALIGN = 3


@pytest.fixture(scope="module")
def lib():
    from deepseek_sparse_attention_indexer_gb300 import _build, _lib
    return _lib.load(_build.build())


@pytest.fixture(scope="module")
def no_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("calls that pass the checks of their arguments would launch")


def prefill(lib, rows, top_k, N, ws, size, q=P):
    return lib.mla_sparse_attn_prefill_q4(q, P, P, P, rows, N, top_k, 0.0625, P, 0, None, ws, size, None)


def prefill_paged(lib, rows, top_k, N, ws, size, q=P):
    return lib.mla_sparse_attn_prefill_q4_paged(q, P, P, P, 64, 64, P, rows, N, top_k, 0.0625, P, 0, None, ws, size, None)


@pytest.mark.parametrize("call", [prefill, prefill_paged])
def test_alignment_of_the_workspace(lib, no_gpu, call):
    """16 bytes, as for the 8-bit cache; 32 where the rows are expanded there."""
    direct, expanded = (4, 2048, 2048), (64, 2048, 2048)
    assert call(lib, *direct, P + 8, 1 << 24) == ALIGN and call(lib, *expanded, P + 8, 1 << 24) == ALIGN
    assert call(lib, *expanded, P + 16, 1 << 24) == ALIGN
    past = call(lib, *direct, P, 1 << 24)                                 # the device's turn: there is none
    assert past > ALIGN and call(lib, *direct, P + 16, 1 << 24) == past
    assert call(lib, *expanded, P + 32, 1 << 24) == past
