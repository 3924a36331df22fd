"""The 4-bit cache calls at the ends of what they accept, against the 8-bit calls over the same values, bit for bit."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_cache_q4 import SCALE, as_q8, choose, gen, make_cache, paged, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deepseek_sparse_attention_indexer_gb300 import _build, _lib
    _build.build()
    _lib.load()
    _lib.device_status(reset=True)
    yield _lib
    _lib.device_status(reset=True)


# ------------------------------------------------------------------------------------------------ workspaces

@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("rest", [0, 8])
def test_prefill_without_room_for_its_rows(dsa, rest, page):
    """A workspace of the size for N = 0 (nothing, where no query is cut): the same bits, and nothing behind it written."""
    g = gen(21 + rest)
    L, N, K = torch.cuda.get_device_properties(0).multi_processor_count + rest, 700, 640
    cache, scale = make_cache(g, N, exponents=1)
    q, idx = randn(g, L, 64, 576).bfloat16(), choose(g, [N] * L, N, K)
    small, full = dsa.attn_q4_workspace_size(L, K), dsa.attn_q4_workspace_size(L, K, N)
    assert full > small + 640 * N and (small > 0) == (rest > 0)
    ws = torch.full((small + 512,), 0xEE, dtype=torch.uint8, device="cuda")
    pool, pscale, table, _ = paged(g, cache[None], scale[None], [N], page or 16)

    def call(workspace):
        if page:
            return dsa.mla_sparse_attn_prefill_q4_paged(q, pool, pscale, table[0], page, idx, SCALE, N, want_lse=True, workspace=workspace)
        return dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE, want_lse=True, workspace=workspace)

    want = dsa.mla_sparse_attn_prefill_q8(q, as_q8(cache), scale, idx, SCALE, want_lse=True)
    for got in (call(None), call(ws[:small]), call(ws[16:16 + small]) if rest else call(ws[:0])):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((ws[small + 16:] == 0xEE).all()) and dsa.device_status() == 0
    for n in (1, small + 1, small + 512) + ((small - 1,) if rest else ()):   # neither size
        with pytest.raises(dsa.DsaError):
            call(ws[:n])


def test_key_weights_without_room_for_their_rows(dsa):
    g = gen(23)
    L, N, K, page = 320, 500, 450, 16
    cache, scale = make_cache(g, N)
    idx, q = choose(g, [N - 20] * L, N, K), randn(g, L, 64, 576).bfloat16()
    lse = dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE, want_lse=True)[1]
    small = dsa.key_weights_workspace_size(L, K, N)
    assert small == 8 * N and dsa.key_weights_workspace_size(L, K, N, 2) > small + 640 * N
    want = dsa.mla_key_weights_prefill(q, as_q8(cache), idx, lse, SCALE, cache_scale=scale)
    ws = torch.full((small + 512,), 0xEE, dtype=torch.uint8, device="cuda")
    assert torch.equal(dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale), want)
    assert torch.equal(dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale, workspace=ws[:small]), want)
    pool, pscale, table, _ = paged(g, cache[None], scale[None], [N], page)
    assert torch.equal(dsa.mla_key_weights_prefill(q, pool, idx, lse, SCALE, cache_scale=pscale, block_table=table[0], page_size=page,
                                                   N=N, workspace=ws[:small]), want)
    assert bool((ws[small:] == 0xEE).all()) and dsa.device_status() == 0
    for n in (small - 8, small + 8):
        with pytest.raises(dsa.DsaError):
            dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale, workspace=ws[:n])
