"""The 4-bit cache calls at the ends of what they accept, against the 8-bit calls over the same values, bit for bit."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_cache_q4 import SCALE, angles, as_q8, attention64, choose, close, gen, i32, make_cache, paged, randn, values  # noqa: E402

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


# ------------------------------------------------------------------------------------------------ write

def test_write_of_tokens_that_are_not_finite(dsa):
    """NaN and infinite latent dims leave finite numbers in their token's row (the 8-bit row holds NaN), and no other row."""
    g = gen(26)
    R = 12
    kv_a, w, cs, at = randn(g, R, 576).bfloat16(), torch.exp(0.3 * randn(g, 512)), angles(R), torch.arange(R, device="cuda").int()
    bad = kv_a.clone()
    bad[2, 7], bad[5, 500], bad[8, :512], bad[9, 30:60] = float("nan"), float("inf"), float("nan"), -float("inf")
    odd = torch.zeros(R, dtype=torch.bool, device="cuda")
    odd[[2, 5, 8, 9]] = True
    rows = []
    for x in (kv_a, bad):
        cache, scale = torch.full((R, 416), 0xEE, dtype=torch.uint8, device="cuda"), torch.zeros(R, device="cuda")
        dsa.mla_cache_write_q4(x, w, 1e-6, cs, at, at, cache, scale)
        rows.append((cache, scale))
        assert bool(torch.isfinite(dsa.mla_cache_read_q4(cache, scale, at).float()).all()) and bool(torch.isfinite(scale).all())
    for x, y in zip(*rows):
        assert torch.equal(x[~odd], y[~odd])
    eight, scale = torch.zeros(R, 640, dtype=torch.uint8, device="cuda"), torch.zeros(R, device="cuda")
    dsa.mla_cache_write_q8(bad, w, 1e-6, cs, at, at, eight, scale)
    assert torch.equal(torch.isnan(dsa.mla_cache_read_q8(eight, scale, at).float()).any(1), odd)
    assert dsa.device_status() == 0


# ------------------------------------------------------------------------------------------------ many queries a CTA

def short_selections(g, rows, N, K, every):
    """Selections of none to K keys, -1 behind; every `every`-th at most a tile."""
    many = torch.randint(0, K + 1, (rows, 1), generator=g, device="cuda")
    many[::every] = many[::every] % 129
    return choose(g, [N] * rows, N, K).masked_fill(torch.arange(K, device="cuda") >= many, -1)


@pytest.mark.parametrize("direct", [True, False])
def test_prefill_of_many_queries(dsa, direct):
    """Five queries a CTA of none to three tiles, over the rows as they are and over expanded ones; both types of the output."""
    g = gen(24)
    L, N, K = 740, 900, 300
    cache, scale = make_cache(g, N, exponents=2)
    q, idx = randn(g, L, 64, 576).bfloat16(), short_selections(g, L, N, K, 3)
    size = dsa.attn_q4_workspace_size(L, K, 0 if direct else N)
    assert dsa.attn_q4_workspace_size(L, K, N) >= dsa.attn_q4_workspace_size(L, K) + 644 * N
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out, lse = dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE, want_lse=True, workspace=ws)
    kv = values(cache, scale)
    close(out, lse, attention64(q, lambda s: kv[idx[s].clamp(min=0).long()], idx >= 0, SCALE))
    twin = dsa.mla_sparse_attn_prefill_q8(q, as_q8(cache), scale, idx, SCALE, want_lse=True)
    assert torch.equal(out, twin[0]) and torch.equal(lse, twin[1])
    for _ in range(20):
        o16, l16 = dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE, want_lse=True, workspace=ws, out_dtype=torch.bfloat16)
        assert torch.equal(o16, out.bfloat16()) and torch.equal(l16, lse)   # the float32 result, rounded
    assert dsa.device_status() == 0


def test_decode_of_many_sequences(dsa):
    """Five sequences a CTA, every length from none on."""
    g = gen(25)
    B, N, K = 740, 310, 300
    cache, scale = make_cache(g, B * N, exponents=1)
    cache, scale = cache.view(B, N, 416), scale.view(B, N)
    lens = [(b * 7919) % (N + 1) for b in range(B)]
    idx, q, kv_len = choose(g, lens, N, K), randn(g, B, 64, 576).bfloat16(), i32(*lens)
    out, lse = dsa.mla_sparse_attn_decode_q4(q, cache, scale, kv_len, idx, SCALE, want_lse=True)
    kv = values(cache, scale)
    close(out, lse, attention64(q, lambda s: torch.stack([kv[b][idx[b].clamp(min=0).long()] for b in range(B)[s]]), idx >= 0, SCALE))
    twin = dsa.mla_sparse_attn_decode_q8(q, as_q8(cache), scale, kv_len, idx, SCALE, want_lse=True)
    assert torch.equal(out, twin[0]) and torch.equal(lse, twin[1])
    for _ in range(20):
        o16, l16 = dsa.mla_sparse_attn_decode_q4(q, cache, scale, kv_len, idx, SCALE, want_lse=True, out_dtype=torch.bfloat16)
        assert torch.equal(o16, out.bfloat16()) and torch.equal(l16, lse)
    assert dsa.device_status() == 0
