"""The attention over the 8-bit latent cache at both ends of its scales' range, with rows of zeros and with queries that
hold NaN, under the tightest bound its number formats allow.

Tolerances, from the arithmetic:

* attention, per element: a weight w_t = p_t c_t (probability times the row's scale) enters the value product as
  hi + lo / 16 in e4m3, from a half-precision number: a relative error of at most 2^-9 + 2^-11 < 2^-8 where lo is not
  among e4m3's smallest numbers, and at most half of lo's last step, 2^-10 / 16 = 2^-14, elsewhere, beside a head's
  largest weight of at least 2^4.5.  So |out - ref| <= 2^-8 sum_t w_t |code_t| + 2^-18.5 max_t w_t sum_t |code_t|, with the
  maximum over rows that hold a code other than 0 (the others add nothing).  The half-precision number and the
  exponential before it add 2^-10 of either part; the float32 logits (576 products and their sum, the scale, the
  exponent) and sums at most 2^-12 of the first.  Where a logit's terms sum to S in absolute value, S in the hundreds,
  (e^(2 d) - 1) of the first part more, d = 576 * 2^-24 S.  A bf16 output adds 2^-8 |ref|.
* lse: 2^-12 absolute for logits of a few tens, d more for large ones.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_cache_q8 import F8, SCALE, angles, choose, gen, make_cache, paged, randn, values  # noqa: E402


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


# ------------------------------------------------------------------------------------------------ attention

def attention64(q, cache, scale, idx, sm=SCALE):
    """(out, lse, sum_t w_t |code_t|, floor): one cache for all queries, in float64 on the tensors' device."""
    have = idx >= 0
    at = idx.clamp(min=0).long()
    kv = values(cache, scale)
    code = cache[..., :512].contiguous().view(F8).double()
    out, lse, A, low = [], [], [], []
    for i in range(idx.shape[0]):
        ok, rows, c = have[i], kv[at[i]], code[at[i]]
        x = (q[i].double() @ rows.t() * sm).masked_fill(~ok[None], -math.inf)
        p = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
        w = p * scale[at[i]].double()
        out.append(p @ rows[:, :512])
        lse.append(torch.logsumexp(x, -1))
        A.append(w @ c.abs())
        used = ok & (c != 0).any(1)
        top = (w * used).amax(1, keepdim=True)
        low.append(top * (c.abs() * ok[:, None]).sum(0, keepdim=True))
    return tuple(torch.stack(t) for t in (out, lse, A, low))


def bound(ref, S=0.0, dtype=torch.float32):
    out, _, A, low = ref
    d = 576 * 2.0 ** -24 * S
    b = ((2.0 ** -8 + 2.0 ** -12 + math.expm1(2 * d)) * A + 2.0 ** -18.5 * low) * (1 + 2.0 ** -10)
    return b + 2.0 ** -8 * out.abs() if dtype == torch.bfloat16 else b


def close(out, lse, ref, S=0.0):
    err, b = (out.double() - ref[0]).abs(), bound(ref, S, out.dtype)
    assert bool((err <= b).all()), float((err / b.clamp(min=1e-300)).nan_to_num(nan=math.inf).max())
    dead = torch.isneginf(ref[1])
    assert torch.equal(torch.isneginf(lse), dead)
    assert bool(((lse.double() - ref[1]).abs()[~dead] <= 2.0 ** -12 + 576 * 2.0 ** -24 * S).all())


def both_ways(dsa, q, cache, scale, idx, sm=SCALE, S=0.0):
    """The few queries (whose keys may be cut into parts) and as many as SMs (whole queries, tile after tile)."""
    ref = attention64(q, cache, scale, idx, sm)
    many = torch.arange(torch.cuda.get_device_properties(0).multi_processor_count, device="cuda") % idx.shape[0]
    out = lse = None
    for rows in (many, many[:idx.shape[0]]):
        out, lse = dsa.mla_sparse_attn_prefill_q8(q[rows].contiguous(), cache, scale, idx[rows].contiguous(), sm, want_lse=True)
        assert dsa.device_status() == 0
        close(out, lse, tuple(t[rows] for t in ref), S)
        o16 = dsa.mla_sparse_attn_prefill_q8(q[rows].contiguous(), cache, scale, idx[rows].contiguous(), sm,
                                             out_dtype=torch.bfloat16)
        assert torch.equal(o16, out.bfloat16())
    return out, lse, ref


@pytest.mark.gpu
@pytest.mark.parametrize("small,large", [(-64, 64), (-64, 50), (-60, 60), (-30, 64), (-64, -20), (-20, 64)])
def test_equal_scores_at_both_ends_of_the_scales(dsa, small, large):
    """Keys of equal score whose scales lie as far apart as they may: each has its part of the softmax's sum, whether
    the tile of large scales comes last, first, or is the same tile."""
    g = gen(32)
    N, n = 320, 128
    cache, _ = make_cache(g, N)
    cache[:, 512:] = 0
    q = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda")
    idx = torch.arange(N, dtype=torch.int32, device="cuda")
    some = torch.zeros(N, dtype=torch.bool, device="cuda")
    some[n:n + 1] = True                                                  # one key behind a whole tile of others
    half = torch.arange(N, device="cuda") < n
    mixed = torch.arange(N, device="cuda") % 3 == 1
    for big in (some, half, ~half, mixed):
        scale = torch.where(big, 2.0 ** large, 2.0 ** small).float()
        for order in (idx, idx.flip(0)):
            for k in (129, N):
                both_ways(dsa, q, cache, scale, order[None, :k].contiguous())


@pytest.mark.gpu
def test_scores_against_scales(dsa):
    """Scores that make up for the scales, fall with them, or have nothing to do with them, over the scales' whole range;
    references that move by more than 126 in one tile."""
    g = gen(33)
    N = 700
    cache, _ = make_cache(g, N)
    k = torch.randint(-64, 65, (N,), generator=g, device="cuda")
    idx = torch.randperm(N, generator=g, device="cuda")[:600].int()[None].repeat(4, 1).contiguous()
    idx[1] = idx[1][k[idx[1].long()].argsort()]                           # smallest scales first
    idx[2] = idx[1].flip(0)
    rope = torch.zeros(N, 64, device="cuda")
    rope[:, 0] = k.float()
    rope[:, 1:] = 0.5 * randn(g, N, 63)
    cache[:, 512:] = rope.bfloat16().view(torch.uint8)
    q = torch.zeros(4, 64, 576, device="cuda")
    q[:, :, 512] = torch.linspace(-16 * math.log(2.0), 16 * math.log(2.0), 64, device="cuda")[None]   # scores ln 2 [-k, k]
    q[:, :, 513:] = randn(g, 4, 64, 63)
    q[3, :, 512] = 0.0
    q[3, ::2, 512] = 100.0                                                # scores of -400 .. 400
    S = float((q[:, :, 512:].abs() @ rope.abs().t()).max()) * SCALE
    both_ways(dsa, q.bfloat16(), cache, torch.exp2(k.float()), idx, S=S)


@pytest.mark.gpu
@pytest.mark.parametrize("c", [-6, -11, -27, -60])
def test_rows_of_zeros_take_no_range(dsa, c):
    """A row of zeros is written with scale 1; among rows of small scale it adds its part of the sum and nothing else.
    A row that only begins with zeros is one like the others."""
    g = gen(34)
    N = 400
    cache, scale = make_cache(g, N)
    scale = torch.full((N,), 2.0 ** c, device="cuda")
    zero = torch.zeros(1, 576, dtype=torch.bfloat16, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    for at in (3, 130, 399):
        dsa.mla_cache_write_q8(zero, torch.ones(512, device="cuda"), 1e-6, angles(1), one, one + at, cache, scale)
        assert float(scale[at]) == 1.0
    cache[130, :512] = 0x80                                               # zeros of either sign
    cache[200, :512], cache[200, 1:512:2], scale[200] = 0, 0x80, 1.0
    cache[5, :480], cache[6, :4], cache[7, 4:512] = 0, 0, 0               # part of the row alone
    q = (0.5 * randn(g, 2, 64, 576)).bfloat16()
    idx = torch.arange(N, dtype=torch.int32, device="cuda").repeat(2, 1)
    idx[1] = idx[1].flip(0)
    both_ways(dsa, q, cache, scale, idx)
    only = torch.tensor([[3, 130, 200]], dtype=torch.int32, device="cuda")
    out, _, _ = both_ways(dsa, q[:1].contiguous(), cache, scale, only)
    assert bool((out == 0).all())


@pytest.mark.gpu
def test_pages_outside_the_pool_take_no_range(dsa):
    """Keys of a page outside the pool read as zeros beside rows of small scale."""
    g = gen(35)
    N, page = 300, 64
    cache, _ = make_cache(g, N)
    scale = torch.full((N,), 2.0 ** -27, device="cuda")
    q = (0.5 * randn(g, 1, 64, 576)).bfloat16()
    idx = torch.arange(N, dtype=torch.int32, device="cuda")[None].contiguous()
    pool, pscale, table, pages = paged(g, cache[None], scale[None], [N], page)
    table[0, 1] = pages
    out, lse = dsa.mla_sparse_attn_decode_q8_paged(q, pool, pscale, torch.tensor([N], dtype=torch.int32, device="cuda"), table,
                                                   page, idx, SCALE, N, want_lse=True)
    assert dsa.device_status() == 7
    cache[page:2 * page] = 0
    close(out, lse, attention64(q, cache, scale, idx))


@pytest.mark.gpu
@pytest.mark.parametrize("where", [0, 100, 511, 512, 575])
def test_nan_query_heads(dsa, where):
    """A NaN in a query makes its head's output and lse NaN, the same in a cut query, a whole one and a decode step, and
    changes no other head."""
    g = gen(36)
    N, K = 700, 600
    cache, scale = make_cache(g, N)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    idx = choose(g, [N] * 2, N, K)
    q = randn(g, 2, 64, 576).bfloat16()
    bad = q.clone()
    heads = torch.tensor([0, 17, 18, 63], device="cuda")
    bad[1, heads, where] = math.nan
    rest = torch.ones(2, 64, dtype=torch.bool, device="cuda")
    rest[1, heads] = False
    many = torch.arange(sms, device="cuda") % 2
    for rows in (torch.arange(2, device="cuda"), many):
        assert (dsa.attn_q8_workspace_size(len(rows), K) > 0) == (len(rows) == 2)
        i = idx[rows].contiguous()
        cs = cache[None].expand(len(rows), -1, -1).contiguous(), scale[None].expand(len(rows), -1).contiguous()
        kv_len = torch.full((len(rows),), N, dtype=torch.int32, device="cuda")
        for call in (lambda x: dsa.mla_sparse_attn_prefill_q8(x, cache, scale, i, SCALE, want_lse=True),
                     lambda x: dsa.mla_sparse_attn_decode_q8(x, *cs, kv_len, i, SCALE, want_lse=True)):
            good, glse = call(q[rows].contiguous())
            out, lse = call(bad[rows].contiguous())
            keep = rest[rows]
            assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], glse[keep])
            assert bool(out[~keep].isnan().all()) and bool(lse[~keep].isnan().all())
    assert dsa.device_status() == 0
