"""The ends of what the 8-bit latent cache calls accept: rows of any size, scales at both ends of their range, rows of
zeros, queries that hold NaN; and the attention under the tightest bound its number formats allow.

Tolerances, from the arithmetic:

* codes and scales of the write: exact, but for values within 2^-40 (relative) of a midpoint or of the scale's border,
  as the latent dims are computed to about 2^-44.
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


# ------------------------------------------------------------------------------------------------ write

def check_nearest(kv_a, w, eps, codes, scale):
    """Codes and scales are the formula's in float64; a row of zeros has codes 0 and scale 1."""
    x, got = kv_a[:, :512].double(), codes.double()
    u = torch.nan_to_num(x / torch.sqrt((x * x).mean(1, keepdim=True) + eps)) * w.double()   # 0 / 0: a row of zeros
    big = u.abs().amax(1)
    assert bool(((big < 2.0 ** -152) | (big > 2.0 ** -148)).all())
    zero = big < 2.0 ** -152                                              # below float32's smallest step
    assert bool((got[zero] == 0).all()) and bool((scale[zero] == 1).all())
    u, big, got, sc = u[~zero], big[~zero], got[~zero], scale[~zero].double()
    assert torch.equal(sc, torch.exp2(torch.ceil(torch.log2(big / 448.0)).clamp(-64, 64)))
    border = torch.log2(big / 448.0)
    assert bool(((border - border.round()).abs() > 2.0 ** -40).all())     # the data stay clear of it
    v = (u / sc[:, None]).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    near = ((v / step).frac().abs() - 0.5).abs() * step <= 2.0 ** -40 * v.abs()
    assert bool(((got == torch.round(v / step) * step) | near).all()) and int(near.sum()) < 10


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30, 1e-6, 1.0, 1e30, 2.9e38])
def test_write_rows_of_any_size(dsa, eps):
    """Rows from bf16's smallest numbers to its largest, alone and next to one outlier, and a row of zeros: squares and
    1 / sqrt leave float32's range at both ends, the quotient does not."""
    g = gen(31)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    amp = [0.0] + [2.0 ** e for e in (-131, -126, -100, -84, -64, -50, -41, -39, 0, 39, 41, 59, 61, 64, 90, 120, 125)]
    R = len(amp)
    kv_a = (randn(g, R, 576).clamp(-3.9, 3.9) * torch.tensor(amp, device="cuda")[:, None]).bfloat16()
    outlier = torch.randn(3, 576, generator=g, device="cuda").bfloat16()
    outlier[0, 100], outlier[1, 511], outlier[2] = 3e38, -1e25, outlier[2] * 1e-30
    outlier[2, 7] = 1e-3
    kv_a = torch.cat([kv_a, outlier])
    kv_a[:, 512:] = 1.0
    R += 3
    w = torch.exp(0.3 * randn(g, 512))
    slots, zero = torch.arange(R, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    cache, scale = torch.full((R, 640), 0x55, dtype=torch.uint8, device="cuda"), torch.full((R,), 7.0, device="cuda")
    dsa.mla_cache_write_q8(kv_a, w, eps, angles(1), zero, slots, cache, scale)
    assert dsa.device_status() == 0
    check_nearest(kv_a, w, eps, cache[:, :512].contiguous().view(F8), scale)


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
    many = torch.rand(N, generator=g, device="cuda") < 0.5                # half of the rows, one tile of nothing else
    many[128:256] = True
    many[300] = False
    cache[many, :512], scale[many] = 0, 1.0
    scale[300] = 1.0 if c < -20 else scale[300]                           # scale 1 and no zeros
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


# ------------------------------------------------------------------------------------------------ the bound

def cpu_cache(g, rows, k):
    cache = torch.empty(rows, 640, dtype=torch.uint8)
    cache[:, :512] = (torch.randn(rows, 512, generator=g) * 64.0).to(F8).view(torch.uint8)
    cache[:, 512:] = torch.randn(rows, 64, generator=g).bfloat16().view(torch.uint8)
    return cache, torch.exp2(k)


def far_apart(g):
    """Scales of 2^-40 .. 2^40, some rows of zeros, logits from the rope dims alone."""
    cache, scale = cpu_cache(g, 600, torch.randint(-40, 41, (600,), generator=g).float())
    cache[::7, :512] = 0
    q = torch.zeros(2, 64, 576)
    q[:, :, 512:] = torch.randn(2, 64, 64, generator=g)
    return q.bfloat16(), cache, scale, torch.randperm(600, generator=g)[:1000].int().view(2, 300).sort(1).values


def queries_of_every_size(g):
    """Query heads of 2^-30 .. 2^3, dims of a head 2^20 apart."""
    cache, scale = cpu_cache(g, 300, torch.full((300,), -6.0))
    q = torch.randn(2, 64, 576, generator=g) * torch.exp2(torch.linspace(-30, 3, 64))[None, :, None]
    q[1] = q[1] * torch.exp2(-torch.randint(0, 20, (64, 576), generator=g).float())
    return q.bfloat16(), cache, scale, torch.randperm(300, generator=g)[:256].int().repeat(2, 1)


def usual(g):
    cache, scale = cpu_cache(g, 500, torch.randint(-8, -3, (500,), generator=g).float())
    return torch.randn(2, 64, 576, generator=g).bfloat16(), cache, scale, torch.randperm(500, generator=g)[:400].int().repeat(2, 1)


def growing(g):
    """Scores that grow from tile to tile, or fall, and one outlier over a flat rest."""
    N = 1024
    cache, scale = cpu_cache(g, N, torch.full((N,), -6.0))
    rope = torch.zeros(N, 64)
    rope[:, 0], rope[:, 1], rope[700, 2] = torch.arange(N) / 16.0, torch.arange(N, 0, -1) / 16.0, 256.0
    cache[:, 512:] = rope.bfloat16().view(torch.uint8)
    q = torch.zeros(3, 64, 576)
    q[0, :, 512], q[1, :, 513], q[2, :, 514] = torch.arange(64) / 4.0, 16.0, torch.arange(64) / 32.0
    return q.bfloat16(), cache, scale, torch.arange(N, dtype=torch.int32).repeat(3, 1)


DATA = [far_apart, queries_of_every_size, growing, usual]


def with_weights(q, cache, scale, idx, made):
    """The output when made() stands in for the weights P', whose largest of a head is `top`."""
    out = []
    code = cache[:, :512].contiguous().view(F8).double()
    kv = values(cache, scale)
    for i in range(idx.shape[0]):
        at = idx[i].long()
        p = torch.softmax(q[i].double() @ kv[at].t() * SCALE, -1)
        w = p * scale[at].double() * (code[at] != 0).any(1)
        top = w.amax(1, keepdim=True)
        out.append(made(w / top) * top @ code[at])
    return torch.stack(out)


def e4m3(x):
    return x.half().to(F8).double()


def parts(top, lo):
    """Weights (the largest 1) as e4m3 parts when the largest lies at 2^top."""
    def made(w):
        x = w * 2.0 ** top
        hi = e4m3(x)
        return (hi + (e4m3((x.half().double() - hi) * 16) / 16 if lo else 0)) / 2.0 ** top
    return made


@pytest.mark.parametrize("data", DATA)
def test_bound_admits_two_parts_and_not_one(data):
    """The bound lets hi + lo / 16 pass at either end of the reference's range, and not hi alone (on the CPU)."""
    g = torch.Generator().manual_seed(37)
    q, cache, scale, idx = data(g)
    ref = attention64(q, cache, scale, idx)
    b = bound(ref)
    for top in (4.5, 6.0, 8.75):
        assert bool(((with_weights(q, cache, scale, idx, parts(top, True)) - ref[0]).abs() <= b).all())
        over = (with_weights(q, cache, scale, idx, parts(top, False)) - ref[0]).abs() > b
        assert float(over.double().mean()) > 0.01
    assert float((ref[0].abs() > b).double().mean()) > 0.5               # zeros do not pass


@pytest.mark.gpu
@pytest.mark.parametrize("data", DATA)
def test_attention_within_its_formats(dsa, data):
    q, cache, scale, idx = data(torch.Generator().manual_seed(38))
    both_ways(dsa, q.cuda(), cache.cuda(), scale.cuda(), idx.cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 127, 129, 1000, 2048])
def test_attention_of_any_length_within_its_formats(dsa, K):
    g = gen(K)
    N = 2 * K + 3
    cache, scale = make_cache(g, N, exponents=6)
    idx = choose(g, [N, max(1, K // 3), N], N, K)
    both_ways(dsa, randn(g, 3, 64, 576).bfloat16(), cache, scale, idx)


# ------------------------------------------------------------------------------------------------ waits

@pytest.mark.gpu
@pytest.mark.parametrize("warp", [False, True])
def test_polled_waits_give_up(dsa, warp):
    """Both forms of the attention's wait, on barriers nothing arrives on, give up after their polls and record
    DSA_ERR_DEVICE_TIMEOUT (6); the attention then runs as before."""
    g = gen(39)
    cache, scale = make_cache(g, 200)
    idx = torch.arange(200, dtype=torch.int32, device="cuda")[None].contiguous()
    q = randn(g, 1, 64, 576).bfloat16()
    want = dsa.mla_sparse_attn_prefill_q8(q, cache, scale, idx, SCALE)
    assert dsa.device_status() == 0
    for polls in (1, 256, 100000):
        dsa.selftest_poll_timeout(warp=warp, polls=polls)
        assert dsa.device_status() == 6
        assert dsa.device_status() == 0                                   # read and cleared
    assert torch.equal(dsa.mla_sparse_attn_prefill_q8(q, cache, scale, idx, SCALE), want)
    assert dsa.device_status() == 0


def test_polled_wait_selftest_refusals():
    """A form other than 0 or 1 and a limit outside 1 .. 2^26 are refused on the host (DSA_ERR_INVALID_ARG)."""
    from deepseek_sparse_attention_indexer_gb300 import _build, _lib
    f = _lib.load(_build.build()).dsa_selftest_poll_timeout
    for warp, polls in ((2, 256), (-1, 256), (0, 0), (1, 0), (0, (1 << 26) + 1), (1, 1 << 31)):
        assert f(warp, polls, None) == 1
