"""Eviction by attention weight on the GPU (the keys' weights, the plan, the moves), against plain float64 or integer
implementations written here.

Tolerances, from the arithmetic: a key's weight is a sum of exp(s - lse), s = scale * q . k.  The 576 products are exact,
their float32 sum is off by at most 576 * 2^-24 S, S the largest sum of their absolute values times scale, whatever
the order; the scale and the exponent add three float32 roundings of numbers up to M = S + |lse|, 2^-22 M; the exponential
2^-22 of itself (the unit's bound), the sum over 64 heads 64 * 2^-24, a prefill's last rounding to float32 and decode's
additions 2^-24 each.  All are relative to the weight: expm1(576 * 2^-24 S + 2^-22 M) + 2^-17.  A prefill's weights are whole
numbers of 2^-shift, half of one off a query: L * 2^-(shift + 1), and 2^-shift < 2 L 2^-55.
Plans and moves are exact.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
SCALE = 1.0 / 16.0
FORMATS = ["bf16", "q8", "q4"]
WIDTH = {"q8": 640, "q4": 416}


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deepseek_sparse_attention_indexer_gb300 import _build, _lib
    _build.build()
    _lib.load()
    _lib.device_status(reset=True)
    return _lib


@pytest.fixture(autouse=True)
def clean_status(dsa):
    yield
    dsa.device_status(reset=True)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make_cache(g, fmt, rows):
    """(cache, scales or None) of random rows; every code of a format, small scales."""
    if fmt == "bf16":
        return randn(g, rows, 576).bfloat16(), None
    cache = torch.empty(rows, WIDTH[fmt], dtype=torch.uint8, device="cuda")
    scale = torch.exp2(torch.randint(-1, 2, (rows,), generator=g, device="cuda").float() - 5.0)
    if fmt == "q8":
        cache[:, :512] = (randn(g, rows, 512) * 32.0).to(F8).view(torch.uint8)
        cache[::3, :64] = torch.arange(64, dtype=torch.uint8, device="cuda") % 16      # e4m3's subnormal numbers
    else:
        cache[:, :256] = torch.randint(0, 256, (rows, 256), generator=g, device="cuda").byte()
        cache[:, 256:288] = torch.randint(15, 33, (rows, 32), generator=g, device="cuda").byte()
        cache[::3, 256:266] = torch.tensor([0, 1, 2, 3, 4, 5, 35, 36, 40, 255], dtype=torch.uint8, device="cuda")
    cache[:, -128:] = randn(g, rows, 64).bfloat16().view(torch.uint8)
    return cache, scale


def values(fmt, cache, scale):
    """float64 rows [.., 576]."""
    if fmt == "bf16":
        return cache.double()
    rope = cache[..., -128:].contiguous().view(torch.bfloat16).double()
    if fmt == "q8":
        lat = cache[..., :512].contiguous().view(F8).double()
    else:
        index, neg = [], []
        for d in range(8):
            index.append(cache[..., d // 2:256:4].int() >> (4 * (d % 2)) & 7)
            neg.append(cache[..., d % 4:256:4].int() >> (7 if d < 4 else 3) & 1)
        mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")[torch.stack(index, -1).flatten(-2).long()]
        steps = torch.tensor([(1 + m / 4) * 2.0 ** (a - 6) for a in range(12) for m in range(3)] + [0.0] * 220,
                             dtype=torch.float64, device="cuda")
        step = steps[cache[..., 256:288].long()].repeat_interleave(16, -1)
        lat = torch.where(torch.stack(neg, -1).flatten(-2) > 0, -mag, mag) * step
    return torch.cat([lat * scale[..., None].double(), rope], -1)


def paged(g, cache, scale, lens, page, extra=3):
    """Dense [B, N, row] rows laid out over a shuffled pool; junk everywhere no sequence has a key."""
    B, N = cache.shape[:2]
    used = [-(-n // page) for n in lens]
    pages = sum(used) + extra
    perm = torch.randperm(pages, generator=g, device="cuda")
    pool = torch.full((pages * page, cache.shape[2]), 0xFF if cache.dtype == torch.uint8 else math.nan, dtype=cache.dtype,
                      device="cuda")
    pscale = None if scale is None else torch.full((pages * page,), math.nan, device="cuda")
    table = torch.full((B, -(-N // page)), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        for lp in range(used[b]):
            pg = int(perm[at])
            at += 1
            table[b, lp] = pg
            m = min(page, n - lp * page)
            pool[pg * page:pg * page + m] = cache[b, lp * page:lp * page + m]
            if scale is not None:
                pscale[pg * page:pg * page + m] = scale[b, lp * page:lp * page + m]
    return pool, pscale, table, pages


def choose(g, counts, N, top_k):
    """Ascending random selections of min(top_k, count) keys, -1 padded."""
    c = torch.tensor(counts, device="cuda")
    r = torch.rand(len(counts), N, generator=g, device="cuda")
    r.masked_fill_(torch.arange(N, device="cuda")[None] >= c[:, None], -1.0)
    val, idx = r.topk(min(top_k, N), 1)
    idx = idx.masked_fill(val < 0, N).sort(1).values
    idx = idx.masked_fill(idx == N, -1).int()
    return torch.nn.functional.pad(idx, (0, top_k - idx.shape[1]), value=-1).contiguous()


# ------------------------------------------------------------------------------------------------ weights

def weights64(q, rows, idx, scale=SCALE):
    """(lse f32 [R, 64], weights [R, K] float64 with that lse, relative tolerance): rows(slice) [r, K, 576] float64."""
    lse, w, S, M = [], [], 0.0, 0.0
    for i in range(0, q.shape[0], 32):
        kv, ok = rows(slice(i, i + 32)), (idx[i:i + 32] >= 0)[:, None]
        kv = torch.where(ok[:, 0, :, None], kv, 0.0)
        qq = q[i:i + 32].double()
        x = torch.where(ok, torch.einsum("rhd,rkd->rhk", qq, kv) * scale, -math.inf)
        S = max(S, float(torch.einsum("rhd,rkd->rhk", qq.abs(), kv.abs()).amax()) * scale)
        l32 = torch.logsumexp(x, -1).float()
        fine = torch.where(torch.isneginf(l32), 0.0, l32.double())
        M = max(M, S + float(fine.abs().amax()))
        lse.append(l32)
        w.append(torch.exp(x - fine[..., None]).sum(1))
    return torch.cat(lse), torch.cat(w), math.expm1(576 * 2.0 ** -24 * S + 2.0 ** -22 * M) + 2.0 ** -17


DECODE = [(1, 1, 1, 0), (1, 4096, 2048, 0), (2, 130, 129, 16), (5, 1000, 2048, 64), (3, 700, 127, 0), (37, 515, 400, 16),
          (170, 300, 256, 0)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,N,top_k,page", DECODE)
def test_decode_weights(dsa, fmt, B, N, top_k, page):
    g = gen(B * N)
    lens = [N if b == 0 else (b * 7919) % (N + 1) for b in range(B)]      # every length from none on
    cache, scale = make_cache(g, fmt, B * N)
    cache, scale = cache.view(B, N, -1), None if scale is None else scale.view(B, N)
    idx, kv_len = choose(g, lens, N, top_k), i32(*lens)
    q = randn(g, B, 64, 576).bfloat16()
    kv = values(fmt, cache, scale)
    lse, w, tol = weights64(q, lambda s: torch.stack([kv[b][idx[b].clamp(min=0).long()] for b in range(B)[s]]), idx)
    want = torch.zeros(B, N, dtype=torch.float64, device="cuda")
    want.scatter_add_(1, idx.clamp(min=0).long(), torch.where(idx >= 0, w, 0.0))
    if page:
        pool, pscale, table, _ = paged(g, cache, scale, lens, page)
        call = lambda acc=None: dsa.mla_key_weights_decode(q, pool, kv_len, idx, lse, SCALE, acc=acc, cache_scale=pscale,  # noqa: E731
                                                           block_table=table, page_size=page, Nmax=N)
    else:
        call = lambda acc=None: dsa.mla_key_weights_decode(q, cache, kv_len, idx, lse, SCALE, acc=acc, cache_scale=scale)  # noqa: E731
    got = call()
    assert dsa.device_status() == 0
    assert bool(((got.double() - want).abs() <= tol * want).all()), float(((got.double() - want).abs() / want.clamp(min=1e-300)).max())
    before = torch.rand(B, N, generator=g, device="cuda") * 10
    acc = before.clone()
    assert call(acc) is acc                                               # added: one rounding to float32
    assert torch.equal(acc, before + got)


PREFILL = [(1, 1, 1, 0), (1, 64, 64, 16), (64, 1024, 256, 0), (37, 1000, 100, 64), (300, 300, 128, 0), (200, 2300, 2048, 16)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("L,N,top_k,page", PREFILL)
def test_prefill_weights(dsa, fmt, L, N, top_k, page):
    g = gen(L + N)
    cache, scale = make_cache(g, fmt, N)
    idx = choose(g, [N - L + i + 1 for i in range(L)], N, top_k)
    if L > 3:
        idx[L // 2] = -1                                                  # nothing selected
        idx[1] = idx[1][torch.randperm(top_k, generator=g, device="cuda")]   # any order, -1 between
        idx[2, :3] = idx[2, 0]                                            # a key given several times counts so often
    q = randn(g, L, 64, 576).bfloat16()
    kv = values(fmt, cache, scale)
    lse, w, tol = weights64(q, lambda s: kv[idx[s].clamp(min=0).long()], idx)
    want = torch.zeros(N, dtype=torch.float64, device="cuda")
    want.index_add_(0, idx.clamp(min=0).long().flatten(), torch.where(idx >= 0, w, 0.0).flatten())
    if page:
        pool, pscale, table, _ = paged(g, cache[None], None if scale is None else scale[None], [N], page)
        call = lambda acc=None: dsa.mla_key_weights_prefill(q, pool, idx, lse, SCALE, acc=acc, cache_scale=pscale,  # noqa: E731
                                                            block_table=table[0], page_size=page, N=N)
    else:
        call = lambda acc=None: dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, acc=acc, cache_scale=scale)  # noqa: E731
    got = call()
    assert dsa.device_status() == 0
    assert bool(((got.double() - want).abs() <= tol * want + 2 * L * L * 2.0 ** -56).all())
    acc = torch.full((N,), 3.0, device="cuda")
    assert call(acc) is acc and torch.equal(acc, 3.0 + got)
    for _ in range(5):                                                    # whatever the order of the queries
        assert torch.equal(call(), got)


@pytest.mark.parametrize("fmt", FORMATS)
def test_weights_of_the_attention_itself(dsa, fmt):
    """With the lse that the attention returned, a query's weights sum to its heads."""
    g = gen(3)
    L, N, K = 40, 900, 500
    cache, scale = make_cache(g, fmt, N)
    idx, q = choose(g, [N - L + i + 1 for i in range(L)], N, K), randn(g, L, 64, 576).bfloat16()
    if fmt == "bf16":
        _, lse = dsa.mla_sparse_attn_prefill(q, cache, idx, SCALE, want_lse=True)
    else:
        _, lse = getattr(dsa, f"mla_sparse_attn_prefill_{fmt}")(q, cache, scale, idx, SCALE, want_lse=True)
    acc = dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale)
    # lse is within 2^-12 (its bound in the attentions' tests), which is a factor of every weight
    assert abs(float(acc.double().sum()) - 64 * L) <= 64 * L * 2.0 ** -11
    one = dsa.mla_key_weights_decode(q[:1], cache[None].contiguous(), i32(N), idx[:1].contiguous(), lse[:1].contiguous(), SCALE,
                                     cache_scale=None if scale is None else scale[None].contiguous())
    assert abs(float(one.double().sum()) - 64) <= 64 * 2.0 ** -11
    alone = dsa.mla_key_weights_prefill(q[:1], cache, idx[:1].contiguous(), lse[:1].contiguous(), SCALE, cache_scale=scale)
    assert torch.equal(one[0], alone)


def test_weights_of_odd_numbers(dsa):
    """NaN and infinite rows, a lse of -inf, +inf or NaN: weights of 0 or cut at 128, and no other key's."""
    g = gen(4)
    N = 300
    kv = randn(g, N, 576).bfloat16()
    q = randn(g, 1, 64, 576).bfloat16()
    idx = torch.arange(N, dtype=torch.int32, device="cuda")[None].contiguous()
    lse, _, _ = weights64(q, lambda s: kv.double()[None], idx)
    want = dsa.mla_key_weights_prefill(q, kv, idx, lse, SCALE)
    bad = kv.clone()
    bad[7, 3] = math.nan
    bad[9] = math.inf
    got = dsa.mla_key_weights_prefill(q, bad, idx, lse, SCALE)
    got1 = dsa.mla_key_weights_decode(q, bad[None], i32(N), idx, lse, SCALE)[0]
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[[7, 9]] = False
    for x in (got, got1):
        assert torch.equal(x[rest], want[rest]) and float(x[7]) == 0.0 and 0.0 <= float(x[9]) <= 128.0
    for value, least, most in ((math.inf, 0.0, 0.0), (math.nan, 0.0, 0.0), (-math.inf, 128.0, 128.0), (-1e30, 128.0, 128.0)):
        odd = torch.full_like(lse, value)
        for x in (dsa.mla_key_weights_prefill(q, kv, idx, odd, SCALE), dsa.mla_key_weights_decode(q, kv[None], i32(N), idx, odd, SCALE)):
            assert bool((x >= least).all()) and bool((x <= most).all())
    assert dsa.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_weights_record_keys_outside_the_cache(dsa, fmt):
    g = gen(5)
    B, N, K, page = 3, 100, 40, 16
    cache, scale = make_cache(g, fmt, B * N)
    cache, scale = cache.view(B, N, -1), None if scale is None else scale.view(B, N)
    lens = [100, 50, 10]
    idx = choose(g, lens, N, K)
    q, lse = randn(g, B, 64, 576).bfloat16(), torch.full((B, 64), 4.0, device="cuda")
    want = dsa.mla_key_weights_decode(q, cache, i32(*lens), idx, lse, SCALE, cache_scale=scale)
    more = torch.cat([idx, torch.full((B, 1), 2 ** 31 - 1, dtype=torch.int32, device="cuda"), i32(*lens)[:, None]], 1).contiguous()
    got = dsa.mla_key_weights_decode(q, cache, i32(*lens), more, lse, SCALE, cache_scale=scale)
    assert dsa.device_status() == 7 and torch.equal(got, want)
    pool, pscale, table, pages = paged(g, cache, scale, lens, page)
    kept = dsa.mla_key_weights_decode(q, pool, i32(*lens), idx, lse, SCALE, cache_scale=pscale, block_table=table, page_size=page, Nmax=N)
    assert torch.equal(kept, want) and dsa.device_status() == 0
    table[0, 2] = pages + 5
    got = dsa.mla_key_weights_decode(q, pool, i32(*lens), idx, lse, SCALE, cache_scale=pscale, block_table=table, page_size=page, Nmax=N)
    assert dsa.device_status() == 7
    want[0, 2 * page:3 * page] = 0.0
    assert torch.equal(got, want)


@pytest.mark.parametrize("page", [0, 16])
def test_weights_over_expanded_rows(dsa, page):
    """A 4-bit prefill that selects each key many times: the weights of the 8-bit rows of the same values; a page outside
    the pool is recorded where a query selects it, and only there."""
    g = gen(8)
    N, L, K = 500, 320, 450
    assert dsa.key_weights_workspace_size(L, K, N, 2) > N * 648
    cache, scale = make_cache(g, "q4", N)
    eight = torch.cat([(values("q4", cache, scale)[:, :512] / scale[:, None].double()).float().to(F8).view(torch.uint8), cache[:, 288:]], 1)
    idx, q, lse = choose(g, [N - 20] * L, N, K), randn(g, L, 64, 576).bfloat16(), torch.full((L, 64), 6.0, device="cuda")
    want = dsa.mla_key_weights_prefill(q, eight, idx, lse, SCALE, cache_scale=scale)
    if not page:
        assert torch.equal(dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale), want)
        ws = torch.full((dsa.key_weights_workspace_size(L, K, N, 2) + 64,), 0xEE, dtype=torch.uint8, device="cuda")
        got = dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale, workspace=ws[:-64])
        assert torch.equal(got, want) and bool((ws[-64:] == 0xEE).all())
        # as many queries as are read directly, a few at a time
        few = torch.zeros(N, device="cuda", dtype=torch.float64)
        for i in range(0, L, 8):
            few += dsa.mla_key_weights_prefill(q[i:i + 8], cache, idx[i:i + 8], lse[i:i + 8], SCALE, cache_scale=scale).double()
        assert bool(((few - want.double()).abs() <= 2.0 ** -22 * want.double()).all())   # roundings to float32: 41 of them
        return
    pool, pscale, table, pages = paged(g, cache[None], scale[None], [N], page)
    table[0, -1] = pages                                                  # keys that nothing selects
    call = lambda: dsa.mla_key_weights_prefill(q, pool, idx, lse, SCALE, cache_scale=pscale, block_table=table[0],  # noqa: E731
                                               page_size=page, N=N)
    assert torch.equal(call(), want) and dsa.device_status() == 0
    table[0, 2] = -1
    got = call()
    assert dsa.device_status() == 7
    want[2 * page:3 * page] = 0.0
    assert torch.equal(got, want)


def test_weights_past_32_bits(dsa):
    g = gen(6)
    N = (1 << 32) // 1152 + 3000
    kv = torch.zeros(N, 576, dtype=torch.bfloat16, device="cuda")
    some = torch.cat([torch.arange(100, device="cuda"), torch.arange(N - 400, N, device="cuda")])
    rows = randn(g, len(some), 576).bfloat16()
    kv[some] = rows
    q, lse = randn(g, 1, 64, 576).bfloat16(), torch.full((1, 64), 5.0, device="cuda")
    got = dsa.mla_key_weights_prefill(q, kv, some.int()[None].contiguous(), lse, SCALE)
    near = dsa.mla_key_weights_prefill(q, rows, torch.arange(len(some), dtype=torch.int32, device="cuda")[None].contiguous(), lse, SCALE)
    assert torch.equal(got[some], near) and float(got.double().sum()) == float(near.double().sum())


def test_weights_streams_and_graphs(dsa):
    g = gen(7)
    N, K, L = 1500, 700, 5
    kv = randn(g, N, 576).bfloat16()
    qs = [randn(g, L, 64, 576).bfloat16() for _ in range(2)]
    idx, lse = choose(g, [N] * L, N, K), torch.full((L, 64), 5.0, device="cuda")
    want = [dsa.mla_key_weights_prefill(q, kv, idx, lse, SCALE) for q in qs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.mla_key_weights_prefill(qs[0], kv, idx, lse, SCALE, stream=side)
    one = dsa.mla_key_weights_decode(qs[0][:1], kv[None], i32(N), idx[:1].contiguous(), lse[:1].contiguous(), SCALE, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    assert torch.equal(one, dsa.mla_key_weights_decode(qs[0][:1], kv[None], i32(N), idx[:1].contiguous(), lse[:1].contiguous(), SCALE))
    graphs = []
    for q in qs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = dsa.mla_key_weights_prefill(q, kv, idx, lse, SCALE)
        graphs.append((graph, y))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for (_, y), w in zip(graphs, want))


# ------------------------------------------------------------------------------------------------ plan

def plan_by_sorting(acc, pos, kv_len, keep, recent, sink):
    """The plan by a stable sort on the host, sequence by sequence."""
    B, N = acc.shape
    M = min(keep, N - keep)
    src, dst, left = torch.full((B, M), -1, dtype=torch.int32), torch.full((B, M), -1, dtype=torch.int32), []
    for b in range(B):
        n = max(0, min(int(kv_len[b]), N))
        left.append(min(n, keep))
        if n <= keep:
            continue
        w, p = acc[b, :n].double(), pos[b, :n].long()
        safe = (p > int(p.max()) - recent) & (recent > 0) | (p < sink)
        # protected ones first, by index alone, NaN last of all: three sorts of one order
        nan = torch.isnan(w) & ~safe
        w = torch.where(safe | nan, 0.0, w)
        order = torch.sort(w, descending=True, stable=True).indices
        order = order[torch.sort(nan[order].int(), stable=True).indices]
        order = torch.cat([safe.nonzero()[:, 0], order[~safe[order]]])
        stay = torch.zeros(n, dtype=torch.bool)
        stay[order[:keep]] = True
        gaps = (~stay[:keep]).nonzero()[:, 0]
        movers = stay[keep:].nonzero()[:, 0] + keep
        assert len(gaps) == len(movers)
        dst[b, :len(gaps)], src[b, :len(gaps)] = gaps.int(), movers.int()
    return src, dst, torch.tensor(left, dtype=torch.int32)


def check_plan(dsa, acc, pos, kv_len, keep, recent, sink):
    want = plan_by_sorting(acc.cpu(), pos.cpu(), kv_len.cpu(), keep, recent, sink)
    got = dsa.cache_evict_plan(acc, pos, kv_len, keep, recent=recent, sink=sink)
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)
    return got


PLANS = [(1, 2, 1, 0, 0), (3, 3, 2, 1, 1), (70, 100, 37, 5, 2), (2, 2048, 2047, 100, 4), (5, 2049, 1, 1, 0), (5, 2049, 1000, 0, 0),
         (3, 5000, 4999, 0, 7), (8, 4096, 2048, 256, 4), (2, 16385, 8000, 8000, 0), (40, 9001, 3000, 300, 3), (1, 70001, 65536, 4096, 4),
         (1, 389000, 200000, 1000, 0), (1, 400001, 100000, 512, 4)]


@pytest.mark.parametrize("B,N,keep,recent,sink", PLANS)
def test_plan(dsa, B, N, keep, recent, sink):
    g = gen(N + keep)
    acc = torch.exp(3 * randn(g, B, N))
    acc[torch.rand(B, N, generator=g, device="cuda") < 0.2] = 0.0         # ties
    pos = torch.rand(B, N, generator=g, device="cuda").argsort(1).int() * 3
    lens = [N if b == 0 else (b * 7919) % (N + 2) for b in range(B)]
    lens[-1] = N + 100 if B > 2 else N                                    # more than there are
    if B > 3:
        lens[1], lens[2] = 0, keep
    check_plan(dsa, acc, pos, i32(*lens), keep, recent, sink)
    assert dsa.device_status() == 0


@pytest.mark.parametrize("N", [40, 3000, 20000])
def test_plan_of_odd_weights(dsa, N):
    """Equal weights everywhere, signed zeros, infinities, NaN, numbers that differ in their last bit."""
    g = gen(N)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None].repeat(6, 1).contiguous()
    acc = torch.zeros(6, N, device="cuda")
    acc[1] = 1.5
    acc[2] = torch.where(torch.rand(N, generator=g, device="cuda") < 0.5, 0.0, -0.0)
    acc[3] = randn(g, N)
    acc[3, ::7], acc[3, 1::7], acc[3, 2::7] = math.inf, -math.inf, math.nan
    acc[4] = (1.0 + torch.randint(0, 3, (N,), generator=g, device="cuda") * 2.0 ** -23)
    acc[5] = torch.rand(N, generator=g, device="cuda") * 1e-41             # subnormal
    kv_len = i32(*[N] * 6)
    for keep in (1, N // 3, N - 1):
        for recent, sink in ((0, 0), (keep // 2, keep - keep // 2)):
            check_plan(dsa, acc, pos, kv_len, keep, recent, sink)


def test_plan_of_odd_positions(dsa):
    """Positions at the ends of 32 bits, negative ones, the same position for all."""
    g = gen(9)
    N = 500
    acc = torch.rand(4, N, generator=g, device="cuda")
    pos = torch.randperm(N, generator=g, device="cuda").int()[None].repeat(4, 1)
    pos[0] += 2 ** 31 - 1 - N
    pos[1] -= 2 ** 31 - 1
    pos[2] = 7
    for keep, recent, sink in ((100, 50, 50), (100, 100, 0), (1, 0, 1)):
        check_plan(dsa, acc, pos.contiguous(), i32(N, N, N, 300), keep, recent, sink)


def test_plan_streams_graphs_and_repeats(dsa):
    g = gen(10)
    B, N, keep = 6, 6000, 2500
    acc, pos = torch.rand(B, N, generator=g, device="cuda"), torch.rand(B, N, generator=g, device="cuda").argsort(1).int()
    kv_len = i32(6000, 100, 2500, 2501, 0, 5999)
    want = check_plan(dsa, acc, pos, kv_len, keep, 64, 4)
    for _ in range(50):
        assert all(torch.equal(x, y) for x, y in zip(dsa.cache_evict_plan(acc, pos, kv_len, keep, 64, 4), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.cache_evict_plan(acc, pos, kv_len, keep, 64, 4, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dsa.cache_evict_plan(acc, pos, kv_len, keep, 64, 4)
        dsa.cache_move_rows(got[0], got[1], dense=(acc, pos))
    keepers = acc.clone(), pos.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    moved = [t.clone() for t in keepers]
    dsa.cache_move_rows(want[0], want[1], dense=moved)
    assert torch.equal(moved[0], acc) and torch.equal(moved[1], pos)


# ------------------------------------------------------------------------------------------------ moves

def moved_by_hand(t, src, dst, rows):
    """t with its rows moved; rows(b, j): the row of key j of sequence b in t, flat."""
    t = t.clone()
    b, m = ((src >= 0) & (dst >= 0)).nonzero(as_tuple=True)
    t[rows(b, dst[b, m].long())] = t[rows(b, src[b, m].long())].clone()
    return t


@pytest.mark.parametrize("B,N,keep,page", [(1, 2, 1, 0), (3, 100, 40, 16), (9, 1000, 700, 64), (2, 9000, 4000, 256),
                                           (700, 40, 20, 16), (5000, 3, 2, 0)])
def test_moves(dsa, B, N, keep, page):
    """Rows of 4 to 2048 bytes, 16-byte ones and others, dense and paged in one call; all other rows stay."""
    g = gen(B * N)
    acc = torch.rand(B, N, generator=g, device="cuda")
    pos = torch.rand(B, N, generator=g, device="cuda").argsort(1).int()
    lens = [N if b == 0 else (b * 7919) % (N + 1) for b in range(B)]
    src, dst, left = dsa.cache_evict_plan(acc, pos, i32(*lens), keep, recent=0, sink=0)
    pick = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda").byte()  # noqa: E731
    dense = [acc, pos, pick(B, N, 12), pick(B, N, 256), pick(B, N, 1152)]
    flat = lambda b, j: b * N + j  # noqa: E731
    if page:
        stride = -(-N // page)
        table = torch.randperm(B * stride + 2, generator=g, device="cuda")[:B * stride].int().view(B, stride).contiguous()
        rows = (B * stride + 2) * page
        pools = [pick(rows, 416), pick(rows, 2048), pick(rows, 20)]
        place = lambda b, j: table[b, j // page].long() * page + j % page  # noqa: E731
    else:
        table, pools, place = None, [], None
    want = [moved_by_hand(t.flatten(0, 1), src, dst, flat).view_as(t) for t in dense]
    want += [moved_by_hand(t, src, dst, place) for t in pools]
    dsa.cache_move_rows(src, dst, dense=dense, paged=pools, block_table=table, page_size=page)
    assert dsa.device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(dense + pools, want))
    if page:                                                              # paged tensors alone
        again = [moved_by_hand(t, src, dst, place) for t in pools]
        dsa.cache_move_rows(src, dst, paged=pools, block_table=table, page_size=page)
        assert all(torch.equal(x, y) for x, y in zip(pools, again))


def test_moves_record_what_is_out_of_range(dsa):
    N, page = 64, 16
    t = torch.arange(2 * N, dtype=torch.int32, device="cuda").view(2, N)
    src = i32(5, 64, 7, -1, 2 ** 31 - 1, 9, 60, 61, -5, 62).view(2, 5)
    dst = i32(0, 1, 64, 3, 4, 1, 2, -1, 4, 5).view(2, 5)
    want = t.clone()
    want[0, 0], want[1, 1], want[1, 2], want[1, 5] = t[0, 5], t[1, 9], t[1, 60], t[1, 62]
    dsa.cache_move_rows(src, dst, dense=(t,))
    assert dsa.device_status() == 7 and torch.equal(t, want)
    pool = torch.arange(6 * page, dtype=torch.int32, device="cuda")[:, None].contiguous()
    table = i32(0, 1, 2, 99, 3, 4, -1, 5).view(2, 4)
    before = pool.clone()
    dsa.cache_move_rows(i32(1, 50, 20, 2).view(2, 2), i32(17, 2, 1, 40).view(2, 2), paged=(pool,), block_table=table, page_size=page)
    before[17], before[3 * page + 1] = 1, 4 * page + 4
    assert dsa.device_status() == 7 and torch.equal(pool, before)


def test_moves_of_odd_tensors(dsa):
    """A sequence of one row, whose strides say nothing; bases that are not 16-byte aligned; a row of 4000 bytes."""
    one = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2).t()[:1].t()     # [3, 1], strides of a wider tensor
    one = one.as_strided((3, 1), (1, 77))
    assert one.is_contiguous()
    before = one.clone()
    dsa.cache_move_rows(i32(0, 0, 0)[:, None].contiguous(), i32(0, 0, 0)[:, None].contiguous(), dense=(one,))
    assert torch.equal(one, before)
    flat = torch.arange(1 + 2 * 8 * 8, dtype=torch.int32, device="cuda")
    odd, long = flat[1:].view(2, 8, 8), torch.arange(2 * 8 * 1000, dtype=torch.int32, device="cuda").view(2, 8, 1000)
    want = odd.clone(), long.clone()
    for t in want:
        t[0, 1], t[1, 2], t[1, 0] = t[0, 6].clone(), t[1, 7].clone(), t[1, 4].clone()
    dsa.cache_move_rows(i32(6, -1, 7, 4).view(2, 2), i32(1, -1, 2, 0).view(2, 2), dense=(odd, long))
    assert torch.equal(odd, want[0]) and torch.equal(long, want[1]) and int(flat[0]) == 0 and dsa.device_status() == 0


def test_moves_past_32_bits(dsa):
    N = (1 << 32) // 2048 + 4000
    t = torch.zeros(1, N, 512, dtype=torch.int32, device="cuda")
    t[0, N - 2], t[0, N - 1] = 5, torch.arange(512, device="cuda").int()
    dsa.cache_move_rows(i32(N - 1, N - 2)[None], i32(3, N - 10)[None], dense=(t,))
    assert torch.equal(t[0, 3], torch.arange(512, device="cuda").int()) and bool((t[0, N - 10] == 5).all())
    assert dsa.device_status() == 0 and int((t[0, 4:N - 10] != 0).sum()) == 0


# ------------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt,page", [("bf16", 0), ("q8", 16), ("q4", 64), ("q4", 0)])
def test_decode_with_eviction(dsa, fmt, page):
    """Steps of decode with running weights, an eviction, and steps after it: every step's output is that of the same
    keys in a cache that nothing was moved in."""
    g = gen(20)
    B, N, keep, recent, K = 3, 400, 150, 20, 128
    start = [300, 120, 250]
    cache, scale = make_cache(g, fmt, B * N)
    cache, scale = cache.view(B, N, -1), None if scale is None else scale.view(B, N)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None].repeat(B, 1).contiguous()
    acc = torch.zeros(B, N, device="cuda")
    whole, whole_scale = cache.clone(), None if scale is None else scale.clone()
    if page:
        lens = [N] * B                                                    # pages for all of a sequence's keys
        cache, scale, table, _ = paged(g, cache, scale, lens, page)
        paging = {"block_table": table, "page_size": page, "Nmax": N}
    else:
        paging = {}
    kind = "" if fmt == "bf16" else "_" + fmt

    def attend(c, s, q, kv_len, idx, is_paged):
        first = (q, c) if s is None else (q, c, s)
        if is_paged:
            return getattr(dsa, f"mla_sparse_attn_decode{kind}_paged")(*first, kv_len, table, page, idx, SCALE, N, want_lse=True)
        return getattr(dsa, f"mla_sparse_attn_decode{kind}")(*first, kv_len, idx, SCALE, want_lse=True)

    kv_len = i32(*start)
    for step in range(6):
        q = randn(g, B, 64, 576).bfloat16()
        n = kv_len.tolist()
        idx = choose(g, n, N, K)
        out, lse = attend(cache, scale, q, kv_len, idx, bool(page))
        dsa.mla_key_weights_decode(q, cache, kv_len, idx, lse, SCALE, acc=acc, cache_scale=scale, **paging)
        # the same keys by their positions, in the cache as it was
        old = torch.where(idx >= 0, pos.gather(1, idx.clamp(min=0).long()), -1).contiguous()
        out2, lse2 = attend(whole, whole_scale, q, i32(*[N] * B), old, False)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        if step == 2:
            before, weights = [pos[b, :n[b]].clone() for b in range(B)], acc.clone()
            src, dst, left = dsa.cache_evict_plan(acc, pos, kv_len, keep, recent=recent, sink=2)
            dense, pools = [acc, pos], [cache] + ([] if scale is None else [scale])
            if page:
                dsa.cache_move_rows(src, dst, dense=dense, paged=pools, block_table=table, page_size=page)
            else:
                dsa.cache_move_rows(src, dst, dense=dense + pools)
            assert left.tolist() == [150, 120, 150]
            for b in range(B):
                kept = pos[b, :int(left[b])].long()
                assert len(kept.unique()) == len(kept)
                assert torch.equal(acc[b, :int(left[b])], weights[b][kept])           # still in the order of positions
                gone = torch.ones(n[b], dtype=torch.bool, device="cuda")
                gone[kept] = False
                free = (kept >= 2) & (kept < n[b] - recent)
                if bool(gone.any()):
                    assert float(weights[b][:n[b]][gone].max()) <= float(acc[b, :len(kept)][free].min())
                    assert not bool(gone[:2].any()) and not bool(gone[n[b] - recent:].any())
            kv_len = left
        assert dsa.device_status() == 0


def test_wrapper_refusals(dsa):
    q = torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(2, 8, 576, dtype=torch.bfloat16, device="cuda")
    idx, kv_len, lse = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), i32(8, 8), torch.zeros(2, 64, device="cuda")
    good = dict(q=q, cache=kv, kv_len=kv_len, idx=idx, lse=lse, scale=SCALE)
    dsa.mla_key_weights_decode(**good)
    for bad in (dict(cache=kv[:, :4]), dict(cache=kv.float()), dict(cache_scale=torch.ones(2, 8, device="cuda")),
                dict(cache=torch.zeros(2, 8, 416, dtype=torch.uint8, device="cuda")), dict(lse=lse[:1]), dict(q=q[:, :32]),
                dict(cache=torch.zeros(2, 8, 400, dtype=torch.uint8, device="cuda"), cache_scale=torch.ones(2, 8, device="cuda")),
                dict(block_table=i32(0, 0).view(2, 1)), dict(acc=torch.zeros(2, 9, device="cuda")), dict(kv_len=kv_len.cpu()), dict(Nmax=9)):
        with pytest.raises(ValueError):
            dsa.mla_key_weights_decode(**{**good, **bad})
    with pytest.raises(ValueError):                                       # a table of no pages is not a dense cache
        dsa.mla_key_weights_decode(**{**good, "cache": kv[0]}, block_table=i32().view(2, 0), page_size=16, Nmax=64)
    flat = dict(q=q, cache=kv[0], idx=idx, lse=lse, scale=SCALE)
    dsa.mla_key_weights_prefill(**flat)
    for bad in (dict(N=9), dict(block_table=i32(0)), dict(block_table=i32(0), page_size=16, N=17), dict(idx=idx.long()),
                dict(acc=torch.zeros(7, device="cuda"))):
        with pytest.raises(ValueError):
            dsa.mla_key_weights_prefill(**{**flat, **bad})
    with pytest.raises(dsa.DsaError):
        dsa.mla_key_weights_prefill(**flat, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    acc, pos = torch.zeros(2, 8, device="cuda"), torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    for bad in (dict(keep=8), dict(keep=0), dict(acc=acc[0]), dict(pos=pos[:1]), dict(kv_len=kv_len[:1]), dict(acc=acc.double())):
        with pytest.raises(ValueError):
            dsa.cache_evict_plan(**{**dict(acc=acc, pos=pos, kv_len=kv_len, keep=4), **bad})
    with pytest.raises(dsa.DsaError):
        dsa.cache_evict_plan(acc, pos, kv_len, 4, recent=3, sink=2)
    with pytest.raises(dsa.DsaError):
        dsa.cache_evict_plan(acc, pos, kv_len, 4, recent=1 << 32)          # not a number of 32 bits
    src, dst, _ = dsa.cache_evict_plan(acc, pos, kv_len, 4)
    for bad in (dict(), dict(dense=(acc, pos[:1])), dict(dense=(acc[:, :4],)), dict(paged=(acc,)), dict(dense=(acc,) * 9),
                dict(dense=(acc, torch.zeros(2, 9, device="cuda"))), dict(dense=(acc.cpu(),)),
                dict(dense=(torch.empty(2, 8, (1 << 18) + 1, device="cuda"),))):
        with pytest.raises(ValueError):
            dsa.cache_move_rows(src, dst, **bad)
    with pytest.raises(dsa.DsaError):
        dsa.cache_move_rows(src, dst, dense=(torch.zeros(2, 8, 3, dtype=torch.uint8, device="cuda"),))
