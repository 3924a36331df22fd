"""Eviction at its ends: the keys' weights where a CTA takes many queries and where the heads of a query differ in size, against
float64; moves that are left out.

Tolerances, from the arithmetic: those of test_gpu_evict.py (576 float32 additions of a score, off by at most 576 * 2^-24 of the
sum S of its terms' absolute values, roundings of numbers up to S + |lse|, the exponential's and the sums'), but a head's own S
and lse in place of the largest.  Over 8-bit and 4-bit rows the query's latent dims enter as hi + lo / 16 in e4m3, exact where
a dim is 2^-13 of its head's largest or more; below, lo ends at steps of 2^-9, so a dim is off by at most 2^-10 / 16 beside a
largest of at least 224: 2^-21.8 of it, taken as 2^-21.  A score is off by that times scale * the sum of the key's |latent dims|.
"""
import math
import threading

import pytest

torch = pytest.importorskip("torch")

from test_gpu_evict import SCALE, choose, gen, i32, make_cache, paged, plan_by_sorting, randn, values  # noqa: E402

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


def weights64(q, rows, idx, split):
    """(lse f32 [R, 64], weights [R, K] in float64 with that lse, bounds [R, K]): rows(slice) [r, K, 576] float64; split: the
    query is held as two e4m3 numbers."""
    lse, w, bound = [], [], []
    for i in range(0, q.shape[0], 32):
        kv, ok = rows(slice(i, i + 32)), (idx[i:i + 32] >= 0)[:, None]
        kv, qq = torch.where(ok[:, 0, :, None], kv, 0.0), q[i:i + 32].double()
        x = torch.where(ok, torch.einsum("rhd,rkd->rhk", qq, kv) * SCALE, -math.inf)
        S = torch.einsum("rhd,rkd->rhk", qq.abs(), kv.abs()) * SCALE
        l32 = torch.logsumexp(x, -1).float()
        fine = torch.where(torch.isneginf(l32), 0.0, l32.double())
        off = 576 * 2.0 ** -24 * S + 2.0 ** -22 * (S + fine.abs()[..., None])
        if split:
            off = off + 2.0 ** -21 * SCALE * qq[..., :512].abs().amax(-1)[..., None] * kv[..., :512].abs().sum(-1)[:, None]
        p = torch.exp(x - fine[..., None])
        lse.append(l32)
        w.append(p.sum(1))
        bound.append((p * (torch.expm1(off) + 2.0 ** -17)).sum(1))
    return torch.cat(lse), torch.cat(w), torch.cat(bound)


def summed(x, idx, n):
    """[R, K] numbers of selected keys added up over all rows, [n]."""
    out = torch.zeros(n, dtype=torch.float64, device="cuda")
    return out.index_add_(0, idx.clamp(min=0).long().flatten(), torch.where(idx >= 0, x, 0.0).flatten())


def sized_queries(g, rows):
    """Heads of every size from 1 down to 2^-12, drawn anew for each query."""
    return (randn(g, rows, 64, 576) * torch.exp2(-torch.randint(0, 13, (rows, 64, 1), generator=g, device="cuda").float())).bfloat16()


# ------------------------------------------------------------------------------------------------ many queries a CTA

@pytest.mark.parametrize("fmt,N", [("bf16", 1024), ("q8", 1024), ("q4", 1024), ("q4", 20000)])
def test_prefill_of_many_short_queries(dsa, fmt, N):
    """Nine queries of one tile a CTA (4-bit rows expanded, and read directly): each with its own heads' scales."""
    g = gen(N)
    L, K = 1300, 128
    cache, scale = make_cache(g, fmt, N)
    idx, q = choose(g, [N - (i * 7919) % 100 if i % 50 else 0 for i in range(L)], N, K), sized_queries(g, L)
    assert (dsa.key_weights_workspace_size(L, K, N, 2) > 8 * N) == (N == 1024)
    kv = values(fmt, cache, scale)
    lse, w, bound = weights64(q, lambda s: kv[idx[s].clamp(min=0).long()], idx, fmt != "bf16")
    want, bound = summed(w, idx, N), summed(bound, idx, N)
    got = dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale)
    assert dsa.device_status() == 0
    assert bool(((got.double() - want).abs() <= bound + 2 * L * L * 2.0 ** -56).all()), float(((got.double() - want).abs() / bound).nan_to_num().max())
    for _ in range(20):
        assert torch.equal(dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale), got)


@pytest.mark.parametrize("fmt,N", [("bf16", 3000), ("q8", 3000), ("q4", 3000), ("q4", 100000)])
def test_prefill_of_many_queries_of_all_lengths(dsa, fmt, N):
    """Six queries a CTA of none to six tiles each, one tile and several next to each other."""
    g = gen(N + 1)
    L, K = 900, 700
    cache, scale = make_cache(g, fmt, N)
    q, many = sized_queries(g, L), torch.randint(0, K + 1, (L, 1), generator=g, device="cuda")
    many[::3] = many[::3] % 129
    idx = choose(g, [N] * L, N, K).masked_fill(torch.arange(K, device="cuda") >= many, -1)
    assert (dsa.key_weights_workspace_size(L, K, N, 2) > 8 * N) == (N == 3000)
    kv = values(fmt, cache, scale)
    lse, w, bound = weights64(q, lambda s: kv[idx[s].clamp(min=0).long()], idx, fmt != "bf16")
    want, bound = summed(w, idx, N), summed(bound, idx, N)
    got = dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale)
    assert dsa.device_status() == 0
    assert bool(((got.double() - want).abs() <= bound + 2 * L * L * 2.0 ** -56).all()), float(((got.double() - want).abs() / bound).nan_to_num().max())
    for _ in range(20):
        assert torch.equal(dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale), got)


@pytest.mark.parametrize("fmt", ["bf16", "q8", "q4"])
def test_decode_of_many_short_sequences(dsa, fmt):
    g = gen(2)
    B, N, K = 1300, 140, 128
    lens = [(b * 7919) % (N + 1) for b in range(B)]
    cache, scale = make_cache(g, fmt, B * N)
    idx, q, kv_len = choose(g, lens, N, K), sized_queries(g, B), i32(*lens)
    first = torch.arange(B, device="cuda")[:, None] * N
    at = torch.where(idx >= 0, idx + first, -1)
    kv = values(fmt, cache, scale)
    lse, w, bound = weights64(q, lambda s: kv[at[s].clamp(min=0)], idx, fmt != "bf16")
    want, bound = summed(w, at, B * N).view(B, N), summed(bound, at, B * N).view(B, N)
    cache, scale = cache.view(B, N, -1), None if scale is None else scale.view(B, N)
    got = dsa.mla_key_weights_decode(q, cache, kv_len, idx, lse, SCALE, cache_scale=scale)
    assert dsa.device_status() == 0
    assert bool(((got.double() - want).abs() <= bound).all()), float(((got.double() - want).abs() / bound).nan_to_num().max())
    for _ in range(20):
        assert torch.equal(dsa.mla_key_weights_decode(q, cache, kv_len, idx, lse, SCALE, cache_scale=scale), got)


# ------------------------------------------------------------------------------------------------ heads of one large dim

F8 = torch.float8_e4m3fn


def as_two_e4m3(q):
    """Queries [.., 576] as they enter over 8-bit and 4-bit rows: latent dims hi + lo / 16 times a power of two a head, by which
    the largest is in (224, 448]; both numbers nearest, from half precision."""
    lat = q[..., :512].double()
    top = lat.abs().amax(-1, keepdim=True)
    step = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
    x = (lat / step).half()
    hi = x.float().to(F8).float()
    lo = ((x.float() - hi).half() * 16).float().to(F8).double()
    out = (hi.double() + lo / 16) * step
    assert bool(((out - lat).abs() <= 2.0 ** -21 * top).all())
    assert bool(((out == lat) | (lat.abs() < 2.0 ** -13 * top)).all())    # exact from there on
    return torch.cat([out, q[..., 512:].double()], -1)


@pytest.mark.parametrize("power", [8, 14, 20])
@pytest.mark.parametrize("fmt", ["bf16", "q8", "q4"])
def test_weights_of_heads_with_one_large_dim(dsa, fmt, power):
    """One dim of each head 2^power times the others, where the cache is zero: over bf16 rows nothing is lost, over the others
    the weights are those of the query as two e4m3 numbers, which are the attention's own."""
    g = gen(power)
    L, N, K = 20, 500, 300
    cache, scale = make_cache(g, fmt, N)
    if fmt == "q4":
        cache[:, 18] &= 0x8F                                              # dim 37: the fifth of group 4
    else:
        cache[:, 37] = 0
    kv = values(fmt, cache, scale)
    assert bool((kv[:, 37] == 0).all())
    q, idx = randn(g, L, 64, 576).bfloat16(), choose(g, [N] * L, N, K)
    q[:, :, 37] = torch.exp2(torch.tensor(float(power), device="cuda")) * (1.0 + torch.rand(L, 64, generator=g, device="cuda"))
    held = q.double() if fmt == "bf16" else as_two_e4m3(q)
    lse, w, bound = weights64(held, lambda s: kv[idx[s].long()], idx, False)
    want, bound = summed(w, idx, N), summed(bound, idx, N)
    got = dsa.mla_key_weights_prefill(q, cache, idx, lse, SCALE, cache_scale=scale)
    assert bool(((got.double() - want).abs() <= bound + 2 * L * L * 2.0 ** -56).all()), float(((got.double() - want).abs() / bound).max())
    if fmt == "bf16":
        _, own = dsa.mla_sparse_attn_prefill(q, cache, idx, SCALE, want_lse=True)
    else:
        _, own = getattr(dsa, f"mla_sparse_attn_prefill_{fmt}")(q, cache, scale, idx, SCALE, want_lse=True)
    acc = dsa.mla_key_weights_prefill(q, cache, idx, own, SCALE, cache_scale=scale)
    # the attention's lse is within 2^-12 of its own scores' (its tests' bound), a factor of every weight
    assert abs(float(acc.double().sum()) - 64 * L) <= 64 * L * 2.0 ** -11
    assert dsa.device_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "q8", "q4"])
def test_weights_of_large_scores(dsa, fmt):
    """Scores of 3000 and a lse next to them: the rounded factors of the exponent, and no more.  All numbers are multiples of 1/64
    that float32 holds, so that nothing else is rounded but the exponential and the sums (below 2^-17 together)."""
    R, N = 4, 64
    j, h = torch.arange(N, device="cuda"), torch.arange(64, device="cuda")
    q = torch.zeros(R, 64, 576, device="cuda")
    q[..., 0], q[..., 512] = 8000.0, 2.0                                  # times 6 and -j: 48000 - 2 j
    rope = torch.zeros(N, 64, device="cuda")
    rope[:, 0] = -j.float()
    if fmt == "bf16":
        cache, scale = torch.zeros(N, 576, device="cuda").bfloat16(), None
        cache[:, 0], cache[:, 512:] = 6.0, rope.bfloat16()
    else:
        cache, scale = torch.zeros(N, 640 if fmt == "q8" else 416, dtype=torch.uint8, device="cuda"), torch.ones(N, device="cuda")
        if fmt == "q8":
            cache[:, 0] = torch.tensor(6.0, device="cuda").to(F8).view(torch.uint8)
        else:
            cache[:, 0], cache[:, 256] = 7, 18                            # magnitude 6, block scale 1
        cache[:, -128:] = rope.bfloat16().view(torch.uint8)
    lse = (3000.0 + h / 64).repeat(R, 1).float()
    idx = j.int().repeat(R, 1)
    one = torch.exp(-j[:, None].double() / 8 - h.double() / 64).sum(1)
    tol = math.expm1(2.0 ** -22 * (3000.0 + 3001.0)) + 2.0 ** -17
    got = dsa.mla_key_weights_prefill(q.bfloat16(), cache, idx, lse, SCALE, cache_scale=scale)
    assert bool(((got.double() / R - one).abs() <= tol * one).all()), float((got.double() / R / one - 1).abs().max())
    got = dsa.mla_key_weights_decode(q[:1].bfloat16(), cache[None], i32(N), idx[:1], lse[:1], SCALE,
                                     cache_scale=None if scale is None else scale[None])
    assert bool(((got[0].double() - one).abs() <= tol * one).all()), float((got[0].double() / one - 1).abs().max())
    assert dsa.device_status() == 0


# ------------------------------------------------------------------------------------------------ moves

def test_moves_of_dense_and_paged_tensors_leave_out_whole_entries(dsa):
    """Where a page of either end lies outside the pool, no tensor moves, so that a key's weight stays with its rows."""
    B, N, page = 2, 64, 16
    g = gen(3)
    acc, pos = torch.rand(B, N, generator=g, device="cuda"), torch.arange(B * N, device="cuda").int().view(B, N).contiguous()
    wide = torch.randint(0, 256, (B, N, 48), generator=g, device="cuda").byte()
    pool, keys = torch.randint(0, 256, (6 * page, 416), generator=g, device="cuda").byte(), randn(g, 6 * page, 128).bfloat16()
    table = i32(0, 1, 2, 99, 3, 4, -1, 5).view(B, 4)
    # of sequence 0: source on a page that is not there, destination on one, a good one, one behind the end, one unused; of 1 alike
    src, dst = i32(50, 20, 21, 64, -1, 40, 50, 17, 51, 1).view(B, 5), i32(2, 49, 3, 5, 6, 3, 33, 4, 5, 64).view(B, 5)
    good = [(0, 21, 3), (1, 17, 4), (1, 51, 5)]
    row = lambda b, j: int(table[b, j // page]) * page + j % page  # noqa: E731
    want = [t.clone() for t in (acc, pos, wide, pool, keys)]
    for b, f, t in good:
        for x, w in zip((acc, pos, wide), want[:3]):
            w[b, t] = x[b, f]
        for x, w in zip((pool, keys), want[3:]):
            w[row(b, t)] = x[row(b, f)]
    dsa.cache_move_rows(src, dst, dense=(acc, pos, wide), paged=(pool, keys), block_table=table, page_size=page)
    assert dsa.device_status() == 7
    for x, w in zip((acc, pos, wide, pool, keys), want):
        assert torch.equal(x, w)


# ------------------------------------------------------------------------------------------------ plan

def test_plan_of_as_many_keys_as_there_may_be(dsa):
    """2^31 - 1 keys of one sequence: sums of places and of block sizes stay in 32 bits."""
    N = 2 ** 31 - 1
    acc, pos = torch.rand(1, N, generator=gen(6), device="cuda"), torch.arange(N, dtype=torch.int32, device="cuda")[None]
    heavy = torch.tensor([3, 5, 2 ** 28 - 1, 2 ** 28, 2 ** 30 + 7, N - 9, N - 8, N - 2], device="cuda")
    acc[0, heavy] = 2.0 + torch.arange(8, device="cuda")
    src, dst, left = dsa.cache_evict_plan(acc, pos, i32(N), 9, recent=1)   # and the last position
    assert src[0].tolist() == [2 ** 28 - 1, 2 ** 28, 2 ** 30 + 7, N - 9, N - 8, N - 2, N - 1, -1, -1]
    assert dst[0].tolist() == [0, 1, 2, 4, 6, 7, 8, -1, -1] and int(left[0]) == 9
    src, dst, left = dsa.cache_evict_plan(acc, pos, i32(N - 6), 7)
    assert src[0].tolist() == [2 ** 28 - 1, 2 ** 28, 2 ** 30 + 7, N - 9, N - 8, -1, -1]
    assert dst[0].tolist() == [0, 1, 2, 4, 6, -1, -1] and int(left[0]) == 7
    assert dsa.device_status() == 0


# ------------------------------------------------------------------------------------------------ tokens after a cut

@pytest.mark.parametrize("fmt,page", [("bf16", 0), ("q8", 64), ("q4", 16)])
def test_tokens_appended_after_a_cut(dsa, fmt, page):
    """A loop of decode steps that appends tokens and cuts the caches three times: indexer, top-k and attention over the cut
    caches give what they give over the same keys in order, and the weights by which a cut goes are those each position
    has received since it came."""
    g = gen(5)
    B, N, P, keep, K = 3, 160, 200, 60, 48
    seq = torch.arange(B, device="cuda")
    everything, every_scale = make_cache(g, fmt, B * P)                   # by positions
    everything, every_scale = everything.view(B, P, -1), None if every_scale is None else every_scale.view(B, P)
    index_keys = randn(g, B, P, 128).bfloat16()
    start = [100, 59, 130]
    kv_len, n_pos = i32(*start), torch.tensor(start, device="cuda")
    if page:
        cache, scale, table, _ = paged(g, everything[:, :N], None if every_scale is None else every_scale[:, :N], [N] * B, page)
        kind = "_paged"
        place = lambda at: table[seq, at // page].long() * page + at % page  # noqa: E731
        paging = {"block_table": table, "page_size": page, "Nmax": N}
    else:
        cache, scale, kind, paging = everything[:, :N].clone(), None if every_scale is None else every_scale[:, :N].clone(), "", {}
    keys = index_keys[:, :N].clone()
    acc, pos = torch.zeros(B, N, device="cuda"), torch.arange(N, device="cuda").int()[None].repeat(B, 1).contiguous()
    acc[:, 50:] = 1e9                                                     # places without a key hold anything
    acc[torch.arange(N, device="cuda") < kv_len[:, None]] = 0.0
    received = torch.zeros(B, P, device="cuda")                           # by positions
    low = "" if fmt == "bf16" else "_" + fmt
    rows = lambda c, s: (c,) if s is None else (c, s)  # noqa: E731
    cuts = 0
    for step in range(30):
        at = kv_len.long()                                                # a token's place
        pos[seq, at], acc[seq, at], keys[seq, at] = n_pos.int(), 0.0, index_keys[seq, n_pos]
        if page:
            cache[place(at)] = everything[seq, n_pos]
            if scale is not None:
                scale[place(at)] = every_scale[seq, n_pos]
        else:
            cache[seq, at] = everything[seq, n_pos]
            if scale is not None:
                scale[seq, at] = every_scale[seq, n_pos]
        n_pos, kv_len = n_pos + 1, kv_len + 1
        q, q_idx, w = randn(g, B, 64, 576).bfloat16(), randn(g, B, 1, 32, 128).bfloat16(), randn(g, B, 1, 32)
        last = kv_len - 1
        idx = dsa.topk(dsa.indexer_scores(q_idx, keys, w, last, kv_len), last, kv_len, N, K)[:, 0].contiguous()
        named = torch.where(idx >= 0, pos.gather(1, idx.clamp(min=0).long()), -1).contiguous()
        # the keys that are left, in the order of their positions
        held = torch.where(torch.arange(N, device="cuda") < kv_len[:, None], pos, 1 << 20).sort(1).values
        ordered = index_keys[seq[:, None], held.clamp(max=P - 1).long()].contiguous()
        first = dsa.topk(dsa.indexer_scores(q_idx, ordered, w, last, kv_len), last, kv_len, N, K)[:, 0]
        assert torch.equal(torch.where(first >= 0, held.gather(1, first.clamp(min=0).long()).int(), -1).sort(1).values, named.sort(1).values)
        head = (q, *rows(cache, scale), kv_len) + ((table, page) if page else ()) + (idx, SCALE) + ((N,) if page else ())
        out, lse = getattr(dsa, f"mla_sparse_attn_decode{low}{kind}")(*head, want_lse=True)
        whole = getattr(dsa, f"mla_sparse_attn_decode{low}")(q, *rows(everything, every_scale), i32(*[P] * B), named, SCALE, want_lse=True)
        assert torch.equal(out, whole[0]) and torch.equal(lse, whole[1])
        dsa.mla_key_weights_decode(q, cache, kv_len, idx, lse, SCALE, acc=acc, cache_scale=scale, **paging)
        received += dsa.mla_key_weights_decode(q, everything, i32(*[P] * B), named, lse, SCALE, cache_scale=every_scale)
        mine = torch.arange(N, device="cuda") < kv_len[:, None]
        tracked = received.gather(1, pos.long().clamp(0, P - 1))
        assert torch.equal(acc[mine], tracked[mine])
        if step % 10 == 7:
            want = plan_by_sorting(tracked.cpu(), pos.cpu(), kv_len.cpu(), keep, 8, 2)
            src, dst, left = dsa.cache_evict_plan(acc, pos, kv_len, keep, recent=8, sink=2)
            assert all(torch.equal(x.cpu(), y) for x, y in zip((src, dst, left), want))
            latent = [cache] + ([] if scale is None else [scale])
            if page:
                dsa.cache_move_rows(src, dst, dense=(acc, pos, keys), paged=latent, block_table=table, page_size=page)
            else:
                dsa.cache_move_rows(src, dst, dense=[acc, pos, keys] + latent)
            kv_len, cuts = left, cuts + 1
        assert dsa.device_status() == 0
    assert cuts == 3


# ------------------------------------------------------------------------------------------------ calls at once

def test_calls_of_three_threads_at_once(dsa):
    """Attention over the 4-bit cache, weights, plans and moves by three threads on a stream each give the bits of the same
    calls one after the other."""
    work = []
    for t in range(3):
        g = gen(40 + t)
        L, B, N, K, keep = 170 + t, 5, 900 + 70 * t, 300, 400
        cache, scale = make_cache(g, "q4", B * N)
        q, idx = randn(g, L, 64, 576).bfloat16(), choose(g, [N] * L, N, K)
        one, few, kv_len = randn(g, B, 64, 576).bfloat16(), choose(g, [N - 50 * b for b in range(B)], N, K), i32(*[N - 50 * b for b in range(B)])
        acc, pos = torch.rand(B, N, generator=g, device="cuda"), torch.rand(B, N, generator=g, device="cuda").argsort(1).int()

        def calls(cache=cache, scale=scale, q=q, idx=idx, one=one, few=few, kv_len=kv_len, acc=acc, pos=pos, B=B, N=N, keep=keep):
            out, lse = dsa.mla_sparse_attn_prefill_q4(q, cache[:N], scale[:N], idx, SCALE, want_lse=True)
            batch, bscale = cache.view(B, N, -1), scale.view(B, N)
            out1, lse1 = dsa.mla_sparse_attn_decode_q4(one, batch, bscale, kv_len, few, SCALE, want_lse=True)
            w = dsa.mla_key_weights_prefill(q, cache[:N], idx, lse, SCALE, cache_scale=scale[:N])
            w1 = dsa.mla_key_weights_decode(one, batch, kv_len, few, lse1, SCALE, cache_scale=bscale)
            src, dst, left = dsa.cache_evict_plan(acc, pos, kv_len, keep, recent=20, sink=2)
            moved = [acc.clone(), pos.clone(), batch.clone(), bscale.clone()]
            dsa.cache_move_rows(src, dst, dense=moved)
            return [out, lse, out1, lse1, w, w1, src, dst, left] + moved

        work.append((calls, calls()))
    torch.cuda.synchronize()
    wrong = []

    def repeat(calls, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(60):
                    got = calls()
                    wrong.extend(i for i, (x, y) in enumerate(zip(got, want)) if not torch.equal(x, y))
        except Exception as error:                                        # for the thread that asserts
            wrong.append(error)

    threads = [threading.Thread(target=repeat, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and dsa.device_status() == 0
