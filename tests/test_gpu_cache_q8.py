"""The 8-bit latent cache (write, read back, attention over it) and the indexer's input pass on the
GPU, against plain float64 implementations written here.

Tolerances, from the arithmetic:

* codes: the kernel's value of u * 2^-k, in pairs of floats, is within about 2^-44 (relative) of the exact one;
  test_write_codes_are_the_nearest holds it to that.  Elsewhere 2^-20, what a float32 chain (a sum of 512 squares, one
  rsqrt, two products) would need, is allowed: |code - value| <= half a step, and 2^-20 |value| more.
* bf16 outputs of the norms and rotations: half a step, 2^-8 |value|, and 2^-18 of the pair's length for the
  float32 arithmetic before it (the turned value may cancel).  Below 2^-126 a bf16 step is 2^-133 whatever the
  value, so half of it, 2^-134, comes on top there.
* attention, per element: the probabilities enter the value product as hi + lo / 16 in e4m3: relative error at
  most 2^-4 2^-4 = 2^-8 each, so |out - ref| <= 2^-8 A with A = sum_t p_t |v_t|; the float32 logits (576 products
  and their sum, the scale, the exponent) and sums add at most 2^-12 A for the data here.  Small weights are held
  to half of lo's last step, 2^-9 / 16 / 2 = 2^-14, where the largest weight of the head is at least 2^4.5:
  2^-18.5 of it a key, 2^-7.5 max_t |v_t| for 2048 keys.  A bf16 output adds 2^-8 |ref|.  For normal data the
  framework's bound holds as well: max|err| <= 1e-2 max|ref|, sum|err| <= 2e-3 sum|ref|.
* lse: float32 logits and sums: 2^-12 absolute for logits of a few tens.  Where a logit's 576 terms sum to S in
  absolute value (S in the hundreds), its float32 sum is off by at most d = 576 * 2^-24 S, whatever the order
  (each of the additions rounds a partial sum of at most S by 2^-24): lse by d, each probability, and so the
  output, by a factor e^(2 d): (e^(2 d) - 1) A more.
"""
import math
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
SCALE = 1.0 / 16.0


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


def angles(n):
    f = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def turned(x, cs, interleave):
    """x [R, H, 64] float64 with its 32 pairs turned; and each element's pair length."""
    c, s = cs[:, None, :32].double(), cs[:, None, 32:].double()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleave else (x[..., :32], x[..., 32:])
    u, v, n = a * c - b * s, b * c + a * s, torch.hypot(a, b)
    if interleave:
        return torch.stack([u, v], -1).flatten(-2), torch.stack([n, n], -1).flatten(-2)
    return torch.cat([u, v], -1), torch.cat([n, n], -1)


def make_cache(g, rows, exponents=0, amp=1.0):
    """An 8-bit cache: codes of normal data, scales 2^k with k spread over +-exponents."""
    cache = torch.empty(rows, 640, dtype=torch.uint8, device="cuda")
    cache[:, :512] = (randn(g, rows, 512) * 64.0).to(F8).view(torch.uint8)
    cache[:, 512:] = randn(g, rows, 64).bfloat16().view(torch.uint8)
    k = torch.randint(-exponents, exponents + 1, (rows,), generator=g, device="cuda") if exponents else torch.zeros(rows, device="cuda")
    return cache, torch.exp2(k.float() - 6.0) * amp


def values(cache, scale):
    """Float64 rows [.., 576]."""
    lat = cache[..., :512].contiguous().view(F8).double() * scale[..., None].double()
    return torch.cat([lat, cache[..., 512:].contiguous().view(torch.bfloat16).double()], -1)


def paged(g, cache, scale, lens, page, extra=3):
    """Dense [B, N] rows laid out over a shuffled pool; junk (NaN rows) everywhere no sequence has a key."""
    B, N = scale.shape
    used = [-(-n // page) for n in lens]
    pages = sum(used) + extra
    perm = torch.randperm(pages, generator=g, device="cuda")
    pool = torch.full((pages * page, 640), 0x7F, dtype=torch.uint8, device="cuda")
    pscale = torch.full((pages * page,), math.nan, device="cuda")
    table = torch.full((B, -(-N // page)), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        for lp in range(used[b]):
            pg = int(perm[at])
            at += 1
            table[b, lp] = pg
            m = min(page, n - lp * page)
            pool[pg * page:pg * page + m] = cache[b, lp * page:lp * page + m]
            pscale[pg * page:pg * page + m] = scale[b, lp * page:lp * page + m]
    return pool, pscale, table, pages


# ------------------------------------------------------------------------------------------------ write

def check_written(kv_a, w, eps, cs, interleave, codes, rope, scale):
    """The rows' contents against the formula in float64."""
    x = kv_a.double()
    c = x[:, :512]
    u = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * w.double()
    big = u.abs().amax(1)
    want = torch.exp2(torch.ceil(torch.log2(big / 448.0)).clamp(-64, 64))
    # u is a float32: below half of its smallest step, 2^-150, a row is one of zeros
    want = torch.where(big < 2.0 ** -150, torch.ones_like(want), want)
    border = torch.log2(big.clamp(min=1e-300) / 448.0)
    near = (border - border.round()).abs() < 2.0 ** -19                 # a float32 maximum could fall on either side
    sc = scale.double()
    assert bool(((sc == want) | (near & ((sc == 2 * want) | (2 * sc == want)))).all())
    v = (u / sc[:, None]).clamp(-448, 448)
    got = codes.double()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    assert bool(((got - v).abs() <= step / 2 + 2.0 ** -20 * v.abs()).all())
    r, n = turned(x[:, None, 512:], cs, interleave)
    assert bool(((rope.double()[:, None] - r).abs() <= 2.0 ** -8 * r.abs() + 2.0 ** -18 * n + 2.0 ** -134).all())


@pytest.mark.parametrize("R,ld,interleave", [(1, 576, True), (3, 584, False), (8, 2048, True), (33, 576, False),
                                             (1000, 640, True), (4100, 576, True)])
def test_write(dsa, R, ld, interleave):
    g = gen(R)
    rows, eps = 2 * R + 5, 1e-6
    kv_a = (randn(g, R, ld) * torch.exp(2 * randn(g, R, 1))).bfloat16()[:, :576]
    w = torch.exp(randn(g, 512))
    cs = angles(5000)
    pos = torch.randint(0, 5000, (R,), generator=g, device="cuda").int()
    slots = torch.randperm(rows, generator=g, device="cuda")[:R].int()
    if R > 4:
        slots[R // 2] = -1
        slots[R - 1] = -1000
        pos[R - 1] = -5                                                   # a padding token's position is not looked at
        kv_a[R // 3] = 0.0                                                # scale 1, codes 0
    cache = torch.randint(0, 256, (rows, 640), generator=g, device="cuda").byte()
    scale = torch.rand(rows, generator=g, device="cuda")
    before, sbefore = cache.clone(), scale.clone()
    dsa.mla_cache_write_q8(kv_a, w, eps, cs, pos, slots, cache, scale, interleave=interleave)
    assert dsa.device_status() == 0
    kept = slots >= 0
    to = slots[kept].long()
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[to] = False
    assert torch.equal(cache[rest], before[rest]) and torch.equal(scale[rest], sbefore[rest])
    check_written(kv_a[kept], w, eps, cs[pos[kept].long()], interleave, cache[to, :512].view(F8),
                  cache[to, 512:].contiguous().view(torch.bfloat16), scale[to])


def test_write_codes_are_the_nearest(dsa):
    """Every code is the e4m3 number nearest the formula's value: the kernel's pairs of floats are off by about 2^-44,
    the float64 reference by 2^-50, so only a value within 2^-40 of a midpoint could go either way."""
    g = gen(24)
    R = 4096
    kv_a, w = randn(g, R, 576).bfloat16(), torch.exp(0.3 * randn(g, 512))
    cs = angles(4)
    zero, slots = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.arange(R, dtype=torch.int32, device="cuda")
    cache, scale = torch.zeros(R, 640, dtype=torch.uint8, device="cuda"), torch.zeros(R, device="cuda")
    eps = 2.0 ** -20                                                      # a float32 number
    dsa.mla_cache_write_q8(kv_a, w, eps, cs, zero, slots, cache, scale)
    x = kv_a[:, :512].double()
    u = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * w.double()
    k = torch.exp2(torch.ceil(torch.log2(u.abs().amax(1) / 448.0)))
    assert torch.equal(scale.double(), k)
    v = u / k[:, None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    near = ((v / step).frac().abs() - 0.5).abs() * step <= 2.0 ** -40 * v.abs()
    want = torch.round(v / step) * step
    got = cache[:, :512].contiguous().view(F8).double()
    assert bool(((got == want) | near).all()) and int(near.sum()) < 10


def test_write_extremes(dsa):
    """Tiny, huge and zero rows; weights that reach the scale's clamps and saturate past them."""
    g = gen(5)
    amp = torch.tensor([0.0, 1e-38, 1e-20, 1.0, 1e15, 0.0], device="cuda")
    kv_a = (randn(g, 6, 576) * amp[:, None]).bfloat16()
    kv_a[5, 7] = 2.0 ** -60
    cs = angles(4)
    pos = torch.tensor([0, 1, 2, 3, 0, 1], dtype=torch.int32, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    for w in (1.0, 2.0 ** -60, 2.0 ** 60, 2.0 ** 80):
        wt = torch.full((512,), w, device="cuda")
        cache = torch.zeros(6, 640, dtype=torch.uint8, device="cuda")
        scale = torch.zeros(6, device="cuda")
        dsa.mla_cache_write_q8(kv_a, wt, 1e-6, cs, pos, slots, cache, scale)
        check_written(kv_a, wt, 1e-6, cs[pos.long()], True, cache[:, :512].view(F8),
                      cache[:, 512:].contiguous().view(torch.bfloat16), scale)
        assert bool((scale >= 2.0 ** -64).all()) and bool((scale <= 2.0 ** 64).all())


def test_write_records_what_is_out_of_range(dsa):
    g = gen(6)
    kv_a = randn(g, 4, 576).bfloat16()
    cs = angles(10)
    w = torch.ones(512, device="cuda")
    for pos, slots in (([1, 10, 2, 3], [0, 1, 2, 3]), ([1, -1, 2, 3], [0, 1, 2, 3]), ([1, 1, 2, 3], [0, 9, 2, 3])):
        cache = torch.full((9, 640), 17, dtype=torch.uint8, device="cuda")
        scale = torch.full((9,), 3.0, device="cuda")
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        dsa.mla_cache_write_q8(kv_a, w, 1e-6, cs, i32(pos), i32(slots), cache, scale)
        assert dsa.device_status() == 7
        assert bool((cache[[1, 4, 8]] == 17).all()) and bool((scale[[1, 4, 8]] == 3.0).all())
        to = torch.tensor([0, 2, 3], device="cuda")
        check_written(kv_a[to], w, 1e-6, cs[i32(pos)[to].long()], True, cache[to, :512].view(F8),
                      cache[to, 512:].contiguous().view(torch.bfloat16), scale[to])


# ------------------------------------------------------------------------------------------------ read back

@pytest.mark.parametrize("R", [1, 2, 9, 500, 10007])
def test_read_by_slot(dsa, R):
    g = gen(R)
    rows = R + 50
    cache, scale = make_cache(g, rows, exponents=20)
    slots = torch.randint(-2, rows, (R,), generator=g, device="cuda").int()
    out = dsa.mla_cache_read_q8(cache, scale, slots)
    want = values(cache, scale)[slots.clamp(min=0).long()]
    want[slots < 0] = 0.0
    assert torch.equal(out.double(), want)                               # exact: power-of-two scales
    assert dsa.device_status() == 0
    odd = scale * 1.37                                                    # any scale: one rounding, to the nearest bf16
    out = dsa.mla_cache_read_q8(cache, odd, slots)
    want = (cache[:, :512].view(F8).float() * odd[:, None]).bfloat16()[slots.clamp(min=0).long()]
    want[slots < 0] = 0.0
    assert torch.equal(out[:, :512], want)
    slots[R // 2] = rows
    out = dsa.mla_cache_read_q8(cache, scale, slots)
    assert dsa.device_status() == 7 and bool((out[R // 2] == 0).all())


@pytest.mark.parametrize("lens,N,page", [([1], 1, 16), ([0, 5, 64, 63], 64, 64), ([300, 0, 17, 299, 1], 300, 16),
                                         ([4096, 4000], 4100, 256)])
def test_read_paged(dsa, lens, N, page):
    g = gen(N)
    B = len(lens)
    cache, scale = make_cache(g, B * N, exponents=8)
    cache, scale = cache.view(B, N, 640), scale.view(B, N)
    pool, pscale, table, pages = paged(g, cache, scale, lens, page)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((B, N, 576), -3.0, dtype=torch.bfloat16, device="cuda")
    dsa.mla_cache_read_q8_paged(pool, pscale, kv_len, table, page, N, out=out)
    assert dsa.device_status() == 0
    want = values(cache, scale)
    for b, n in enumerate(lens):
        assert torch.equal(out[b, :n].double(), want[b, :n])
        assert bool((out[b, n:] == -3.0).all())
    fresh = dsa.mla_cache_read_q8_paged(pool, pscale, kv_len, table, page, N)
    assert all(bool((fresh[b, n:] == 0).all()) for b, n in enumerate(lens))
    b = max(range(B), key=lambda i: lens[i])
    if lens[b]:
        table[b, 0] = pages                                               # a page outside the pool: zeros, recorded
        out = dsa.mla_cache_read_q8_paged(pool, pscale, kv_len, table, page, N)
        n = min(page, lens[b])
        assert dsa.device_status() == 7 and bool((out[b, :n] == 0).all())
        assert torch.equal(out[b, n:lens[b]].double(), want[b, n:lens[b]])


# ------------------------------------------------------------------------------------------------ indexer inputs

@pytest.mark.parametrize("R,norm,q_norm,bias,interleave,strided",
                         [(1, "layer", False, True, True, False), (3, "rms", True, False, False, True),
                          (17, "layer", True, True, False, False), (100, "rms", False, False, True, True),
                          (1025, "layer", False, True, True, False), (2, None, False, False, True, False)])
def test_norm_rope(dsa, R, norm, q_norm, bias, interleave, strided):
    g = gen(R)
    rows = R + 7
    wide = (4.0 * randn(g, R, 4096 + 256) + 1.0).bfloat16()
    if strided:
        q, k = wide[:, :4096].unflatten(1, (32, 128)), wide[:, 4096 + 64:4096 + 192]
    else:
        q, k = wide[:, :4096].reshape(R, 32, 128).contiguous(), wide[:, 4096:4224].contiguous()
    weight = lambda: torch.exp(0.5 * randn(g, 128))                       # noqa: E731
    k_w = weight() if norm else None
    q_w = weight() if q_norm else None
    k_b = 0.3 * randn(g, 128) if bias else None
    q_b = 0.3 * randn(g, 128) if bias and q_norm else None
    cs = angles(700)
    pos = torch.randint(0, 700, (R,), generator=g, device="cuda").int()
    slots = torch.randperm(rows, generator=g, device="cuda")[:R].int()
    if R > 2:
        slots[1] = -1
    k_cache = torch.full((rows, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    eps = 1e-5
    out = dsa.indexer_norm_rope(q, k, k_w, k_b, eps, cs, pos, slots, k_cache, q_w=q_w, q_b=q_b, norm=norm or "rms",
                                interleave=interleave)
    assert dsa.device_status() == 0

    def ref(x, w, b):
        x = x.double()
        size = x.abs()
        if w is not None:
            if norm == "layer":
                x = x - x.mean(-1, keepdim=True)
            f = w.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
            size, x = size * f.abs(), x * f
        if b is not None:
            x = x + b.double()
            size = size + b.double().abs()
        t, n = turned(x[..., :64], cs[pos.long()], interleave)
        # the terms a result is summed from: the pair's two elements, the mean's part of each, the bias
        s = size[..., :64]
        pair = (s.unflatten(-1, (32, 2)).sum(-1).repeat_interleave(2, -1) if interleave
                else s.unflatten(-1, (2, 32)).sum(-2).repeat(*[1] * (s.dim() - 1), 2))
        mean = size.mean(-1, keepdim=True)
        return torch.cat([t, x[..., 64:]], -1), torch.cat([pair, size[..., 64:]], -1) + 2 * mean

    def near(got, want, size):
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * size).all())

    near(out, *ref(q, q_w, q_b))
    kept = slots >= 0
    want, size = ref(k[:, None], k_w, k_b)
    near(k_cache[slots[kept].long()], want[kept, 0], size[kept, 0])
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[slots[kept].long()] = False
    assert bool((k_cache[rest] == 5.0).all())
    if not strided:                                                       # in place
        again = q.clone()
        dsa.indexer_norm_rope(again, k, k_w, k_b, eps, cs, pos, slots, k_cache, q_w=q_w, q_b=q_b, norm=norm or "rms",
                              interleave=interleave, q_out=again)
        assert torch.equal(again, out)


def test_norm_rope_records_what_is_out_of_range(dsa):
    g = gen(8)
    q, k = randn(g, 3, 32, 128).bfloat16(), randn(g, 3, 128).bfloat16()
    cs = angles(10)
    w = torch.ones(128, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")    # noqa: E731
    good = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    want = dsa.indexer_norm_rope(q, k, w, None, 1e-6, cs, i32(1, 2, 3), i32(0, 1, 2), good)
    for pos, slots in ((i32(1, 10, 3), i32(0, 1, 2)), (i32(1, -1, 3), i32(0, 1, 2)), (i32(1, 2, 3), i32(0, 4, 2))):
        cache = torch.zeros_like(good)
        out = torch.full_like(q, 9.0)
        dsa.indexer_norm_rope(q, k, w, None, 1e-6, cs, pos, slots, cache, q_out=out)
        assert dsa.device_status() == 7
        assert torch.equal(out[[0, 2]], want[[0, 2]]) and torch.equal(cache[[0, 2]], good[[0, 2]])
        assert bool((cache[[1, 3]] == 0).all())
        assert bool((out[1] == 9.0).all()) == (int(slots[1]) == 1)


# ------------------------------------------------------------------------------------------------ attention

def attention64(q, rows, have, scale):
    """(out, lse, A, vmax) in float64: q [R, 64, 576], rows [R, K, 576], have [R, K]."""
    out, lse, A, vm = [], [], [], []
    for i in range(0, q.shape[0], 32):
        kv, ok = rows(slice(i, i + 32)), have[i:i + 32]
        kv = torch.where(ok[..., None], kv, torch.zeros_like(kv))
        x = torch.einsum("rhd,rkd->rhk", q[i:i + 32].double(), kv) * scale
        x = torch.where(ok[:, None], x, -math.inf)
        p = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
        v = kv[..., :512]
        out.append(p @ v)
        A.append(p @ v.abs())
        lse.append(torch.logsumexp(x, -1))
        vm.append(v.abs().amax(1, keepdim=True).expand(-1, 64, -1))
    return torch.cat(out), torch.cat(lse), torch.cat(A), torch.cat(vm)


def close(got, lse, ref, normal=True, S=0.0):
    out, l64, A, vm = ref
    err = (got.double() - out).abs()
    d = 576 * 2.0 ** -24 * S
    bound = (2.0 ** -8 + 2.0 ** -12 + math.expm1(2 * d)) * A + 2.0 ** -7.5 * vm
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * out.abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())
    if normal:
        assert float(err.max()) <= 1e-2 * float(out.abs().max())
        assert float(err.sum()) <= (2e-3 if got.dtype == torch.float32 else 4e-3) * float(out.abs().sum())
    if lse is not None:
        dead = torch.isneginf(l64)
        assert torch.equal(torch.isneginf(lse), dead)
        assert bool(((lse.double() - l64).abs()[~dead] <= 2.0 ** -12 + d).all())


def choose(g, counts, N, top_k):
    """Ascending random selections of min(top_k, count) keys, -1 padded."""
    R = len(counts)
    c = torch.tensor(counts, device="cuda")
    r = torch.rand(R, N, generator=g, device="cuda")
    r.masked_fill_(torch.arange(N, device="cuda")[None] >= c[:, None], -1.0)
    val, idx = r.topk(min(top_k, N), 1)
    idx = idx.masked_fill(val < 0, N).sort(1).values
    idx = idx.masked_fill(idx == N, -1).int()
    return torch.nn.functional.pad(idx, (0, top_k - idx.shape[1]), value=-1).contiguous()


DECODE = [(1, 1, 1, 0), (1, 4096, 2048, 0), (2, 130, 129, 16), (5, 1000, 2048, 64), (8, 4096, 2048, 64), (3, 700, 127, 0),
          (37, 515, 400, 16), (170, 300, 256, 0), (40, 2500, 2048, 256)]


@pytest.mark.parametrize("B,N,top_k,page", DECODE)
def test_decode(dsa, B, N, top_k, page):
    g = gen(B * N)
    lens = [N if b == 0 else (b * 7919) % (N + 1) for b in range(B)]      # every length from none on
    cache, scale = make_cache(g, B * N, exponents=2)
    cache, scale = cache.view(B, N, 640), scale.view(B, N)
    idx = choose(g, lens, N, top_k)
    q = randn(g, B, 64, 576).bfloat16()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kv = values(cache, scale)
    ref = attention64(q, lambda s: torch.stack([kv[b][idx[b].clamp(min=0).long()] for b in range(B)[s]]), idx >= 0, SCALE)
    if page:
        pool, pscale, table, _ = paged(g, cache, scale, lens, page)
        call = lambda **k: dsa.mla_sparse_attn_decode_q8_paged(q, pool, pscale, kv_len, table, page, idx, SCALE, N,   # noqa: E731
                                                               want_lse=True, **k)
    else:
        call = lambda **k: dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, idx, SCALE, want_lse=True, **k)     # noqa: E731
    out, lse = call()
    assert dsa.device_status() == 0
    close(out, lse, ref)
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((out[b] == 0).all())
    o16, l16 = call(out_dtype=torch.bfloat16)
    assert torch.equal(o16, out.bfloat16()) and torch.equal(l16, lse)     # the float32 result, rounded


PREFILL = [(1, 1, 1, 0), (1, 64, 64, 16), (64, 1024, 256, 0), (37, 1000, 100, 64), (300, 300, 128, 0), (200, 2300, 2048, 16),
           (333, 5001, 2048, 64)]


@pytest.mark.parametrize("L,N,top_k,page", PREFILL)
def test_prefill(dsa, L, N, top_k, page):
    g = gen(L + N)
    cache, scale = make_cache(g, N, exponents=2)
    idx = choose(g, [N - L + i + 1 for i in range(L)], N, top_k)
    if L > 3:
        idx[L // 2] = -1                                                  # nothing selected
        idx[1] = idx[1][torch.randperm(top_k, generator=g, device="cuda")]   # any order, -1 between
    q = randn(g, L, 64, 576).bfloat16()
    kv = values(cache, scale)
    ref = attention64(q, lambda s: kv[idx[s].clamp(min=0).long()], idx >= 0, SCALE)
    if page:
        pool, pscale, table, _ = paged(g, cache[None], scale[None], [N], page)
        out, lse = dsa.mla_sparse_attn_prefill_q8_paged(q, pool, pscale, table[0], page, idx, SCALE, N, want_lse=True)
    else:
        out, lse = dsa.mla_sparse_attn_prefill_q8(q, cache, scale, idx, SCALE, want_lse=True)
    assert dsa.device_status() == 0
    close(out, lse, ref)
    if not page:                                                          # the bf16 calls over the rows read back
        back = dsa.mla_cache_read_q8(cache, scale, torch.arange(N, dtype=torch.int32, device="cuda"))
        other = dsa.mla_sparse_attn_prefill(q, back, idx, SCALE)
        err = (out - other).abs().double()
        assert float(err.sum()) <= 4e-3 * float(ref[0].abs().sum())


def one_row(dsa, q, cache, scale, idx, sm=SCALE, large=False):
    kv = values(cache, scale)
    S = float(torch.einsum("rhd,kd->rhk", q.double().abs(), kv[idx[idx >= 0].long().unique()].abs()).max()) * sm if large else 0.0
    ref = attention64(q, lambda s: kv[idx[s].clamp(min=0).long()], idx >= 0, sm)
    out, lse = dsa.mla_sparse_attn_prefill_q8(q, cache, scale, idx, sm, want_lse=True)
    close(out, lse, ref, normal=False, S=S)
    # as many rows as SMs: whole queries, tile after tile, where the few rows above are cut into parts
    R = idx.shape[0]
    many = torch.arange(torch.cuda.get_device_properties(0).multi_processor_count, device="cuda") % R
    assert dsa.attn_q8_workspace_size(len(many), idx.shape[1]) == 0
    out2, lse2 = dsa.mla_sparse_attn_prefill_q8(q[many].contiguous(), cache, scale, idx[many].contiguous(), sm, want_lse=True)
    close(out2[:R], lse2[:R], ref, normal=False, S=S)
    assert torch.equal(out2, out2[:R][many]) and torch.equal(lse2, lse2[:R][many])
    return out, lse, ref


def test_attention_peaked_and_growing_scores(dsa):
    """Scores that grow from tile to tile (the running maximum moves each time), one outlier over a flat
    rest, and heads of all zeros."""
    g = gen(11)
    N = 1024
    cache, scale = make_cache(g, N)
    idx = torch.arange(N, dtype=torch.int32, device="cuda")[None].repeat(3, 1).contiguous()
    rope = torch.zeros(N, 64, device="cuda")
    rope[:, 0] = torch.arange(N, device="cuda") / 16.0                    # grows by 8 a 128-key tile
    rope[:, 1] = torch.arange(N, 0, -1, device="cuda") / 16.0
    rope[700, 2] = 256.0
    cache[:, 512:] = rope.bfloat16().view(torch.uint8)
    q = torch.zeros(3, 64, 576, device="cuda")
    q[0, :, 512] = torch.arange(64, device="cuda") / 4.0                  # 0 .. 15.75: up to 63 / tile, after the scale 8
    q[1, :, 513] = 16.0
    q[2, :, 514] = torch.arange(64, device="cuda") / 32.0                 # the outlier's weight: e^0 .. e^31
    q = q.bfloat16()
    out, lse, ref = one_row(dsa, q, cache, scale, idx)
    back = idx.flip(1).contiguous()
    one_row(dsa, q, cache, scale, back)


def test_attention_scales_far_apart(dsa):
    """Rows whose scales span 2^-40 .. 2^40: values and logits of every size, some rows of zeros."""
    g = gen(12)
    N = 600
    cache, scale = make_cache(g, N)
    k = torch.randint(-40, 41, (N,), generator=g, device="cuda").float()
    scale = torch.exp2(k)
    cache[::7, :512] = 0
    idx = choose(g, [N] * 4, N, 500)
    q = torch.zeros(4, 64, 576, device="cuda")
    q[:, :, 512:] = randn(g, 4, 64, 64)                                   # logits from the rope dims alone
    q = q.bfloat16()
    one_row(dsa, q, cache, scale, idx)
    odd = torch.exp2(k / 8.0) * 1.3                                       # scales that are no powers of two
    q = (0.02 * randn(g, 4, 64, 576)).bfloat16()
    one_row(dsa, q, cache, odd, idx, large=True)


def test_attention_query_of_every_size(dsa):
    """Query heads from 2^-30 to 2^6, dims of one head 2^20 apart, and a head of zeros."""
    g = gen(13)
    N = 300
    cache, scale = make_cache(g, N)
    idx = choose(g, [N] * 2, N, 256)
    q = randn(g, 2, 64, 576) * torch.exp2(torch.linspace(-30, 3, 64, device="cuda"))[None, :, None]
    q[1] = q[1] * torch.exp2(-torch.randint(0, 20, (64, 576), generator=g, device="cuda").float())
    q[:, 5] = 0.0
    one_row(dsa, q.bfloat16(), cache, scale, idx)


def test_attention_reads_only_selected_rows(dsa):
    """NaN rows that nothing selects, a first tile of padding, the same key selected many times."""
    g = gen(14)
    N = 400
    cache, scale = make_cache(g, N)
    idx = torch.full((3, 300), -1, dtype=torch.int32, device="cuda")
    idx[0, 200:] = torch.arange(100, 200, device="cuda").int()
    idx[1, ::3] = 7
    idx[1, 1] = 9
    idx[2, 299] = 399
    q = randn(g, 3, 64, 576).bfloat16()
    want = one_row(dsa, q, cache, scale, idx)
    used = torch.zeros(N, dtype=torch.bool, device="cuda")
    used[idx[idx >= 0].long()] = True
    bad, bscale = cache.clone(), scale.clone()
    bad[~used] = 0x7F                                                     # NaN codes, NaN rope
    bscale[~used] = math.nan
    out, lse = dsa.mla_sparse_attn_prefill_q8(q, bad, bscale, idx, SCALE, want_lse=True)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_attention_records_keys_outside_the_cache(dsa):
    g = gen(15)
    B, N, K = 3, 200, 150
    cache, scale = make_cache(g, B * N)
    cache, scale = cache.view(B, N, 640), scale.view(B, N)
    lens = [200, 120, 0]
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    idx = choose(g, lens, N, K)
    q = randn(g, B, 64, 576).bfloat16()
    good = dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, idx, SCALE)
    assert dsa.device_status() == 0
    bad = idx.clone()
    bad[1, K - 1] = 120                                                   # at kv_len: skipped, recorded
    bad[2, 3] = 2 ** 31 - 1
    out = dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, bad, SCALE)
    assert dsa.device_status() == 7
    assert torch.allclose(out, good, rtol=0, atol=2.0 ** -8 * float(good.abs().max()))
    assert bool((out[2] == 0).all())
    pool, pscale, table, pages = paged(g, cache, scale, lens, 64)
    table[0, 1] = pages                                                   # keys 64..127 of sequence 0 read as zeros
    out, lse = dsa.mla_sparse_attn_decode_q8_paged(q, pool, pscale, kv_len, table, 64, idx, SCALE, N, want_lse=True)
    assert dsa.device_status() == 7
    kv = values(cache, scale)
    kv[0, 64:128] = 0
    ref = attention64(q, lambda s: torch.stack([kv[b][idx[b].clamp(min=0).long()] for b in range(B)[s]]), idx >= 0, SCALE)
    close(out, lse, ref, normal=False)


def test_offsets_past_32_bits(dsa):
    """Rows at the far end of a cache of more than 2^32 bytes: written, read back and attended to."""
    rows = 6836 * 1024                                                    # 4.48 GB
    cache = torch.zeros(rows, 640, dtype=torch.uint8, device="cuda")
    scale = torch.ones(rows, device="cuda")
    g = gen(16)
    R = 300
    kv_a, w, cs = randn(g, R, 576).bfloat16(), torch.ones(512, device="cuda"), angles(16)
    pos = torch.zeros(R, dtype=torch.int32, device="cuda")
    slots = (rows - 1 - 3 * torch.arange(R, device="cuda")).int()
    dsa.mla_cache_write_q8(kv_a, w, 1e-6, cs, pos, slots, cache, scale)
    check_written(kv_a, w, 1e-6, cs[pos.long()], True, cache[slots.long(), :512].view(F8),
                  cache[slots.long(), 512:].contiguous().view(torch.bfloat16), scale[slots.long()])
    back = dsa.mla_cache_read_q8(cache, scale, slots)
    assert torch.equal(back.double(), values(cache[slots.long()], scale[slots.long()]))
    idx = slots.flip(0)[None].contiguous()
    q = randn(g, 1, 64, 576).bfloat16()
    out, lse = dsa.mla_sparse_attn_prefill_q8(q, cache, scale, idx, SCALE, want_lse=True)
    kv = values(cache[idx[0].long()], scale[idx[0].long()])[None]
    close(out, lse, attention64(q, lambda s: kv[s], idx >= 0, SCALE))
    page = 1024
    pages = rows // page
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    base = (pages - 1) * page
    local = (slots[(slots >= base) & (slots < base + page)] - base).sort().values
    out = dsa.mla_sparse_attn_decode_q8_paged(q, cache, scale, torch.tensor([page], dtype=torch.int32, device="cuda"), table,
                                              page, local[None].contiguous(), SCALE, page)
    at = local.long() + base
    kv = values(cache[at], scale[at])[None]
    close(out, None, attention64(q, lambda s: kv[s], local[None] >= 0, SCALE))
    assert dsa.device_status() == 0


# ------------------------------------------------------------------------------------------------ streams, graphs, refusals

def test_streams_and_graphs(dsa):
    """The same decode step eagerly, on two streams at once, and captured and replayed on new inputs:
    the same bits."""
    g = gen(17)
    B, N, K = 6, 900, 512
    cache, scale = make_cache(g, B * N)
    cache, scale = cache.view(B, N, 640), scale.view(B, N)
    kv_len = torch.full((B,), N, dtype=torch.int32, device="cuda")
    qs = [randn(g, B, 64, 576).bfloat16() for _ in range(4)]
    ids = [choose(g, [N] * B, N, K) for _ in range(4)]
    want = [dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, i, SCALE) for q, i in zip(qs, ids)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, i, SCALE, stream=streams[n % 2])
               for n, (q, i) in enumerate(zip(qs, ids))]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    q, i, out = qs[0].clone(), ids[0].clone(), torch.empty(B, 64, 512, device="cuda")
    graphs = []
    for _ in range(2):                                                    # two graphs of the same buffers
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, i, SCALE, out=out)
        graphs.append(gr)
    for n in range(4):
        q.copy_(qs[n])
        i.copy_(ids[n])
        out.fill_(math.nan)
        graphs[n % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[n])


def test_decode_workspace(dsa):
    """A workspace of exactly the size asked for, two calls at once with their own, and one too small."""
    g = gen(21)
    for B, K in ((1, 2048), (3, 900), (8, 1000), (300, 256)):
        N = 600
        cache, scale = make_cache(g, B * N)
        cache, scale = cache.view(B, N, 640), scale.view(B, N)
        kv_len = torch.full((B,), N, dtype=torch.int32, device="cuda")
        idx, q = choose(g, [N] * B, N, K), randn(g, B, 64, 576).bfloat16()
        need = dsa.attn_q8_workspace_size(B, K)
        assert (need == 0) == (B == 300)
        guard = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        out = dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, idx, SCALE, workspace=guard[:need] if need else None)
        assert bool((guard[need:] == 0xA5).all())
        assert torch.equal(out, dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, idx, SCALE))
        if need:
            with pytest.raises(dsa.DsaError) as e:
                dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, idx, SCALE, workspace=guard[:need - 16])
            assert e.value.code == 4


@pytest.mark.parametrize("more,K,page", [(1, 2048, 0), (8, 640, 16), (30, 1000, 0)])
def test_rows_behind_the_last_round(dsa, more, K, page):
    """A few queries more than a round of the SMs takes: those are cut and merged, the others run whole."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert dsa.attn_q8_workspace_size(sms + more, K) > 0 and dsa.attn_q8_workspace_size(sms, K) == 0
    test_prefill(dsa, sms + more, K + 77, K, page)
    test_decode(dsa, sms + more, K + 5, K, page)
    g = gen(23)
    cache, scale = make_cache(g, 64)
    q, idx = randn(g, sms + more, 64, 576).bfloat16(), torch.zeros(sms + more, K, dtype=torch.int32, device="cuda")
    small = torch.empty(dsa.attn_q8_workspace_size(sms + more, K) - 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(dsa.DsaError) as e:
        dsa.mla_sparse_attn_prefill_q8(q, cache, scale, idx, SCALE, workspace=small)
    assert e.value.code == 4


@pytest.mark.parametrize("B,N,K", [(153, 2053, 2048), (152, 1000, 900), (304, 1000, 512), (37, 1003, 700)])
def test_same_bits_every_time(dsa, B, N, K):
    """The order of every sum is fixed, so a call's bits are; 60 calls of uneven sequences in a row, whose tiles of
    several lengths meet the kernel's roles in every relative position, and the first of them right."""
    g = gen(B + N)
    lens = [N if b == 0 else (b * 7919) % (N + 1) for b in range(B)]
    cache, scale = make_cache(g, B * N, exponents=2)
    cache, scale = cache.view(B, N, 640), scale.view(B, N)
    idx, q = choose(g, lens, N, K), randn(g, B, 64, 576).bfloat16()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kv = values(cache, scale)
    ref = attention64(q, lambda s: torch.stack([kv[b][idx[b].clamp(min=0).long()] for b in range(B)[s]]), idx >= 0, SCALE)
    out, lse = dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, idx, SCALE, want_lse=True)
    close(out, lse, ref)
    for _ in range(60):
        o, l = dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, idx, SCALE, want_lse=True)
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert dsa.device_status() == 0


def test_threads_on_one_stream(dsa):
    """Decode calls of two threads on the same stream, which may enqueue their kernels in any order: the bits of
    calls made alone, and no workspace of one in the hands of the other."""
    g = gen(22)
    B, N, K = 4, 900, 700
    cache, scale = make_cache(g, B * N)
    cache, scale = cache.view(B, N, 640), scale.view(B, N)
    kv_len = torch.full((B,), N, dtype=torch.int32, device="cuda")
    qs = [randn(g, B, 64, 576).bfloat16() for _ in range(2)]
    ids = [choose(g, [N] * B, N, K) for _ in range(2)]
    want = [dsa.mla_sparse_attn_decode_q8(q, cache, scale, kv_len, i, SCALE) for q, i in zip(qs, ids)]
    torch.cuda.synchronize()
    got, held, start = [[], []], [None, None], threading.Barrier(2)

    def work(n):
        start.wait()
        for _ in range(100):
            got[n].append(dsa.mla_sparse_attn_decode_q8(qs[n], cache, scale, kv_len, ids[n], SCALE))
        held[n] = {w.data_ptr() for w in dsa._workspaces.by_stream.values()}
        start.wait()

    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert held[0] and held[1] and not held[0] & held[1]
    for n in range(2):
        assert len(got[n]) == 100 and all(torch.equal(o, want[n]) for o in got[n])


def test_wrapper_refusals(dsa):
    g = gen(18)
    cache, scale = make_cache(g, 32)
    q = randn(g, 2, 64, 576).bfloat16()
    idx = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    ok = dict(q=q, cache=cache, cache_scale=scale, idx=idx, scale=SCALE)
    dsa.mla_sparse_attn_prefill_q8(**ok)
    for bad in (dict(cache=cache[:, :576]), dict(cache_scale=scale[:31]), dict(cache=cache.int()), dict(idx=idx.long()),
                dict(q=q.float()), dict(q=q[:1]), dict(out_dtype=torch.float16), dict(cache_scale=scale.double()),
                dict(cache=cache.cpu()), dict(out=torch.empty(1, 64, 512, device="cuda")),
                dict(idx=idx.t()), dict(lse=torch.empty(2, 32, device="cuda"))):
        with pytest.raises(ValueError):
            dsa.mla_sparse_attn_prefill_q8(**{**ok, **bad})
    with pytest.raises(dsa.DsaError):
        dsa.mla_sparse_attn_prefill_q8(**{**ok, "scale": 0.0})
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        dsa.mla_cache_read_q8(cache, scale, slots.long())
    with pytest.raises(ValueError):
        dsa.mla_cache_read_q8(cache, scale, slots, out=torch.empty(2, 576, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(dsa.DsaError):
        dsa.mla_cache_read_q8(cache, scale, slots[:0])                    # nothing to do is refused, as elsewhere
    kv_a = randn(g, 3, 576).bfloat16()
    w, cs = torch.ones(512, device="cuda"), angles(4)
    for bad in (dict(kv_a=kv_a.float()), dict(kv_a=kv_a[:, :512]), dict(norm_w=w.bfloat16()), dict(pos=slots[:2]),
                dict(slots=slots.long()), dict(cos_sin=cs[:, :32]), dict(kv_a=kv_a.t().contiguous().t())):
        with pytest.raises(ValueError):
            dsa.mla_cache_write_q8(**{**dict(kv_a=kv_a, norm_w=w, eps=1e-6, cos_sin=cs, pos=slots, slots=slots, cache=cache,
                                             cache_scale=scale), **bad})


# ------------------------------------------------------------------------------------------------ together

def test_serving_steps_together(dsa):
    """Two sequences over a paged 8-bit cache: a prompt's rows written, a chunk attended to, then decode steps
    of one token each -- indexer inputs, cache write, scores, selection, attention -- against the same
    steps in float64 on what the caches hold."""
    g = gen(19)
    B, page, pages, N, K = 2, 16, 40, 260, 128
    lens = [230, 97]
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    table = perm[:2 * 17].view(2, 17).contiguous()
    cs = angles(N)
    w = torch.exp(0.3 * randn(g, 512))
    k_w, k_b = torch.exp(0.3 * randn(g, 128)), 0.1 * randn(g, 128)
    cache, scale = torch.zeros(pages * page, 640, dtype=torch.uint8, device="cuda"), torch.ones(pages * page, device="cuda")
    k_cache = torch.zeros(pages * page, 128, dtype=torch.bfloat16, device="cuda")

    def slots_of(b, pos):
        return table[b, (pos // page).long()] * page + pos % page

    def put(b, pos):
        R = pos.numel()
        qi = dsa.indexer_norm_rope(randn(g, R, 32, 128).bfloat16(), randn(g, R, 128).bfloat16(), k_w, k_b, 1e-6, cs, pos,
                                   slots_of(b, pos), k_cache)
        dsa.mla_cache_write_q8(randn(g, R, 576).bfloat16(), w, 1e-6, cs, pos, slots_of(b, pos), cache, scale)
        return qi

    def expected(b, n, q, idx):
        at = slots_of(b, torch.arange(n, device="cuda", dtype=torch.int32)).long()
        kv = values(cache[at], scale[at])
        return attention64(q, lambda s: kv[idx[s].clamp(min=0).long()], idx >= 0, SCALE)

    def selected(scores, idx, n):
        """idx holds a best selection of the n keys of `scores` (the library's float32 scores)."""
        got = idx[idx >= 0].long()
        assert got.numel() == min(n, K) and got.unique().numel() == got.numel()
        assert float(scores[got].min()) >= float(scores[:n].topk(min(n, K)).values.min())

    # a prompt chunk of each sequence
    for b in range(B):
        pos = torch.arange(lens[b], device="cuda", dtype=torch.int32)
        qi = put(b, pos)
        wi = randn(g, 1, lens[b], 32)
        p0, kl = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([lens[b]], dtype=torch.int32, device="cuda")
        S = dsa.indexer_scores_paged(qi[None], k_cache, wi, p0, kl, table[b:b + 1].contiguous(), page, N)
        idx = dsa.topk(S, p0, kl, N, K)[0]
        q = randn(g, lens[b], 64, 576).bfloat16()
        out, lse = dsa.mla_sparse_attn_prefill_q8_paged(q, cache, scale, table[b], page, idx, SCALE, lens[b], want_lse=True)
        close(out, lse, expected(b, lens[b], q, idx))
        for i in (0, K - 1, K, lens[b] - 1):
            if i < lens[b]:
                selected(S[0, i], idx[i], i + 1)
    # decode
    for step in range(3):
        pos = torch.tensor([n + step for n in lens], dtype=torch.int32, device="cuda")
        both = torch.stack([slots_of(b, pos[b:b + 1])[0] for b in range(B)]).int()
        qi = dsa.indexer_norm_rope(randn(g, B, 32, 128).bfloat16(), randn(g, B, 128).bfloat16(), k_w, k_b, 1e-6, cs, pos, both,
                                   k_cache)
        dsa.mla_cache_write_q8(randn(g, B, 576).bfloat16(), w, 1e-6, cs, pos, both, cache, scale)
        kl = pos + 1
        S = dsa.indexer_scores_paged(qi[:, None].contiguous(), k_cache, randn(g, B, 1, 32), pos, kl, table, page, N)
        idx = dsa.topk(S, pos, kl, N, K)[:, 0].contiguous()
        q = randn(g, B, 64, 576).bfloat16()
        out, lse = dsa.mla_sparse_attn_decode_q8_paged(q, cache, scale, kl, table, page, idx, SCALE, N, want_lse=True)
        back = dsa.mla_cache_read_q8_paged(cache, scale, kl, table, page, N)
        for b in range(B):
            n = int(kl[b])
            ref = expected(b, n, q[b:b + 1], idx[b:b + 1])
            close(out[b:b + 1], lse[b:b + 1], ref)
            at = slots_of(b, torch.arange(n, device="cuda", dtype=torch.int32)).long()
            assert torch.equal(back[b, :n].double(), values(cache[at], scale[at]))
            selected(S[b, 0], idx[b], n)
    assert dsa.device_status() == 0
