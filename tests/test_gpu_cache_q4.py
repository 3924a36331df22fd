"""The 4-bit latent cache (write, read back, attention over it) on the GPU, against plain float64 implementations
written here, and against the calls over the 8-bit cache of the same values, whose bits must be the same.

Tolerances, from the arithmetic:

* codes: the kernel's value of u, in pairs of floats rounded to odd, is within about 2^-44 (relative) of the exact one,
  the float64 reference here within 2^-49: only a value within 2^-40 of a border between two codes, two block scales
  or two row scales can fall on either side.  Values below float32's smallest step, 2^-149, may be zeros.
* rope: half a bf16 step, 2^-8 |value| (2^-134 where the step is 2^-133), and 2^-18 of the pair's length for the
  float32 arithmetic before it.
* reading back is exact for power-of-two scales; for any other the product is a float32 rounded to bf16: 2^-8 + 2^-24.
* attention, per element, as over the 8-bit cache: the probabilities enter the value product with eight significant
  bits, 2^-8 A with A = sum_t p_t |v_t|, the float32 logits and sums 2^-12 A more; weights are held to half of 2^-13
  where the head's largest is at least 2^4.5: 2^-18.5 a key, 2^-7.5 max|v| for 2048 of them.  A bf16 output adds
  2^-8 |ref|; lse 2^-12 absolute.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
SCALE = 1.0 / 16.0
MAG = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
STEPS = [(1 + m / 4) * 2.0 ** (a - 6) for a in range(12) for m in range(3)]


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


def angles(n):
    f = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def codes_of(rows):
    """Magnitude indices and signs [.., 512] of rows [.., 416], dim after dim."""
    index, neg = [], []
    for d in range(8):
        byte = rows[..., d // 2:256:4].int()
        index.append(byte >> (4 * (d % 2)) & 7)
        sign = rows[..., d % 4:256:4].int()
        neg.append(sign >> (7 if d < 4 else 3) & 1)
    return torch.stack(index, -1).flatten(-2), torch.stack(neg, -1).flatten(-2)


def parts(rows):
    """e4m3 * row scale's e4m3 values [.., 512] float64 and rope dims [.., 64] float64 of rows [.., 416]."""
    index, neg = codes_of(rows)
    table = torch.tensor(STEPS + [0.0] * 220, dtype=torch.float64, device="cuda")
    step = table[rows[..., 256:288].long()].repeat_interleave(16, -1)
    mag = torch.tensor(MAG, dtype=torch.float64, device="cuda")[index.long()]
    return torch.where(neg > 0, -mag, mag) * step, rows[..., 288:].contiguous().view(torch.bfloat16).double()


def values(rows, scale):
    lat, rope = parts(rows)
    return torch.cat([lat * scale[..., None].double(), rope], -1)


def as_q8(rows):
    """The same rows in the 8-bit format."""
    lat, _ = parts(rows)
    codes = lat.float().to(F8)
    assert torch.equal(codes.double(), lat)                              # every product of a code and a block is e4m3
    return torch.cat([codes.view(torch.uint8), rows[..., 288:]], -1)


def make_cache(g, rows, exponents=0, junk=False):
    """Random codes; block bytes near the top of the range or (junk) of every value; scales 2^k, k spread over +-exponents."""
    cache = torch.randint(0, 256, (rows, 416), generator=g, device="cuda").byte()
    if not junk:
        cache[:, 256:288] = torch.randint(24, 33, (rows, 32), generator=g, device="cuda").byte()
    cache[:, 288:] = randn(g, rows, 64).bfloat16().view(torch.uint8)
    k = torch.randint(-exponents, exponents + 1, (rows,), generator=g, device="cuda") if exponents else torch.zeros(rows, device="cuda")
    return cache, torch.exp2(k.float() - 5.0)


def paged(g, cache, scale, lens, page, extra=3):
    """Dense [B, N] rows laid out over a shuffled pool; NaN rows and scales everywhere no sequence has a key."""
    B, N = scale.shape
    used = [-(-n // page) for n in lens]
    pages = sum(used) + extra
    perm = torch.randperm(pages, generator=g, device="cuda")
    pool = torch.full((pages * page, 416), 0x7F, dtype=torch.uint8, device="cuda")
    pool[:, 288:] = 0xFF
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

def check_written(kv_a, w, eps, cs, interleave, rows, scale):
    """The rows' contents against the formula in float64: every code, block byte and scale, but next to a border."""
    x = kv_a.double()
    c = x[:, :512]
    u = torch.nan_to_num(c / torch.sqrt((c * c).mean(1, keepdim=True) + eps), nan=0.0) * w.double()
    top = u.abs().view(-1, 32, 16).amax(2)
    tiny = 2.0 ** -40
    # block scale: the smallest of (1, 1.25, 1.5) 2^j at or above top / 6
    e = torch.floor(torch.log2((top / 6).clamp(min=1e-300)))
    f = (top / 6).clamp(min=1e-300) / torch.exp2(e)
    m = torch.where(f <= 1, 0, torch.where(f <= 1.25, 1, torch.where(f <= 1.5, 2, 3)))
    j, m = torch.where(m == 3, e + 1, e), torch.where(m == 3, 0, m)
    near = torch.stack([(f / t - 1).abs() for t in (1.0, 1.25, 1.5, 2.0)]).amin(0) <= tiny
    j = torch.where(top == 0, torch.full_like(j, -4000.0), j)
    k = (j.amax(1) - 5).clamp(-64, 64)
    row_near = (near & (j >= j.amax(1, keepdim=True) - 1)).any(1)
    assert bool(((scale.double() == torch.exp2(k)) | row_near).all())
    k = torch.log2(scale.double())                                        # its own row scale from here on
    a = j - k[:, None] + 6
    want = torch.where(a < 0, 0, torch.where(a > 11, 35, 3 * a + m))
    got = rows[:, 256:288].double()
    assert bool(((got == want) | near).all()) and bool((got < 36).all())
    step = torch.tensor(STEPS, dtype=torch.float64, device="cuda")[rows[:, 256:288].long()] * torch.exp2(k)[:, None]
    v = u.abs() / step.repeat_interleave(16, 1)
    index, neg = codes_of(rows)
    mag = torch.tensor(MAG, dtype=torch.float64, device="cuda")
    dist = (v.clamp(max=6.0)[..., None] - mag).abs()
    least = dist.amin(-1, keepdim=True)
    tie = dist <= least + tiny * v.clamp(max=6.0)[..., None]              # the magnitudes that may be meant
    assert bool(tie.gather(-1, index.long()[..., None]).all())
    even = (dist == least) & (torch.arange(8, device="cuda") % 2 == 0)
    exact_tie = ((dist == least).sum(-1) == 2) & (v == (v * 4).round() / 4)
    assert bool((~exact_tie | even.gather(-1, index.long()[..., None])[..., 0]).all())
    # u is held as a float32, whose smallest step is 2^-149: what is below may be a zero, which has no sign
    assert bool(((neg == 1) == (u < 0))[u.abs() >= 2.0 ** -149].all())
    cc, ss = cs[:, :32].double(), cs[:, 32:].double()
    r = x[:, 512:]
    p, q = (r[:, 0::2], r[:, 1::2]) if interleave else (r[:, :32], r[:, 32:])
    z, n = (p * cc - q * ss, q * cc + p * ss), torch.hypot(p, q)
    if interleave:
        z, n = torch.stack(z, -1).flatten(1), torch.stack([n, n], -1).flatten(1)
    else:
        z, n = torch.cat(z, 1), torch.cat([n, n], 1)
    rope = rows[:, 288:].contiguous().view(torch.bfloat16).double()
    assert bool(((rope - z).abs() <= 2.0 ** -8 * z.abs() + 2.0 ** -18 * n + 2.0 ** -134).all())


@pytest.mark.parametrize("R,ld,interleave", [(1, 576, True), (3, 584, False), (8, 2048, True), (33, 576, False),
                                             (1000, 640, True), (4100, 576, True)])
def test_write(dsa, R, ld, interleave):
    g = gen(R)
    rows, eps = 2 * R + 5, 2.0 ** -20
    kv_a = (randn(g, R, ld) * torch.exp(2 * randn(g, R, 1))).bfloat16()[:, :576]
    w = torch.exp(randn(g, 512))
    w[::7] *= 2.0 ** -9                                                   # blocks far below the row's largest
    cs = angles(5000)
    pos = torch.randint(0, 5000, (R,), generator=g, device="cuda").int()
    slots = torch.randperm(rows, generator=g, device="cuda")[:R].int()
    if R > 4:
        slots[R // 2] = -1
        slots[R - 1] = -1000
        pos[R - 1] = -5                                                   # a padding token's position is not looked at
        kv_a[R // 3] = 0.0
        kv_a[0, 16:48] = 0.0                                              # blocks of zeros
    cache = torch.randint(0, 256, (rows, 416), generator=g, device="cuda").byte()
    scale = torch.rand(rows, generator=g, device="cuda")
    before, sbefore = cache.clone(), scale.clone()
    dsa.mla_cache_write_q4(kv_a, w, eps, cs, pos, slots, cache, scale, interleave=interleave)
    assert dsa.device_status() == 0
    kept = slots >= 0
    to = slots[kept].long()
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[to] = False
    assert torch.equal(cache[rest], before[rest]) and torch.equal(scale[rest], sbefore[rest])
    check_written(kv_a[kept], w, eps, cs[pos[kept].long()], interleave, cache[to], scale[to])


def test_write_ties_and_borders(dsa):
    """Rows whose norm is a power of two, so that values lie on the borders themselves: 1.125, 1.5 and 1.875 times a
    power of two are the largest values of their block scales, halves between two magnitudes go to the even one."""
    grid = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 5.5])
    rows = []
    for f in (1.0, 1.25, 1.5):
        block = grid * f
        rows.append(torch.cat([block * (-1) ** b * 2.0 ** -(b % 14) for b in range(32)]))
    kv = torch.zeros(3, 576)
    kv[:, :512] = torch.stack(rows)
    kv = kv.bfloat16().cuda()
    assert torch.equal(kv[:, :512].double().cpu(), torch.stack(rows).double())
    # a weight of sqrt(mean square) would not be exact: with a weight of one and eps that completes the mean square to
    # 2^20 the quotient is the row times 2^-10, if the sum is exact in float32
    ms = (kv[:, :512].double() ** 2).mean(1)
    cs, w = angles(1), torch.ones(512, device="cuda")
    for r in range(3):
        eps = 2.0 ** 20 - float(ms[r])
        if float(torch.tensor(eps)) != eps:
            eps = float(torch.tensor(eps))
        cache, scale = torch.zeros(1, 416, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
        dsa.mla_cache_write_q4(kv[r:r + 1], w, eps, cs, i32(0), i32(0), cache, scale)
        check_written(kv[r:r + 1], w, float(torch.tensor(eps)), cs, True, cache, scale)


def test_write_extremes(dsa):
    """Tiny, huge and zero rows; weights that reach the scale's clamps and saturate past them."""
    g = gen(5)
    amp = torch.tensor([0.0, 1e-38, 1e-20, 1.0, 1e15, 0.0], device="cuda")
    kv_a = (randn(g, 6, 576) * amp[:, None]).bfloat16()
    kv_a[5, 7] = 2.0 ** -60
    cs = angles(4)
    pos = i32(0, 1, 2, 3, 0, 1)
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    for w in (1.0, 2.0 ** -60, 2.0 ** 60, 2.0 ** 80):
        wt = torch.full((512,), w, device="cuda")
        cache, scale = torch.zeros(6, 416, dtype=torch.uint8, device="cuda"), torch.zeros(6, device="cuda")
        eps = 2.0 ** -20
        dsa.mla_cache_write_q4(kv_a, wt, eps, cs, pos, slots, cache, scale)
        check_written(kv_a, wt, eps, cs[pos.long()], True, cache, scale)
        assert float(scale[0]) == 2.0 ** -64 and bool((cache[0, :288] == 0).all())    # zeros


def test_write_records_what_is_out_of_range(dsa):
    g = gen(6)
    kv_a = randn(g, 4, 576).bfloat16()
    cs, w = angles(10), torch.ones(512, device="cuda")
    for pos, slots in (((1, 10, 2, 3), (0, 1, 2, 3)), ((1, -1, 2, 3), (0, 1, 2, 3)), ((1, 1, 2, 3), (0, 9, 2, 3))):
        cache = torch.full((9, 416), 17, dtype=torch.uint8, device="cuda")
        scale = torch.full((9,), 3.0, device="cuda")
        dsa.mla_cache_write_q4(kv_a, w, 2.0 ** -20, cs, i32(*pos), i32(*slots), cache, scale)
        assert dsa.device_status() == 7
        assert bool((cache[[1, 4, 8]] == 17).all()) and bool((scale[[1, 4, 8]] == 3.0).all())
        to = torch.tensor([0, 2, 3], device="cuda")
        check_written(kv_a[to], w, 2.0 ** -20, cs[i32(*pos)[to].long()], True, cache[to], scale[to])


# ------------------------------------------------------------------------------------------------ read back

@pytest.mark.parametrize("R", [1, 2, 9, 500, 10007])
def test_read_by_slot(dsa, R):
    g = gen(R)
    rows = R + 50
    cache, scale = make_cache(g, rows, exponents=20, junk=True)           # every byte of a block stands for something
    slots = torch.randint(-2, rows, (R,), generator=g, device="cuda").int()
    out = dsa.mla_cache_read_q4(cache, scale, slots)
    want = values(cache, scale)[slots.clamp(min=0).long()]
    want[slots < 0] = 0.0
    assert torch.equal(out.double(), want) and dsa.device_status() == 0
    odd = scale * 1.37
    out = dsa.mla_cache_read_q4(cache, odd, slots)
    want = values(cache, odd)[slots.clamp(min=0).long()]
    want[slots < 0] = 0.0
    assert bool(((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -24) * want.abs()).all())
    slots[0] = rows
    out = dsa.mla_cache_read_q4(cache, scale, slots)
    assert dsa.device_status() == 7 and bool((out[0] == 0).all())


@pytest.mark.parametrize("lens,N,page", [([1], 1, 16), ([0, 5, 64, 63], 64, 64), ([300, 0, 17, 299, 1], 300, 16),
                                         ([1000, 1023], 1024, 256)])
def test_read_paged(dsa, lens, N, page):
    g = gen(N)
    B = len(lens)
    cache, scale = make_cache(g, B * N, exponents=8)
    cache, scale = cache.view(B, N, 416), scale.view(B, N)
    pool, pscale, table, pages = paged(g, cache, scale, lens, page)
    kv_len = i32(*lens)
    out = torch.full((B, N, 576), -3.0, dtype=torch.bfloat16, device="cuda")
    dsa.mla_cache_read_q4_paged(pool, pscale, kv_len, table, page, N, out=out)
    assert dsa.device_status() == 0
    want = values(cache, scale)
    for b, n in enumerate(lens):
        assert torch.equal(out[b, :n].double(), want[b, :n])
        assert bool((out[b, n:] == -3.0).all())
    b = max(range(B), key=lambda i: lens[i])
    table[b, 0] = pages                                                   # a page outside the pool: zeros, recorded
    out = dsa.mla_cache_read_q4_paged(pool, pscale, kv_len, table, page, N)
    n = min(page, lens[b])
    assert dsa.device_status() == 7 and bool((out[b, :n] == 0).all())
    assert torch.equal(out[b, n:lens[b]].double(), want[b, n:lens[b]])


# ------------------------------------------------------------------------------------------------ attention

def attention64(q, rows, have, scale):
    """(out, lse, A, vmax) in float64: q [R, 64, 576], rows(slice) [r, K, 576], have [R, K]."""
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


def close(got, lse, ref):
    out, l64, A, vm = ref
    err = (got.double() - out).abs()
    bound = (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -7.5 * vm
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * out.abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())
    dead = torch.isneginf(l64)
    assert torch.equal(torch.isneginf(lse), dead)
    assert bool(((lse.double() - l64).abs()[~dead] <= 2.0 ** -12).all())


def choose(g, counts, N, top_k):
    """Ascending random selections of min(top_k, count) keys, -1 padded."""
    c = torch.tensor(counts, device="cuda")
    r = torch.rand(len(counts), N, generator=g, device="cuda")
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
    cache, scale = cache.view(B, N, 416), scale.view(B, N)
    idx = choose(g, lens, N, top_k)
    q = randn(g, B, 64, 576).bfloat16()
    kv_len = i32(*lens)
    kv = values(cache, scale)
    ref = attention64(q, lambda s: torch.stack([kv[b][idx[b].clamp(min=0).long()] for b in range(B)[s]]), idx >= 0, SCALE)
    if page:
        pool, pscale, table, _ = paged(g, cache, scale, lens, page)
        call = lambda **k: dsa.mla_sparse_attn_decode_q4_paged(q, pool, pscale, kv_len, table, page, idx, SCALE, N,   # noqa: E731
                                                               want_lse=True, **k)
        twin = dsa.mla_sparse_attn_decode_q8_paged(q, as_q8(pool), pscale, kv_len, table, page, idx, SCALE, N, want_lse=True)
    else:
        call = lambda **k: dsa.mla_sparse_attn_decode_q4(q, cache, scale, kv_len, idx, SCALE, want_lse=True, **k)     # noqa: E731
        twin = dsa.mla_sparse_attn_decode_q8(q, as_q8(cache), scale, kv_len, idx, SCALE, want_lse=True)
    out, lse = call()
    assert dsa.device_status() == 0
    close(out, lse, ref)
    assert torch.equal(out, twin[0]) and torch.equal(lse, twin[1])
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
        out, lse = dsa.mla_sparse_attn_prefill_q4_paged(q, pool, pscale, table[0], page, idx, SCALE, N, want_lse=True)
    else:
        out, lse = dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE, want_lse=True)
    twin = dsa.mla_sparse_attn_prefill_q8(q, as_q8(cache), scale, idx, SCALE, want_lse=True)
    assert dsa.device_status() == 0
    close(out, lse, ref)
    assert torch.equal(out, twin[0]) and torch.equal(lse, twin[1])
    if not page:                                                          # the bf16 calls over the rows read back
        back = dsa.mla_cache_read_q4(cache, scale, torch.arange(N, dtype=torch.int32, device="cuda"))
        other = dsa.mla_sparse_attn_prefill(q, back, idx, SCALE)
        err = (out - other).abs().double()
        assert float(err.sum()) <= 4e-3 * float(ref[0].abs().sum())


@pytest.mark.parametrize("K", [1, 127, 129, 1000, 2048])
def test_attention_over_any_bytes(dsa, K):
    """Block bytes of every value (36 and above: zeros), scales 2^-20 to 2^20 apart, rows of zeros of both kinds."""
    g = gen(K)
    N = 2048
    cache, scale = make_cache(g, N, exponents=20, junk=True)
    cache[::5, :256] &= 0x88                                              # zeros of either sign
    cache[1::5, 256:288] |= 0x80                                          # blocks of zeros
    scale[::10] = 1.0
    q = randn(g, 4, 64, 576).bfloat16()
    idx = torch.stack([torch.randperm(N, generator=g, device="cuda")[:K] for _ in range(4)]).int()
    out, lse = dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, 2.0 ** -24, want_lse=True)
    eight = as_q8(cache)
    twin = dsa.mla_sparse_attn_prefill_q8(q, eight, scale, idx, 2.0 ** -24, want_lse=True)
    # the 8-bit call finds every row of zeros, this one those of zero codes: take the others' scale where it is looked at
    assert dsa.device_status() == 0
    blockzero = (parts(cache)[0] == 0).all(1) & (codes_of(cache)[0] != 0).any(1) & (scale >= 1)
    same = ~blockzero[idx.long()].any(1)
    assert torch.equal(out[same], twin[0][same]) and torch.equal(lse[same], twin[1][same])
    # Scales this far apart: what the value product takes is p c, off by 2^-8 of itself or, where it is small, by half of
    # 2^-13 where the head's largest p c is at least 2^4.5: 2^-18.5 of that.  A key adds that times its code |v| / c.
    # (A row whose codes are zeros counts with 2^-64 where its scale is 1 or more.)
    kv, c = values(cache, scale)[idx.long()], scale[idx.long()].double()
    found = (codes_of(cache)[0] == 0).all(1)[idx.long()] & (c >= 1)
    x = torch.einsum("rhd,rkd->rhk", q.double(), kv) * 2.0 ** -24
    p = torch.softmax(x, -1)
    v = kv[..., :512]
    most = (p * torch.where(found, 2.0 ** -64, c)[:, None]).amax(-1, keepdim=True)
    bound = (2.0 ** -8 + 2.0 ** -12) * (p @ v.abs()) + 2.0 ** -18.5 * most * (v.abs() / c[..., None]).sum(1)[:, None]
    assert bool(((out.double() - p @ v).abs() <= bound).all())
    assert bool(((lse.double() - torch.logsumexp(x, -1)).abs() <= 2.0 ** -12).all())


def test_attention_reads_only_selected_rows(dsa):
    """Rows, scales and pages that no key names may hold anything: NaN rope dims and scales."""
    g = gen(11)
    N, K = 600, 257
    cache, scale = make_cache(g, N)
    q = randn(g, 3, 64, 576).bfloat16()
    idx = choose(g, [N, 300, 40], N, K)
    want = dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE, want_lse=True)
    used = torch.zeros(N, dtype=torch.bool, device="cuda")
    used[idx[idx >= 0].long()] = True
    bad, bscale = cache.clone(), scale.clone()
    bad[~used] = 0xFF
    bscale[~used] = math.nan
    got = dsa.mla_sparse_attn_prefill_q4(q, bad, bscale, idx, SCALE, want_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_records_keys_outside_the_cache(dsa):
    g = gen(12)
    B, N, K, page = 3, 100, 40, 16
    cache, scale = make_cache(g, B * N)
    cache, scale = cache.view(B, N, 416), scale.view(B, N)
    lens = [100, 50, 10]
    idx = choose(g, lens, N, K)
    q = randn(g, B, 64, 576).bfloat16()
    want = dsa.mla_sparse_attn_decode_q4(q, cache, scale, i32(*lens), idx, SCALE)
    more = torch.cat([idx, torch.full((B, 1), 2 ** 31 - 1, dtype=torch.int32, device="cuda"), i32(100, 50, 10)[:, None]], 1)
    got = dsa.mla_sparse_attn_decode_q4(q, cache, scale, i32(*lens), more.contiguous(), SCALE)
    assert dsa.device_status() == 7 and torch.equal(got, want)
    pool, pscale, table, pages = paged(g, cache, scale, lens, page)
    table[0, 2] = pages + 5
    dsa.mla_sparse_attn_decode_q4_paged(q, pool, pscale, i32(*lens), table, page, idx, SCALE, N)
    assert dsa.device_status() == 7


@pytest.mark.parametrize("L,expanded", [(4, False), (150, True)])
def test_prefill_records_pages_outside_the_pool(dsa, L, expanded):
    """Also where the cache is expanded first: a selected key on a page outside the pool is a row of zeros and recorded,
    a page that no query selects may be anything."""
    g = gen(16)
    N, K, page = 1000, 900, 16
    assert (dsa.attn_q4_workspace_size(L, K, N) > dsa.attn_q8_workspace_size(L, K)) == expanded
    cache, scale = make_cache(g, N)
    pool, pscale, table, pages = paged(g, cache[None], scale[None], [N], page)
    q = randn(g, L, 64, 576).bfloat16()
    idx = choose(g, [N - 32] * L, N - 32, K)
    want = dsa.mla_sparse_attn_prefill_q4_paged(q, pool, pscale, table[0], page, idx, SCALE, N, want_lse=True)
    table[0, -1], table[0, -2] = -1, pages                                # keys that nothing selects
    got = dsa.mla_sparse_attn_prefill_q4_paged(q, pool, pscale, table[0], page, idx, SCALE, N, want_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and dsa.device_status() == 0
    table[0, 3] = pages
    got = dsa.mla_sparse_attn_prefill_q4_paged(q, pool, pscale, table[0], page, idx, SCALE, N, want_lse=True)
    assert dsa.device_status() == 7
    gone = cache.clone()
    gone[3 * page:4 * page] = 0
    twin = dsa.mla_sparse_attn_prefill_q4(q, gone, scale, idx, SCALE, want_lse=True)
    close(got[0], got[1], attention64(q, lambda s: values(gone, scale)[idx[s].clamp(min=0).long()], idx >= 0, SCALE))
    close(twin[0], twin[1], attention64(q, lambda s: values(gone, scale)[idx[s].clamp(min=0).long()], idx >= 0, SCALE))


def test_prefill_workspace(dsa):
    """The size the library names is enough and needed; a given workspace gives the same bits."""
    g = gen(17)
    L, N, K = 160, 700, 640
    cache, scale = make_cache(g, N, exponents=1)
    q, idx = randn(g, L, 64, 576).bfloat16(), choose(g, [N] * L, N, K)
    want = dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE)
    need = dsa.attn_q4_workspace_size(L, K, N)
    assert need > dsa.attn_q8_workspace_size(L, K)
    ws = torch.full((need + 256,), 0xEE, dtype=torch.uint8, device="cuda")
    got = dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE, workspace=ws[:need])
    assert torch.equal(got, want) and bool((ws[need:] == 0xEE).all()) and dsa.device_status() == 0
    for bad in (ws[:need - 1], ws[16:]):
        with pytest.raises(dsa.DsaError):
            dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE, workspace=bad)


def test_offsets_past_32_bits(dsa):
    """Rows past the 2^32nd byte of the cache."""
    g = gen(13)
    N = (1 << 32) // 416 + 5000
    cache = torch.zeros(N, 416, dtype=torch.uint8, device="cuda")
    scale = torch.ones(N, device="cuda")
    some = torch.cat([torch.arange(300, device="cuda"), torch.arange(N - 600, N, device="cuda")])
    c, s = make_cache(g, len(some), exponents=1)
    cache[some], scale[some] = c, s
    idx = some.int()[None].contiguous()
    q = randn(g, 1, 64, 576).bfloat16()
    out, lse = dsa.mla_sparse_attn_prefill_q4(q, cache, scale, idx, SCALE, want_lse=True)
    near = torch.arange(len(some), dtype=torch.int32, device="cuda")[None].contiguous()
    want = dsa.mla_sparse_attn_prefill_q4(q, c, s, near, SCALE, want_lse=True)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(dsa.mla_cache_read_q4(cache, scale, idx[0]), dsa.mla_cache_read_q4(c, s, near[0]))
    kv_a = randn(g, 2, 576).bfloat16()
    one = torch.zeros(2, 416, dtype=torch.uint8, device="cuda"), torch.zeros(2, device="cuda")
    args = kv_a, torch.ones(512, device="cuda"), 1e-6, angles(2), i32(0, 1)
    dsa.mla_cache_write_q4(*args, i32(0, 1), *one)
    dsa.mla_cache_write_q4(*args, i32(N - 1, 5), cache, scale)
    assert torch.equal(cache[[N - 1, 5]], one[0]) and torch.equal(scale[[N - 1, 5]], one[1]) and dsa.device_status() == 0


def test_streams_and_graphs(dsa):
    """A given stream; two graphs of the same call, replayed in turn, whose workspaces differ."""
    g = gen(14)
    N, K = 3000, 2048
    cache, scale = make_cache(g, 2 * N)
    cache, scale = cache.view(2, N, 416), scale.view(2, N)
    q = [randn(g, 2, 64, 576).bfloat16() for _ in range(2)]
    idx, kv_len = choose(g, [N, 700], N, K), i32(N, 700)
    want = [dsa.mla_sparse_attn_decode_q4(x, cache, scale, kv_len, idx, SCALE) for x in q]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.mla_sparse_attn_decode_q4(q[0], cache, scale, kv_len, idx, SCALE, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    graphs = []
    for x in q:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = dsa.mla_sparse_attn_decode_q4(x, cache, scale, kv_len, idx, SCALE)
        graphs.append((graph, y))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for (_, y), w in zip(graphs, want))


@pytest.mark.parametrize("B,N,K", [(153, 2053, 2048), (152, 1000, 900), (304, 1000, 512), (37, 1003, 700)])
def test_same_bits_every_time(dsa, B, N, K):
    g = gen(B)
    cache, scale = make_cache(g, B * N, exponents=1)
    cache, scale = cache.view(B, N, 416), scale.view(B, N)
    lens = [N if b % 3 == 0 else (b * 7919) % (N + 1) for b in range(B)]
    idx, kv_len = choose(g, lens, N, K), i32(*lens)
    q = randn(g, B, 64, 576).bfloat16()
    want = dsa.mla_sparse_attn_decode_q8(q, as_q8(cache), scale, kv_len, idx, SCALE, want_lse=True)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    for _ in range(60):
        dsa.mla_sparse_attn_decode_q4(q, cache, scale, kv_len, idx, SCALE, out=out, lse=lse)
        differ += (out != want[0]).sum() + (lse != want[1]).sum()
    assert int(differ) == 0 and dsa.device_status() == 0


def test_serving_steps_together(dsa):
    """A prompt written, attended, then tokens decoded one by one over pages: each against float64 over the cache's own
    values."""
    g = gen(15)
    N0, steps, page, K = 200, 4, 64, 128
    N = N0 + steps
    kv_a, w, cs = randn(g, N, 576).bfloat16(), torch.exp(0.3 * randn(g, 512)), angles(N)
    table = torch.randperm(8, generator=g, device="cuda")[:4].int()[None].contiguous()
    j = torch.arange(N, device="cuda")
    slots = (table[0, j // page].long() * page + j % page).int()
    pool, scale = torch.full((8 * page, 416), 0xFF, dtype=torch.uint8, device="cuda"), torch.full((8 * page,), math.nan, device="cuda")
    dsa.mla_cache_write_q4(kv_a[:N0], w, 1e-6, cs, j[:N0].int(), slots[:N0].contiguous(), pool, scale)
    q = randn(g, N, 64, 576).bfloat16()
    idx = choose(g, list(range(1, N0 + 1)), N, K)
    out, lse = dsa.mla_sparse_attn_prefill_q4_paged(q[:N0].contiguous(), pool, scale, table[0], page, idx, SCALE, N0, want_lse=True)
    rows = lambda: values(pool[slots.long()], scale[slots.long()])        # noqa: E731
    kv = rows()
    close(out, lse, attention64(q[:N0], lambda s: kv[idx[s].clamp(min=0).long()], idx >= 0, SCALE))
    for t in range(N0, N):
        dsa.mla_cache_write_q4(kv_a[t:t + 1], w, 1e-6, cs, i32(t), slots[t:t + 1].contiguous(), pool, scale)
        one = choose(g, [t + 1], N, K)
        out, lse = dsa.mla_sparse_attn_decode_q4_paged(q[t:t + 1], pool, scale, i32(t + 1), table, page, one, SCALE, N,
                                                       want_lse=True)
        kv = rows()
        close(out, lse, attention64(q[t:t + 1], lambda s: kv[one[s].clamp(min=0).long()], one >= 0, SCALE))
    # against the tokens before they were rounded to four bits: a code is off by at most a sixth of its block's largest
    x = kv_a[:, :512].double()
    u = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6) * w.double()
    top = u.abs().view(N, 32, 16).amax(2).repeat_interleave(16, 1)
    assert bool(((kv[:, :512] - u).abs() <= top / 4).all())
    assert dsa.device_status() == 0


def test_wrapper_refusals(dsa):
    q = torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda")
    cache, scale = torch.zeros(2, 8, 416, dtype=torch.uint8, device="cuda"), torch.ones(2, 8, device="cuda")
    idx, kv_len = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), i32(8, 8)
    dsa.mla_sparse_attn_decode_q4(q, cache, scale, kv_len, idx, SCALE)
    for bad in (dict(cache=torch.zeros(2, 8, 640, dtype=torch.uint8, device="cuda")), dict(cache=cache[:, :4]),
                dict(cache_scale=scale.double()), dict(cache_scale=scale[:1]), dict(idx=idx.long()), dict(q=q.float()),
                dict(kv_len=kv_len[:1]), dict(cache=cache.cpu()), dict(q=q[:, :32])):
        with pytest.raises(ValueError):
            dsa.mla_sparse_attn_decode_q4(**{**dict(q=q, cache=cache, cache_scale=scale, kv_len=kv_len, idx=idx, scale=SCALE), **bad})
    with pytest.raises(ValueError):
        dsa.mla_cache_read_q4(torch.zeros(4, 640, dtype=torch.uint8, device="cuda"), torch.ones(4, device="cuda"), i32(0))
    with pytest.raises(ValueError):
        dsa.mla_sparse_attn_prefill_q8(q, cache.view(16, 416), scale.view(16), idx, SCALE)
