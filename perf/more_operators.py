"""Operators that let the latent cache hold longer contexts, as cases to be measured.

Four operators, each in its plain form (elementary torch operations) and as the call a user makes:

* ``store``: new tokens into the 4-bit latent cache (RMS norm of the 512 latent dims, rotation of the 64 rope dims,
  quantisation, scatter), and their rows back as bf16;
* ``decode`` / ``prefill``: sparse absorbed-MLA attention over the 4-bit cache, dense or paged;
* ``weights``: the attention weight that each key of a cache (bf16, 8-bit or 4-bit rows) received, summed over
  heads and queries;
* ``evict``: the keys of each sequence that stay, by that weight, and the moves that close the gaps in its caches.

A row of the 4-bit cache is 416 bytes: 32 blocks of 16 latent dims in 8 bytes each, a byte a block for its scale, 64
rope dims in bf16; beside it a float32 scale a row.  Of a group of eight dims, byte i holds the magnitudes of dims 2i
(bits 0-2) and 2i + 1 (bits 4-6) as indices into MAG, and the signs of dims 4 + i (bit 3) and i (bit 7).  Block byte
3 a + m stands for (1 + m / 4) 2^(a - 6), 36 and above for zero.

``run`` takes the plain form unless ``own`` is set; ``exact`` gives the results in 64 bits.
"""
import math

import torch

own = False

HEADS, QK, LATENT, ROPE = 64, 576, 512, 64                 # attention heads and widths
IDX_DIM = 128                                              # width of an indexer key
BLOCK, ROW4, ROW8 = 16, 416, 640                           # dims of a block; bytes of a 4-bit and of an 8-bit row
MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALE = 1.0 / 16.0                                         # 1 / sqrt(192 + 64)
EPS = 1e-6
TOP = 2048


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one user, one new token over a 4k context: pure latency
        {"name": "decode_b1", "op": "decode", "B": 1, "N": 4096, "top_k": 2048, "page": 0, "ragged": False},
        # an odd batch of short contexts over small pages, fewer keys than a full selection, one slot of the batch unused
        {"name": "decode_b37_short", "op": "decode", "B": 37, "N": 1003, "top_k": 700, "page": 16, "ragged": True},
        # a full serving batch of uneven contexts over pages
        {"name": "decode_b256_paged", "op": "decode", "B": 256, "N": 8192, "top_k": 2048, "page": 64, "ragged": True},
        # a prefill chunk's tail, sizes that fit no tile
        {"name": "prefill_333_paged", "op": "prefill", "L": 333, "N": 5001, "top_k": 2048, "page": 16},
        # the benchmark's prefill chunk: 4096 queries at 16k keys
        {"name": "prefill_16k", "op": "prefill", "L": 4096, "N": 16384, "top_k": 2048, "page": 0},
        # a decode step's new tokens into the cache and back: latency
        {"name": "store_8", "op": "store", "R": 8, "rows": 8 * 4096, "ld": 1024, "interleave": True},
        # a prefill chunk's rows into the cache and back
        {"name": "store_4096", "op": "store", "R": 4096, "rows": 6144, "ld": 576, "interleave": True},
        # the weights of a small batch's decode step over bf16 rows: latency
        {"name": "weights_b8", "op": "weights", "format": "bf16", "B": 8, "N": 4096, "top_k": 2048, "page": 0, "ragged": False},
        # the weights of a serving batch's decode step over a paged 4-bit cache
        {"name": "weights_b128_paged", "op": "weights", "format": "q4", "B": 128, "N": 8192, "top_k": 2048, "page": 64,
         "ragged": True},
        # the weights of the benchmark's prefill chunk
        {"name": "weights_prefill_16k", "op": "weights", "format": "bf16", "L": 4096, "N": 16384, "top_k": 2048, "page": 0},
        # a small batch at 4k keys each, halved
        {"name": "evict_b8", "op": "evict", "B": 8, "N": 4096, "keep": 2048, "recent": 256, "sink": 4, "page": 0, "ragged": False},
        # a serving batch of uneven contexts over pages, cut to 8k keys
        {"name": "evict_b64_paged", "op": "evict", "B": 64, "N": 16384, "keep": 8192, "recent": 512, "sink": 4, "page": 64,
         "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "store", "weights", "weights", "evict"])
    page = rng.choice([0, 16, 64, 256])
    if op == "decode":
        return {"op": op, "B": _log(rng, 1, 255), "N": _log(rng, 1, 8192), "top_k": _log(rng, 1, TOP), "page": page,
                "ragged": rng.random() < 0.5}
    if op == "prefill":
        n = _log(rng, 64, 16384)
        return {"op": op, "L": min(n, _log(rng, 1, 4095)), "N": n, "top_k": _log(rng, 1, TOP), "page": page}
    if op == "store":
        r = _log(rng, 1, 8192)
        return {"op": op, "R": r, "rows": r + rng.randint(0, 4096), "ld": rng.choice([576, 584, 1024]),
                "interleave": rng.random() < 0.5}
    if op == "weights":
        c = {"op": op, "format": rng.choice(["bf16", "q8", "q4"]), "N": _log(rng, 1, 8192), "top_k": _log(rng, 1, TOP),
             "page": page}
        if rng.random() < 0.5:
            return dict(c, B=_log(rng, 1, 255), ragged=rng.random() < 0.5)
        return dict(c, L=min(c["N"], _log(rng, 1, 4095)))
    n = _log(rng, 16, 16384)
    keep = rng.randint(1, n - 1)
    recent = rng.randint(0, keep)
    return {"op": op, "B": _log(rng, 1, 63), "N": n, "keep": keep, "recent": recent, "sink": min(rng.randint(0, 8), keep - recent),
            "page": page, "ragged": rng.random() < 0.5}


def _row_bytes(fmt):
    """Bytes of a key's row, its scale among them."""
    return {"bf16": 2 * QK, "q8": ROW8 + 4, "q4": ROW4 + 4}[fmt]


def work(case):
    op = case["op"]
    if op in ("decode", "prefill", "weights"):
        if "B" in case:
            queries = case["B"]
            lens = _lens(case)
            slots = sum(min(n, case["top_k"]) for n in lens)
            keys = slots                                     # each sequence reads its own rows
        else:
            queries, p0 = case["L"], case["N"] - case["L"]
            full = max(0, min(case["L"], p0 + case["L"] + 1 - case["top_k"]))
            slots = full * case["top_k"] + sum(p0 + i + 1 for i in range(case["L"] - full))
            keys = min(case["N"], slots)                     # the rows are shared by the queries
        shared = keys * _row_bytes(case.get("format", "q4")) + queries * (HEADS * (2 * QK + 4) + 4 * case["top_k"])
        if op == "weights":
            return {"bytes": shared + 4 * case["N"] * case.get("B", 1), "flops": slots * HEADS * QK * 2}
        return {"bytes": shared + queries * HEADS * 2 * LATENT, "flops": slots * HEADS * (QK + LATENT) * 2}
    if op == "store":
        return {"bytes": case["R"] * (2 * QK + 4 * ROPE + 12 + 2 * (ROW4 + 4) + 2 * QK) + 4 * LATENT,
                "flops": case["R"] * (20 * LATENT + 3 * ROPE)}
    lens = _lens(case)
    over = [n for n in lens if n > case["keep"]]
    # of the keys behind the budget's end, the share that stays (a lower bound of what moves)
    moved = sum((n - case["keep"]) * case["keep"] // n for n in over)
    return {"bytes": 8 * sum(lens) + 4 * len(lens) + moved * (8 + 2 * (2 * QK + 2 * IDX_DIM + 8)), "flops": 4 * sum(lens)}


def _lens(case):
    """Keys of each sequence: all N, or uneven ones (the first full, one unused slot in a batch of several)."""
    B, N = case["B"], case["N"]
    if not case.get("ragged"):
        return [N] * B
    lens = [max(1, N - (i * 7919 * N // 10007) % N) for i in range(B)]
    lens[0] = N
    if B > 2:
        lens[B - 1] = 0
    return lens


# ------------------------------------------------------------------------------------------------ inputs

def _angles(n):
    """cos | sin of positions 0..n-1 for 32 frequencies, [n, 64] float32 (angles in 64 bits)."""
    freq = 10000.0 ** (-torch.arange(ROPE // 2, dtype=torch.float64, device="cuda") / (ROPE // 2))
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _latents(g, rows):
    """Values like a normalised latent's."""
    return torch.randn(rows, LATENT, generator=g, device="cuda") * torch.exp(0.4 * torch.randn(LATENT, generator=g, device="cuda"))


def _cache(g, fmt, rows):
    """A filled cache: bf16 rows, or the rows of an 8-bit or 4-bit one with a power-of-two scale a row."""
    u = _latents(g, rows)
    rope = torch.randn(rows, ROPE, generator=g, device="cuda").bfloat16()
    if fmt == "bf16":
        return torch.cat([u.bfloat16(), rope], 1), None
    if fmt == "q4":
        codes, blocks, scale = _pack(u.double())
        return torch.cat([codes, blocks, rope.view(torch.uint8)], 1), scale
    _, e = torch.frexp(u.abs().amax(1) / 448.0)
    scale = torch.ldexp(torch.ones(rows, device="cuda"), e)
    latent = (u / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([latent, rope.view(torch.uint8)], 1), scale


def _pages(g, lens, N, page):
    """A shuffled page table for sequences of these lengths, two pages of the pool unused."""
    stride = -(-N // page)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 2
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), stride), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pages


def _selection(g, count, N, top_k):
    """For each query a random choice of min(top_k, count) of its `count` keys, ascending, -1 padded."""
    order = torch.rand(count.numel(), N, generator=g, device="cuda")
    j = torch.arange(N, device="cuda")
    order.masked_fill_(j[None, :] >= count[:, None], -1.0)
    k = min(top_k, N)
    val, idx = torch.topk(order, k, dim=1)
    idx = idx.masked_fill(val < 0, N).sort(1).values
    idx = idx.masked_fill(idx == N, -1).int()
    if k < top_k:
        idx = torch.cat([idx, torch.full((idx.shape[0], top_k - k), -1, dtype=torch.int32, device="cuda")], 1)
    return idx.contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("decode", "prefill", "weights"):
        N, page, batch = case["N"], case["page"], "B" in case
        lens = _lens(case) if batch else [N]
        if page:
            s["table"], pages = _pages(g, lens, N, page)
            s["cache"], s["scale"] = _cache(g, case.get("format", "q4"), pages * page)
        else:
            s["cache"], s["scale"] = _cache(g, case.get("format", "q4"), len(lens) * N)
            if batch:
                s["cache"] = s["cache"].view(len(lens), N, -1)
                s["scale"] = None if s["scale"] is None else s["scale"].view(len(lens), N)
        s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        count = s["kv_len"] if batch else torch.arange(N - case["L"], N, device="cuda") + 1
        s["idx"] = _selection(g, count, N, case["top_k"])
        s["q"] = torch.randn(count.numel(), HEADS, QK, generator=g, device="cuda").bfloat16()
        s["lse"] = torch.empty(count.numel(), HEADS, device="cuda")
        if op == "weights":
            s["lse"].copy_(_lse(_scores(s)[0])[0])           # of the attention over the same selection
        else:                                                # a serving loop keeps its output buffers
            s["out"] = torch.empty(count.numel(), HEADS, LATENT, dtype=torch.bfloat16, device="cuda")
    elif op == "store":
        R, rows = case["R"], case["rows"]
        s["kv_a"] = (2.0 * torch.randn(R, case["ld"], generator=g, device="cuda")).bfloat16()[:, :QK]
        s["w"] = torch.exp(0.4 * torch.randn(LATENT, generator=g, device="cuda"))
        s["cos_sin"] = _angles(8192)
        s["pos"] = torch.randint(0, 8192, (R,), generator=g, device="cuda").int()
        s["slots"] = torch.randperm(rows, generator=g, device="cuda")[:R].int()
        if R > 2:
            s["slots"][R - 1] = -1                           # a padding row of the batch
        s["cache"], s["scale"] = _cache(g, "q4", rows)
        s["out"] = torch.empty(R, QK, dtype=torch.bfloat16, device="cuda")
    else:
        B, N, page = case["B"], case["N"], case["page"]
        lens = _lens(case)
        s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # what a few hundred steps leave: few heavy keys, many light ones, some that were never selected
        acc = torch.exp(3.0 * torch.randn(B, N, generator=g, device="cuda"))
        s["acc"] = acc.masked_fill_(torch.rand(B, N, generator=g, device="cuda") < 0.1, 0.0)
        # positions of the keys, out of order as earlier evictions leave them
        s["pos"] = torch.rand(B, N, generator=g, device="cuda").argsort(1).int() * 2 + 1
        if page:
            s["table"], pages = _pages(g, lens, N, page)
        rows = pages * page if page else B * N
        shape = (rows,) if page else (B, N)
        s["kv"] = torch.randn(rows, QK, generator=g, device="cuda").bfloat16().view(*shape, QK)
        s["k"] = torch.randn(rows, IDX_DIM, generator=g, device="cuda").bfloat16().view(*shape, IDX_DIM)
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        import deepseek_sparse_attention_indexer_gb300 as dsa
        if c["op"] == "decode":
            if c["page"]:
                dsa.mla_sparse_attn_decode_q4_paged(s["q"], s["cache"], s["scale"], s["kv_len"], s["table"], c["page"],
                                                    s["idx"], SCALE, c["N"], out=s["out"], lse=s["lse"])
            else:
                dsa.mla_sparse_attn_decode_q4(s["q"], s["cache"], s["scale"], s["kv_len"], s["idx"], SCALE, out=s["out"],
                                              lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if c["op"] == "prefill":
            if c["page"]:
                dsa.mla_sparse_attn_prefill_q4_paged(s["q"], s["cache"], s["scale"], s["table"], c["page"], s["idx"], SCALE,
                                                     c["N"], out=s["out"], lse=s["lse"])
            else:
                dsa.mla_sparse_attn_prefill_q4(s["q"], s["cache"], s["scale"], s["idx"], SCALE, out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if c["op"] == "store":
            dsa.mla_cache_write_q4(s["kv_a"], s["w"], EPS, s["cos_sin"], s["pos"], s["slots"], s["cache"], s["scale"],
                                   interleave=c["interleave"])
            dsa.mla_cache_read_q4(s["cache"], s["scale"], s["slots"], out=s["out"])
            return {"rows": s["out"], "scale": s["scale"]}
        if c["op"] == "weights":
            pages = {"block_table": s["table"], "page_size": c["page"]} if c["page"] else {}
            if "B" in c:
                return dsa.mla_key_weights_decode(s["q"], s["cache"], s["kv_len"], s["idx"], s["lse"], SCALE,
                                                  cache_scale=s["scale"], Nmax=c["N"], **pages)
            return dsa.mla_key_weights_prefill(s["q"], s["cache"], s["idx"], s["lse"], SCALE, cache_scale=s["scale"],
                                               N=c["N"], **pages)
        src, dst, left = dsa.cache_evict_plan(s["acc"], s["pos"], s["kv_len"], c["keep"], recent=c["recent"], sink=c["sink"])
        if c["page"]:
            dsa.cache_move_rows(src, dst, dense=(s["acc"], s["pos"]), paged=(s["kv"], s["k"]), block_table=s["table"],
                                page_size=c["page"])
        else:
            dsa.cache_move_rows(src, dst, dense=(s["kv"], s["k"], s["acc"], s["pos"]))
        return _evicted(s, src, dst, left)
    return {"decode": _attention, "prefill": _attention, "store": _store, "weights": _weights, "evict": _evict}[c["op"]](s)


def _evicted(s, src, dst, left):
    """The plan and the caches, as the bits that were moved."""
    return {"src": src, "dst": dst, "left": left, "kv": s["kv"].view(torch.int16), "k": s["k"].view(torch.int16),
            "acc": s["acc"].view(torch.int32), "pos": s["pos"]}


def _pack(u):
    """4-bit rows of u [rows, 512] in float64: codes [rows, 256], block bytes [rows, 32], scale [rows] float32."""
    v = u.abs().unflatten(1, (LATENT // BLOCK, BLOCK))
    m, e = torch.frexp(v.amax(2))                            # amax = m 2^e with m in [1/2, 1); 6 s, s = (1 + q/4) 2^j
    q = torch.where(m <= 0.5625, 2, torch.where(m <= 0.75, 0, torch.where(m <= 0.9375, 1, 2)))
    j = torch.where(m <= 0.5625, e - 4, e - 3)
    j = torch.where(m == 0, torch.full_like(j, -100000), j)
    k = (j.amax(1) - 5).clamp(-64, 64)                       # the heaviest block's scale is (1 + q/4) 2^5 c
    a = j - k[:, None] + 6
    a, q = torch.where(a < 0, 0, torch.where(a > 11, 11, a)), torch.where(a < 0, 0, torch.where(a > 11, 2, q))
    step = torch.ldexp(1.0 + q.double() / 4, a - 6 + k[:, None])[:, :, None]
    code = torch.zeros_like(v, dtype=torch.int32)            # halves go to the even code
    for i, t in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (v >= t * step) if i % 2 else (v > t * step)
    code, neg = code.view(-1, 64, 8), (torch.signbit(u) & (u != 0)).int().view(-1, 64, 8)
    codes = code[:, :, 0::2] | (code[:, :, 1::2] << 4) | (neg[:, :, 4:] << 3) | (neg[:, :, :4] << 7)
    return codes.flatten(1).byte(), (3 * a + q).byte(), torch.ldexp(torch.ones_like(k, dtype=torch.float32), k)


def _rows(cache, scale):
    """Cache rows in float32, [rows, 576]."""
    cache = cache.reshape(-1, cache.shape[-1])
    if scale is None:
        return cache.float()
    scale = scale.reshape(-1)[:, None]
    if cache.shape[1] == ROW8:
        latent = cache[:, :LATENT].view(torch.float8_e4m3fn).float()
    else:
        c = cache[:, :LATENT // 2].int().unflatten(1, (64, 4))
        code = torch.stack([c & 7, (c >> 4) & 7], -1).flatten(2)
        sign = 1 - 2 * torch.cat([c >> 7, (c >> 3) & 1], 2)
        b = cache[:, LATENT // 2:LATENT // 2 + LATENT // BLOCK].int()
        block = torch.where(b < 36, torch.ldexp(1.0 + (b % 3) / 4, b // 3 - 6), 0.0)
        mag = torch.tensor(MAG, device=cache.device)[code]
        latent = (mag * sign).flatten(1).unflatten(1, (-1, BLOCK)).mul(block[:, :, None]).flatten(1)
    return torch.cat([latent * scale, cache[:, -2 * ROPE:].contiguous().view(torch.bfloat16).float()], dim=1)


def _places(s):
    """The pool row of each selected key (0 where nothing is selected)."""
    c, j = s["case"], s["idx"].long().clamp(min=0)
    seq = torch.arange(j.shape[0], device=j.device)[:, None] if "B" in c else torch.zeros_like(j[:, :1])
    if c["page"]:
        return s["table"].long()[seq, j // c["page"]].clamp(min=0) * c["page"] + j % c["page"]
    return seq * c["N"] + j


def _scores(s):
    """Scaled scores [queries, 64, top_k], -inf where nothing is selected, and the selected rows."""
    at = _places(s)
    if "B" not in s["case"]:                                             # queries share rows: widen each row once
        kv = _rows(s["cache"], s["scale"])[at]                           # [queries, top_k, 576]
    else:
        scale = None if s["scale"] is None else s["scale"].reshape(-1)[at]
        kv = _rows(s["cache"].reshape(-1, s["cache"].shape[-1])[at], scale).unflatten(0, at.shape)
    x = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * SCALE
    return x.masked_fill((s["idx"] < 0)[:, None, :], -math.inf), kv


def _lse(x):
    """log of the sum of the exponentials, [queries, 64], the exponentials over the largest, and their sum."""
    m = x.amax(2, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    z = p.sum(2, keepdim=True)
    return (m + z.log())[:, :, 0], p, z


def _attention(s):
    x, kv = _scores(s)
    lse, p, z = _lse(x)
    o = torch.matmul(p, kv[:, :, :LATENT]) / torch.where(z == 0, torch.ones_like(z), z)
    return {"out": o.bfloat16(), "lse": lse}


def _weights(s):
    c = s["case"]
    x, _ = _scores(s)
    lse = torch.where(s["lse"] == -math.inf, 0.0, s["lse"])              # a query without a key
    w = torch.exp(x - lse[:, :, None]).sum(1)                            # [queries, top_k]
    j = torch.where(s["idx"] < 0, 0, s["idx"]).long()                    # weight 0 where nothing is selected
    if "B" in c:
        return torch.zeros(c["B"], c["N"], device=w.device).scatter_add_(1, j, w)
    acc = torch.zeros(c["N"], dtype=torch.float64, device=w.device)      # a long sum: 64 bits
    return acc.index_add_(0, j.flatten(), w.flatten().double()).float()


def _rotate(x, cos_sin, pos, interleave):
    """Rotates the last dim's 32 pairs: neighbours (2i, 2i + 1), or halves (i, i + 32)."""
    t = cos_sin[pos.long()]
    c, n = t[:, :ROPE // 2], t[:, ROPE // 2:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleave else (x[..., :ROPE // 2], x[..., ROPE // 2:])
    u, v = a * c - b * n, b * c + a * n
    return torch.stack([u, v], -1).flatten(-2) if interleave else torch.cat([u, v], -1)


def _scatter(dst, slots, rows):
    """dst with rows[r] at slots[r]; negative slots left out."""
    n = dst.shape[0]
    src = torch.full((n + 1,), -1, dtype=torch.long, device=dst.device)
    src[torch.where(slots < 0, n, slots).long()] = torch.arange(rows.shape[0], device=dst.device)
    src = src[:n]
    mask = (src >= 0).view(-1, *[1] * (dst.dim() - 1))
    dst.copy_(torch.where(mask, rows[src.clamp(min=0)], dst))


def _store(s):
    x = s["kv_a"][:, :LATENT].double()                                   # 64 bits: values next to a border of the codes
    u = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["w"].double()
    codes, blocks, scale = _pack(u)
    rope = _rotate(s["kv_a"][:, LATENT:].float(), s["cos_sin"], s["pos"], s["case"]["interleave"]).bfloat16()
    _scatter(s["cache"], s["slots"], torch.cat([codes, blocks, rope.view(torch.uint8)], 1))
    _scatter(s["scale"], s["slots"], scale)
    at = s["slots"].long().clamp(min=0)
    s["out"].copy_(_rows(s["cache"][at], s["scale"][at]) * (s["slots"] >= 0)[:, None])
    return {"rows": s["out"], "scale": s["scale"]}


def _evict(s):
    c, acc, pos = s["case"], s["acc"], s["pos"]
    B, N = acc.shape
    j = torch.arange(N, device=acc.device)
    have = j < s["kv_len"][:, None]
    newest = torch.where(have, pos, -2 ** 31).amax(1, keepdim=True)
    safe = (pos > newest - c["recent"]) | (pos < c["sink"])
    rank = torch.where(safe, math.inf, acc).masked_fill(~have, -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    stay = torch.zeros_like(have).scatter_(1, order[:, :c["keep"]], True) & have
    src, dst, left = _moves(stay, s["kv_len"], c["keep"])
    b, m = (src >= 0).nonzero(as_tuple=True)
    f, t = src[b, m].long(), dst[b, m].long()
    if c["page"]:
        row = lambda x: s["table"][b, x // c["page"]].long() * c["page"] + x % c["page"]  # noqa: E731
        s["kv"][row(t)], s["k"][row(t)] = s["kv"][row(f)], s["k"][row(f)]
    else:
        s["kv"][b, t], s["k"][b, t] = s["kv"][b, f], s["k"][b, f]
    acc[b, t], pos[b, t] = acc[b, f], pos[b, f]
    return _evicted(s, src, dst, left)


def _moves(stay, kv_len, keep):
    """Source and destination of each move [B, min(keep, N - keep)], -1 padded, and the keys left [B]: the i-th place
    below `keep` whose key goes is filled from the i-th key from `keep` on that stays."""
    B, N = stay.shape
    front = torch.arange(N, device=stay.device) < keep
    much = (kv_len > keep)[:, None]
    most = min(keep, N - keep)

    def listed_places(mask):
        out = torch.full((B, most + 1), -1, dtype=torch.int32, device=mask.device)
        at = torch.where(mask, mask.int().cumsum(1) - 1, most)
        out.scatter_(1, at, torch.where(mask, torch.arange(N, device=mask.device, dtype=torch.int32), -1))
        return out[:, :most].contiguous()

    return listed_places(stay & ~front & much), listed_places(~stay & front & much), kv_len.clamp(max=keep)


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    if case["op"] == "evict":                                            # chooses and moves, computes nothing
        return None
    s = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(s, case)
    return _exact_attention(s, case)


def _exact_quantised(u):
    """Rows of u in float64 as the values that the 4-bit format holds them as, and the scale a row."""
    b = u.view(-1, LATENT // BLOCK, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    # every block scale at the row's scale 1: 36 of them; the smallest that reaches top / 6
    steps = torch.tensor([(1 + m / 4) * 2.0 ** (a - 6) for a in range(12) for m in range(3)], dtype=torch.float64, device=u.device)
    # the row's scale: the power of two by which the largest block's scale lies in [2^5, 2^6)
    want = top.amax((1, 2)) / 6
    e = torch.floor(torch.log2(want))
    f = want / torch.exp2(e)                                             # in [1, 2): above 1.5 the next power of two
    e = torch.where(f > 1.5, e + 1, e)
    c = torch.exp2((e - 5).clamp(-64, 64))
    fits = 6 * steps * c[:, None, None] >= top                           # [rows, blocks, 36]
    step = steps[fits.int().argmax(2)][:, :, None] * c[:, None, None]
    mags = torch.tensor(MAG, dtype=torch.float64, device=u.device)
    v = b.abs() / step
    hi = torch.bucketize(v, mags).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    dl, dh = v - mags[lo], mags[hi] - v
    near = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (torch.sign(b) * mags[near] * step).flatten(1), c


def _exact_store(s, case):
    x = s["kv_a"].double()
    lat = x[:, :LATENT]
    u = lat / (torch.linalg.vector_norm(lat, dim=1, keepdim=True) ** 2 / LATENT + EPS).sqrt() * s["w"].double()
    value, c = _exact_quantised(u)
    pos = s["pos"].long()
    turn = torch.complex(s["cos_sin"][pos, :32].double(), s["cos_sin"][pos, 32:].double())
    pairs = x[:, LATENT:].unflatten(-1, (32, 2)) if case["interleave"] else x[:, LATENT:].unflatten(-1, (2, 32)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    rope = z.flatten(-2) if case["interleave"] else z.transpose(-1, -2).flatten(-2)
    kept = s["slots"] >= 0
    scale = s["scale"].double()
    scale[s["slots"][kept].long()] = c[kept]
    return {"rows": torch.cat([value, rope], 1) * kept[:, None], "scale": scale}


def _exact_row(s, at):
    """Cache rows `at` (any shape) as the float64 values they stand for."""
    raw = s["cache"].reshape(-1, s["cache"].shape[-1])[at]
    if s["scale"] is None:
        return raw.double()
    c = s["scale"].reshape(-1)[at].double().unsqueeze(-1)
    rope = raw[..., -2 * ROPE:].contiguous().view(torch.bfloat16).double()
    if raw.shape[-1] == ROW8:
        return torch.cat([raw[..., :LATENT].contiguous().view(torch.float8_e4m3fn).double() * c, rope], -1)
    d = torch.arange(LATENT, device=raw.device)
    group, i = 4 * (d // 8), d % 8
    mag = (raw[..., group + i // 2] >> (4 * (i % 2)).byte()) & 7
    sign = raw[..., group + i % 4] & torch.where(i < 4, 128, 8).byte()
    block = raw[..., 256 + d // BLOCK].long()
    power = torch.exp2((block.double() / 3).floor() - 6)
    mags = torch.tensor(MAG, dtype=torch.float64, device=raw.device)[mag.long()]
    value = torch.where(sign > 0, -mags, mags) * power * (4 + block.remainder(3)) / 4 * c
    return torch.cat([torch.where(block > 35, 0.0, value), rope], -1)


def _exact_attention(s, case):
    n = s["q"].shape[0]
    batch, weights = "B" in case, case["op"] == "weights"
    out = torch.zeros(n, HEADS, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((n, HEADS), -math.inf, dtype=torch.float64, device="cuda")
    acc = torch.zeros(case.get("B", 1) * case["N"], dtype=torch.float64, device="cuda")
    for i in range(0, n, 32):
        j = s["idx"][i:i + 32].long()
        have = j >= 0
        at = torch.where(have, j, 0)
        seq = torch.arange(i, i + at.shape[0], device="cuda")[:, None] if batch else torch.zeros_like(at[:, :1])
        key = at + seq * case["N"]
        if case["page"]:
            at = s["table"][seq, at // case["page"]].long().clamp(min=0) * case["page"] + at % case["page"]
        else:
            at = key
        kv = _exact_row(s, at)
        x = torch.einsum("qhd,qkd->qhk", s["q"][i:i + 32].double(), kv) * SCALE
        x = torch.where(have[:, None, :], x, -math.inf)
        if weights:
            w = torch.exp(x - s["lse"][i:i + 32].double()[:, :, None]).sum(1)
            acc.index_add_(0, key[have], w[have])
            continue
        lse[i:i + 32] = torch.logsumexp(x, 2)
        p = torch.nan_to_num(torch.softmax(x, 2), nan=0.0)              # no key at all: zeros
        out[i:i + 32] = torch.einsum("qhk,qkd->qhd", p, kv[..., :LATENT])
    if weights:
        return acc.view(case["B"], case["N"]) if batch else acc
    return {"out": out, "lse": lse}
