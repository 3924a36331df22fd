"""The operators around the 8-bit latent cache, as cases to be measured.

Four operators, each in its plain form (elementary torch operations) and as the call a user makes:

* ``write``: RMS norm of the 512 latent dims, rotation of the 64 rope dims, quantisation to a cache row
  (512 x e4m3 | 64 x bf16, one power-of-two scale a row) and the scatter of the rows to their slots;
* ``read``: cache rows back to bf16, by slot list or through a page table;
* ``decode`` / ``prefill``: sparse absorbed-MLA attention over the 8-bit cache, dense or paged;
* ``index``: norm and rotation of the indexer's queries and keys, the keys scattered to their cache.

``run`` takes the plain form unless ``own`` is set; ``exact`` gives the results in 64 bits.
"""
import math

import torch

own = False

HEADS, QK, LATENT, ROPE, ROW = 64, 576, 512, 64, 640      # attention heads, widths, bytes of a cache row
IDX_HEADS, IDX_DIM = 32, 128                               # indexer heads and width
SCALE = 1.0 / 16.0                                         # 1 / sqrt(192 + 64)
EPS = 1e-6
TOP = 2048
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one user, one new token over a 4k context: pure latency
        {"name": "decode_b1", "op": "decode", "B": 1, "N": 4096, "top_k": 2048, "page": 0, "ragged": False},
        # a small serving batch over 64-row pages
        {"name": "decode_b8_paged", "op": "decode", "B": 8, "N": 4096, "top_k": 2048, "page": 64, "ragged": False},
        # an odd batch of short contexts, fewer keys than a full selection, one slot of the batch unused
        {"name": "decode_b37_short", "op": "decode", "B": 37, "N": 1003, "top_k": 700, "page": 0, "ragged": True},
        # a full serving batch of uneven contexts over pages: HBM counts
        {"name": "decode_b256_paged", "op": "decode", "B": 256, "N": 8192, "top_k": 2048, "page": 64, "ragged": True},
        # a prefill chunk's tail, its pages of 16 rows, sizes that fit no tile
        {"name": "prefill_333_paged", "op": "prefill", "L": 333, "N": 5001, "top_k": 2048, "page": 16},
        # the benchmark's prefill chunk: 4096 queries at 16k keys
        {"name": "prefill_16k", "op": "prefill", "L": 4096, "N": 16384, "top_k": 2048, "page": 0},
        # a decode step's new tokens into the cache: latency
        {"name": "write_8", "op": "write", "R": 8, "rows": 8 * 4096, "ld": 1024, "interleave": True},
        # a prefill chunk's rows into the cache
        {"name": "write_4096", "op": "write", "R": 4096, "rows": 6144, "ld": 576, "interleave": True},
        # eight uneven contexts back to bf16
        {"name": "read_b8_paged", "op": "read", "B": 8, "N": 4096, "page": 64},
        # the rows of a 64k context back to bf16, by slot
        {"name": "read_64k", "op": "read", "B": 1, "N": 65536, "page": 0},
        # the indexer's inputs of a decode step
        {"name": "index_8", "op": "index", "R": 8, "rows": 8 * 4096, "norm": "layer", "q_norm": False, "interleave": True},
        # the indexer's inputs of a prefill chunk, queries normalised too, half-split rotation
        {"name": "index_4096", "op": "index", "R": 4096, "rows": 5000, "norm": "rms", "q_norm": True, "interleave": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "write", "read", "index"])
    page = rng.choice([0, 16, 64, 256])
    if op == "decode":
        return {"op": op, "B": _log(rng, 1, 256), "N": _log(rng, 1, 8192), "top_k": _log(rng, 1, TOP), "page": page,
                "ragged": rng.random() < 0.5}
    if op == "prefill":
        n = _log(rng, 64, 32768)
        return {"op": op, "L": min(n, _log(rng, 1, 4095)), "N": n, "top_k": _log(rng, 1, TOP), "page": page}
    if op == "write":
        r = _log(rng, 1, 8192)
        return {"op": op, "R": r, "rows": r + rng.randint(0, 4096), "ld": rng.choice([576, 584, 1024]),
                "interleave": rng.random() < 0.5}
    if op == "read":
        return {"op": op, "B": _log(rng, 1, 16), "N": _log(rng, 1, 8192), "page": page}
    r = _log(rng, 1, 4096)
    return {"op": op, "R": r, "rows": r + rng.randint(0, 4096), "norm": rng.choice(["rms", "layer"]),
            "q_norm": rng.random() < 0.5, "interleave": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op in ("decode", "prefill"):
        if op == "decode":
            queries = case["B"]
            lens = _lens(case)
            slots = sum(min(n, case["top_k"]) for n in lens)
            keys = slots                                     # each sequence reads its own rows
        else:
            queries, p0 = case["L"], case["N"] - case["L"]
            full = max(0, min(case["L"], p0 + case["L"] + 1 - case["top_k"]))
            slots = full * case["top_k"] + sum(p0 + i + 1 for i in range(case["L"] - full))
            keys = min(case["N"], slots)                     # the rows are shared by the queries
        nbytes = keys * (ROW + 4) + queries * (HEADS * (2 * QK + 2 * LATENT + 4) + 4 * case["top_k"])
        return {"bytes": nbytes, "flops": slots * HEADS * (QK + LATENT) * 2}
    if op == "write":
        return {"bytes": case["R"] * (2 * QK + 4 * ROPE + 8 + ROW + 4) + 4 * LATENT, "flops": case["R"] * (6 * LATENT + 3 * ROPE)}
    if op == "read":
        n = sum(_lens(dict(case, ragged=case["B"] > 1)))
        return {"bytes": n * (ROW + 4 + 2 * QK), "flops": n * LATENT}
    per = 2 * IDX_DIM * (IDX_HEADS + 1)
    return {"bytes": case["R"] * (2 * per + 4 * ROPE + 8), "flops": case["R"] * (IDX_HEADS + 1) * 8 * IDX_DIM}


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


def _cache(g, rows):
    """A filled 8-bit cache: values like a normalised latent's, a power-of-two scale a row."""
    w = torch.exp(0.4 * torch.randn(LATENT, generator=g, device="cuda"))
    u = torch.randn(rows, LATENT, generator=g, device="cuda") * w
    _, e = torch.frexp(u.abs().amax(1) / E4M3_MAX)
    scale = torch.ldexp(torch.ones(rows, device="cuda"), e)
    cache = torch.empty(rows, ROW, dtype=torch.uint8, device="cuda")
    cache[:, :LATENT] = (u / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    rope = torch.randn(rows, ROPE, generator=g, device="cuda").bfloat16()
    cache[:, LATENT:] = rope.view(torch.uint8)
    return cache, scale


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
    if op in ("decode", "prefill"):
        N, page = case["N"], case["page"]
        lens = _lens(case) if op == "decode" else [N]
        if page:
            s["table"], pages = _pages(g, lens, N, page)
            s["cache"], s["scale"] = _cache(g, pages * page)
        else:
            s["cache"], s["scale"] = _cache(g, len(lens) * N)
            if op == "decode":
                s["cache"], s["scale"] = s["cache"].view(len(lens), N, ROW), s["scale"].view(len(lens), N)
        s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        count = s["kv_len"] if op == "decode" else torch.arange(N - case["L"], N, device="cuda") + 1
        s["idx"] = _selection(g, count, N, case["top_k"])
        s["q"] = torch.randn(count.numel(), HEADS, QK, generator=g, device="cuda").bfloat16()
        # a serving loop keeps its output buffers
        s["out"] = torch.empty(count.numel(), HEADS, LATENT, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(count.numel(), HEADS, device="cuda")
    elif op == "write":
        R, rows = case["R"], case["rows"]
        s["kv_a"] = (2.0 * torch.randn(R, case["ld"], generator=g, device="cuda")).bfloat16()[:, :QK]
        s["w"] = torch.exp(0.4 * torch.randn(LATENT, generator=g, device="cuda"))
        s["cos_sin"] = _angles(8192)
        s["pos"] = torch.randint(0, 8192, (R,), generator=g, device="cuda").int()
        s["slots"] = torch.randperm(rows, generator=g, device="cuda")[:R].int()
        if R > 2:
            s["slots"][R - 1] = -1                           # a padding row of the batch
        s["cache"], s["scale"] = _cache(g, rows)
        s["latent"] = s["cache"][:, :LATENT].view(torch.float8_e4m3fn)
        s["rope"] = s["cache"][:, LATENT:].view(torch.bfloat16)
    elif op == "read":
        lens = _lens(dict(case, ragged=case["B"] > 1))
        B, N, page = case["B"], case["N"], case["page"]
        if page:
            s["table"], pages = _pages(g, lens, N, page)
            s["cache"], s["scale"] = _cache(g, pages * page)
            s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
            s["out"] = torch.zeros(B, N, QK, dtype=torch.bfloat16, device="cuda")
        else:
            s["cache"], s["scale"] = _cache(g, B * N)
            slots = torch.randperm(B * N, generator=g, device="cuda").view(B, N)
            past = torch.arange(N, device="cuda")[None, :] >= torch.tensor(lens, device="cuda")[:, None]
            s["slots"] = slots.masked_fill(past, -1).flatten().int()
            s["out"] = torch.zeros(B * N, QK, dtype=torch.bfloat16, device="cuda")
    else:
        R, rows = case["R"], case["rows"]
        s["q"] = (3.0 * torch.randn(R, IDX_HEADS, IDX_DIM, generator=g, device="cuda")).bfloat16()
        s["k"] = (3.0 * torch.randn(R, IDX_DIM, generator=g, device="cuda") + 0.5).bfloat16()
        s["k_w"] = torch.exp(0.3 * torch.randn(IDX_DIM, generator=g, device="cuda"))
        s["k_b"] = 0.2 * torch.randn(IDX_DIM, generator=g, device="cuda") if case["norm"] == "layer" else None
        s["q_w"] = torch.exp(0.3 * torch.randn(IDX_DIM, generator=g, device="cuda")) if case["q_norm"] else None
        s["cos_sin"] = _angles(8192)
        s["pos"] = torch.randint(0, 8192, (R,), generator=g, device="cuda").int()
        s["slots"] = torch.randperm(rows, generator=g, device="cuda")[:R].int()
        s["q_out"] = torch.empty_like(s["q"])
        s["k_cache"] = torch.randn(rows, IDX_DIM, generator=g, device="cuda").bfloat16()
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        import deepseek_sparse_attention_indexer_gb300 as dsa
        if c["op"] == "decode":
            if c["page"]:
                dsa.mla_sparse_attn_decode_q8_paged(s["q"], s["cache"], s["scale"], s["kv_len"], s["table"], c["page"],
                                                    s["idx"], SCALE, c["N"], out=s["out"], lse=s["lse"])
            else:
                dsa.mla_sparse_attn_decode_q8(s["q"], s["cache"], s["scale"], s["kv_len"], s["idx"], SCALE, out=s["out"],
                                              lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if c["op"] == "prefill":
            if c["page"]:
                dsa.mla_sparse_attn_prefill_q8_paged(s["q"], s["cache"], s["scale"], s["table"], c["page"], s["idx"], SCALE,
                                                     c["N"], out=s["out"], lse=s["lse"])
            else:
                dsa.mla_sparse_attn_prefill_q8(s["q"], s["cache"], s["scale"], s["idx"], SCALE, out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if c["op"] == "write":
            dsa.mla_cache_write_q8(s["kv_a"], s["w"], EPS, s["cos_sin"], s["pos"], s["slots"], s["cache"], s["scale"],
                                   interleave=c["interleave"])
            return {"latent": s["latent"], "rope": s["rope"], "scale": s["scale"]}
        if c["op"] == "read":
            if c["page"]:
                return dsa.mla_cache_read_q8_paged(s["cache"], s["scale"], s["kv_len"], s["table"], c["page"], c["N"],
                                                   out=s["out"])
            return dsa.mla_cache_read_q8(s["cache"], s["scale"], s["slots"], out=s["out"])
        q = dsa.indexer_norm_rope(s["q"], s["k"], s["k_w"], s["k_b"], EPS, s["cos_sin"], s["pos"], s["slots"], s["k_cache"],
                                  q_w=s["q_w"], norm=c["norm"], interleave=c["interleave"], q_out=s["q_out"])
        return {"q": q, "k": s["k_cache"]}
    return {"decode": _attention, "prefill": _attention, "write": _write, "read": _read, "index": _index}[c["op"]](s)


def _rows(cache, scale):
    """Every cache row in float32, [rows, 576]."""
    cache, scale = cache.reshape(-1, ROW), scale.reshape(-1)
    latent = cache[:, :LATENT].view(torch.float8_e4m3fn).float() * scale[:, None]
    return torch.cat([latent, cache[:, LATENT:].view(torch.bfloat16).float()], dim=1)


def _places(s):
    """The pool row of each selected key (0 where nothing is selected)."""
    c, j = s["case"], s["idx"].long().clamp(min=0)
    seq = torch.arange(j.shape[0], device=j.device)[:, None] if c["op"] == "decode" else torch.zeros_like(j[:, :1])
    if c["page"]:
        return s["table"].long()[seq, j // c["page"]].clamp(min=0) * c["page"] + j % c["page"]
    return seq * c["N"] + j


def _attention(s):
    at = _places(s)
    if s["case"]["op"] == "prefill":                                     # queries share rows: widen each row once
        kv = _rows(s["cache"], s["scale"])[at]                           # [queries, top_k, 576]
    else:
        kv = _rows(s["cache"].reshape(-1, ROW)[at], s["scale"].reshape(-1)[at]).unflatten(0, at.shape)
    x = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * SCALE         # [queries, 64, top_k]
    x = x.masked_fill((s["idx"] < 0)[:, None, :], -math.inf)
    m = x.amax(2, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    z = p.sum(2, keepdim=True)
    o = torch.matmul(p, kv[:, :, :LATENT]) / torch.where(z == 0, torch.ones_like(z), z)
    return {"out": o.bfloat16(), "lse": (m + z.log())[:, :, 0]}


def _rotate(x, cos_sin, pos, interleave):
    """Rotates the last dim's 32 pairs: neighbours (2i, 2i + 1), or halves (i, i + 32)."""
    t = cos_sin[pos.long()]
    c, n = t[:, :ROPE // 2], t[:, ROPE // 2:]
    if x.dim() == 3:
        c, n = c[:, None, :], n[:, None, :]
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


def _write(s):
    x = s["kv_a"].float()
    c = x[:, :LATENT]
    u = c * torch.rsqrt(c.square().mean(1, keepdim=True) + EPS) * s["w"]
    m, e = torch.frexp(u.abs().amax(1))                                  # amax = m 2^e with m in [1/2, 1); 448 = 7/8 2^9
    k = torch.where(m > 0.875, e - 8, e - 9).clamp(-64, 64)
    scale = torch.ldexp(torch.ones_like(m), torch.where(m == 0, torch.zeros_like(k), k))
    latent = (u / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    rope = _rotate(x[:, LATENT:], s["cos_sin"], s["pos"], s["case"]["interleave"]).bfloat16()
    _scatter(s["cache"], s["slots"], torch.cat([latent.view(torch.uint8), rope.view(torch.uint8)], 1))
    _scatter(s["scale"], s["slots"], scale)
    return {"latent": s["latent"], "rope": s["rope"], "scale": s["scale"]}


def _read(s):
    c = s["case"]
    rows = _rows(s["cache"], s["scale"]).bfloat16()
    if c["page"]:
        j = torch.arange(c["N"], device=rows.device)
        at = s["table"].long()[:, j // c["page"]].clamp(min=0) * c["page"] + j % c["page"]
        s["out"].copy_(torch.where((j[None, :] < s["kv_len"][:, None])[:, :, None], rows[at], s["out"]))
    else:
        s["out"].copy_(rows[s["slots"].long().clamp(min=0)] * (s["slots"] >= 0)[:, None])
    return s["out"]


def _norm(x, kind, w, b):
    if w is None:
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    return x if b is None else x + b


def _index(s):
    c = s["case"]

    def made(x, w, b):
        x = _norm(x.float(), c["norm"], w, b)
        return torch.cat([_rotate(x[..., :ROPE], s["cos_sin"], s["pos"], c["interleave"]), x[..., ROPE:]], -1).bfloat16()

    q = made(s["q"], s["q_w"], None)
    _scatter(s["k_cache"], s["slots"], made(s["k"], s["k_w"], s["k_b"]))
    return {"q": q, "k": s["k_cache"]}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("decode", "prefill"):
        return _exact_attention(s, case)
    if op == "read":
        return _exact_read(s, case)
    pos = s["pos"].long()
    turn = torch.complex(s["cos_sin"][pos, :32].double(), s["cos_sin"][pos, 32:].double())

    def rotated(x):
        """x [R, ..., 64] in 64 bits, its pairs turned as complex numbers."""
        pairs = x.unflatten(-1, (32, 2)) if case["interleave"] else x.unflatten(-1, (2, 32)).transpose(-1, -2)
        z = torch.view_as_complex(pairs.contiguous()) * turn.view(turn.shape[0], *[1] * (x.dim() - 2), 32)
        z = torch.view_as_real(z)
        return z.flatten(-2) if case["interleave"] else z.transpose(-1, -2).flatten(-2)

    kept = (s["slots"] >= 0).nonzero()[:, 0]
    to = s["slots"][kept].long()
    if op == "write":
        x = s["kv_a"].double()
        c = x[:, :LATENT]
        u = c / (torch.linalg.vector_norm(c, dim=1, keepdim=True) ** 2 / LATENT + EPS).sqrt() * s["w"].double()
        big = u.abs().amax(1)
        scale = torch.exp2(torch.ceil(torch.log2(big / E4M3_MAX)).clamp(-64, 64))
        scale = torch.where(big == 0, torch.ones_like(scale), scale)
        v = u / scale[:, None]
        # e4m3: 3 fraction bits, smallest step 2^-9, half to even
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        v = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        out = {"latent": s["latent"].double(), "rope": s["rope"].double(), "scale": s["scale"].double()}
        out["latent"][to], out["rope"][to], out["scale"][to] = v[kept], rotated(x[:, LATENT:])[kept], scale[kept]
        return out

    def normed(x, w, b):
        if w is not None:
            centre = x.mean(-1, keepdim=True) if case["norm"] == "layer" else torch.zeros_like(x[..., :1])
            x = (x - centre) / (((x - centre) ** 2).sum(-1, keepdim=True) / IDX_DIM + EPS) ** 0.5 * w.double()
        return x if b is None else x + b.double()

    def made(x, w, b):
        x = normed(x.double(), w, b)
        return torch.cat([rotated(x[..., :ROPE]), x[..., ROPE:]], -1)

    k = s["k_cache"].double()
    k[to] = made(s["k"], s["k_w"], s["k_b"])[kept]
    return {"q": made(s["q"], s["q_w"], None), "k": k}


def _exact_row(s, at):
    """Cache rows `at` (any shape) as the float64 values they stand for."""
    raw = s["cache"].reshape(-1, ROW)[at].contiguous()
    latent = raw[..., :LATENT].contiguous().view(torch.float8_e4m3fn).double() * s["scale"].reshape(-1)[at].double().unsqueeze(-1)
    return torch.cat([latent, raw[..., LATENT:].contiguous().view(torch.bfloat16).double()], -1)


def _exact_read(s, case):
    out = s["out"].double()
    if not case["page"]:
        kept = (s["slots"] >= 0).nonzero()[:, 0]
        out[kept] = _exact_row(s, s["slots"][kept].long())
        return out
    for b, n in enumerate(s["kv_len"].tolist()):
        j = torch.arange(n, device="cuda")
        out[b, :n] = _exact_row(s, s["table"][b, j // case["page"]].long() * case["page"] + j % case["page"])
    return out


def _exact_attention(s, case):
    n = s["q"].shape[0]
    out = torch.zeros(n, HEADS, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((n, HEADS), -math.inf, dtype=torch.float64, device="cuda")
    for i in range(0, n, 64):
        j = s["idx"][i:i + 64].long()
        have = j >= 0
        at = torch.where(have, j, 0)
        seq = torch.arange(i, i + at.shape[0], device="cuda")[:, None] if case["op"] == "decode" else torch.zeros_like(at[:, :1])
        if case["page"]:
            at = s["table"][seq, at // case["page"]].long().clamp(min=0) * case["page"] + at % case["page"]
        else:
            at = at + seq * case["N"]
        kv = _exact_row(s, at)
        x = torch.einsum("qhd,qkd->qhk", s["q"][i:i + 64].double(), kv) * SCALE
        x = torch.where(have[:, None, :], x, -math.inf)
        lse[i:i + 64] = torch.logsumexp(x, 2)
        p = torch.nan_to_num(torch.softmax(x, 2), nan=0.0)              # no key at all: zeros
        out[i:i + 64] = torch.einsum("qhk,qkd->qhd", p, kv[..., :LATENT])
    return {"out": out, "lse": lse}
