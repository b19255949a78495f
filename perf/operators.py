"""The paged key-value cache's operators as measured cases.

Four operators, each in its plain form (elementary torch, fp32) and, where
``own`` is set, as the library's calls:

 append  dsa_cache_append: new queries, keys and values rotated by their
         positions; the queries returned, the keys and values written into
         the pages that a block table names (bf16, or e4m3 with one e8m0
         scale per 32 features);
 pool    dsa_block_pool: the mean key of every block that the last step
         completed, written into the pooled cache the indexer scores;
 dense   dsa_paged_attention_forward: attention of every query token over
         all (or the last ``window``) slots of its sequence's pages;
 blocks  dsa_block_attention_forward: attention over listed blocks of slots
         and over the last ``window`` slots.

Sequence lengths follow from the case alone, so that work(case) can count
them; every value, block table and block list comes from the seed.
"""
import math

import torch

own = False

D = 128                     # the library's head dimension
MX = 32                     # features under one e8m0 scale
DEV = "cuda"


# ---- sizes ------------------------------------------------------------------

def _lengths(case):
    """Slots of each sequence: spread over [lo, hi] by the golden ratio; the
    first is the longest. `empty`: the last sequence holds none."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    got = [hi if i == 0 else lo + int((hi - lo) * math.modf(i * 0.6180339887498949)[0])
           for i in range(n)]
    if case.get("empty") and n > 1:
        got[-1] = 0
    return got


def _new(case):
    """New tokens of each sequence in an append: `T` in all, split evenly
    (the first sequences take the remainder)."""
    n, T = case["seqs"], case["T"]
    return [T // n + (1 if i < T % n else 0) for i in range(n)]


def _pages(case):
    return max(1, -(-case["hi"] // case["page"]))


def _rows(case):
    """(sequence, position) of every query row of an attention case: the last
    `per` tokens of every sequence (one for decoding)."""
    got = []
    for s, n in enumerate(_lengths(case)):
        got += [(s, n - case["per"] + j) if n >= case["per"] - j else (s, -1)
                for j in range(case["per"])]
    return got


def _ranges(case):
    """First new position and last position of every sequence of a pool case:
    the last `new` slots of each were appended since the last call."""
    return [(max(0, n - case["new"]), n - 1) for n in _lengths(case)]


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one decoding step of a 16-sequence batch: 64 query heads, 8 key
        # heads, the leading 64 features rotated in interleaved pairs
        dict(name="append decode step", op="append", seqs=16, lo=2048, hi=32768, T=16, H=64, Hkv=8,
             rope=64, split=False, fp8=False, heads_first=False, values=True, page=64, pad=0),
        # a prompt's chunk, both halves rotated, with a padded tail
        dict(name="append prompt chunk", op="append", seqs=3, lo=5000, hi=9000, T=8192, H=64, Hkv=8,
             rope=128, split=True, fp8=False, heads_first=True, values=True, page=64, pad=57),
        # the indexer's queries and keys of packed prompts, quantised into its
        # paged fp8 cache (one key head, no values); an odd token count
        dict(name="append index keys fp8", op="append", seqs=4, lo=3500, hi=6000, T=12345, H=64, Hkv=1,
             rope=64, split=False, fp8=True, heads_first=False, values=False, page=64, pad=0),
        # a decoding step of 64 sequences: a few of them complete a block
        dict(name="pool decode step", op="pool", seqs=64, lo=1024, hi=32768, new=1, Hkv=1, block=4,
             fp8=False, heads_first=False, page=64),
        # a long prompt's keys pooled 4:1 (the compressed indexer's ratio)
        dict(name="pool prompt 4:1", op="pool", seqs=2, lo=90001, hi=131072, new=131072, Hkv=1, block=4,
             fp8=False, heads_first=False, page=64),
        # blocks of 64 of every key head of an fp8 cache, ragged batch
        dict(name="pool prompt fp8", op="pool", seqs=7, lo=777, hi=32768, new=131072, Hkv=8, block=64,
             fp8=True, heads_first=True, page=128),
        # one user, a short context: latency
        dict(name="dense one sequence", op="dense", seqs=1, lo=1000, hi=1000, per=1, H=64, Hkv=8,
             fp8=False, heads_first=False, page=64, window=0, sinks=False, empty=False),
        # a decode batch of 16 over its whole caches, grouped heads
        dict(name="dense batch", op="dense", seqs=16, lo=2048, hi=32768, per=1, H=64, Hkv=8,
             fp8=False, heads_first=True, page=64, window=0, sinks=False, empty=False),
        # few long contexts, one key head under 128 query heads, with sinks
        dict(name="dense long one key head", op="dense", seqs=4, lo=65000, hi=131072, per=1, H=128, Hkv=1,
             fp8=False, heads_first=False, page=64, window=0, sinks=True, empty=False),
        # a large batch over an fp8 cache, an empty slot in the batch
        dict(name="dense batch fp8", op="dense", seqs=64, lo=1024, hi=32768, per=1, H=64, Hkv=4,
             fp8=True, heads_first=False, page=64, window=0, sinks=False, empty=True),
        # a decode batch, 32 blocks of 64 a key head and the last 64 slots
        dict(name="blocks decode", op="blocks", seqs=16, lo=4096, hi=32768, per=1, H=64, Hkv=8,
             fp8=False, heads_first=False, page=64, window=64, sinks=False, empty=False, block=64,
             n=32, each=True),
        # a prompt's chunk of 1024 queries, each with its own 16 blocks
        dict(name="blocks prompt chunk", op="blocks", seqs=2, lo=20001, hi=32768, per=512, H=64, Hkv=4,
             fp8=False, heads_first=True, page=64, window=64, sinks=False, empty=False, block=64,
             n=16, each=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "pool", "dense", "dense", "blocks", "blocks"])
    case = dict(op=op, page=rng.choice([16, 32, 64, 128, 256]), fp8=rng.random() < 0.4,
                heads_first=rng.random() < 0.5)
    if op == "append":
        T = _log(rng, 1, 9000)
        seqs = rng.randint(1, min(T, 64))
        per = -(-T // seqs)
        H, Hkv = rng.choice([(0, 1), (64, 1), (32, 8), (8, 8), (5, 1), (12, 3), (64, 8)])
        hi = per + _log(rng, 1, 4000)
        case.update(seqs=seqs, lo=rng.randint(per, hi), hi=hi, T=T, H=H, Hkv=Hkv,
                    rope=rng.choice([0, 32, 64, 96, 128]), split=rng.random() < 0.5,
                    values=rng.random() < 0.7, pad=rng.choice([0, 0, 1, 13]))
    elif op == "pool":
        seqs = _log(rng, 1, 64)
        Hkv = rng.choice([1, 1, 2, 8])
        hi = _log(rng, 2, max(2, 700000 // (seqs * Hkv)))
        case.update(seqs=seqs, lo=rng.randint(1, hi), hi=hi, new=rng.choice([1, 7, 131072]), Hkv=Hkv,
                    block=rng.choice([1, 2, 4, 16, 32, 64, 128]))
    else:
        Hkv = rng.choice([1, 1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 5, 8, 8, 12, 16, 32, 64, 128])
        if Hkv * G > 128:
            G = 128 // Hkv
        case.update(Hkv=Hkv, H=Hkv * G, sinks=rng.random() < 0.3, empty=rng.random() < 0.3)
        if op == "dense":
            seqs = _log(rng, 1, 64)
            per = rng.choice([1, 1, 1, 2, 4])
            hi = _log(rng, 1, max(1, min(131072, 4000000 // (seqs * Hkv * per))))
            case.update(seqs=seqs, lo=rng.randint(1, hi), hi=hi, per=per,
                        window=rng.choice([0, 0, 0, _log(rng, 1, hi)]))
        else:
            block = rng.choice([1, 4, 16, 32, 64, 128])
            n = _log(rng, 1, max(1, 2048 // block))
            each = Hkv > 1 and rng.random() < 0.6
            seqs = _log(rng, 1, 16)
            rows = n * block * Hkv * seqs                  # gathered for one query of each sequence
            per = _log(rng, 1, max(1, min(512, 4000000 // rows, 60000000 // (rows * G))))
            hi = per + _log(rng, 1, 32768 // max(1, seqs * Hkv // 16))
            case.update(seqs=seqs, lo=rng.randint(per, hi), hi=hi, per=per, block=block, n=n, each=each,
                        window=rng.choice([0, 1, block, 2 * block + 3]))
    return case


# ---- inputs -----------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _pool_of(case, g, pages, fp8):
    """A pool of random rows as the case lays it out, its scales (fp8), and
    its strides (page, slot, head) in elements."""
    Hkv, ps = case["Hkv"], case["page"]
    shape = (pages, Hkv, ps, D) if case["heads_first"] else (pages, ps, Hkv, D)
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if not fp8:
        return x, None
    # codes of values around +-100 under scales of 2^-8 .. 2^-6
    data = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    scale = torch.randint(119, 122, shape[:-1] + (D // MX,), generator=g, device=DEV, dtype=torch.uint8)
    return data, scale


def _strides(case):
    Hkv, ps = case["Hkv"], case["page"]
    page = Hkv * ps * D
    return (page, D, ps * D) if case["heads_first"] else (page, Hkv * D, D)


def _table(case, g):
    """Block tables over scattered pages; a few pages belong to nobody."""
    n = case["seqs"] * _pages(case)
    total = n + 3
    perm = torch.randperm(total, generator=g, device=DEV)[:n]
    return perm.to(torch.int32).view(case["seqs"], _pages(case)).contiguous(), total


def _cache_desc(m, case, s):
    page, slot, head = _strides(case)
    return m.make_paged_cache(case["page"], _pages(case), s["num_pages"], s["table"],
                              num_seqs=case["seqs"], H_kv=case["Hkv"],
                              dtype=m.DSA_KV_FP8_E4M3_E8M0_B32 if case["fp8"] else m.DSA_KV_BF16,
                              page_stride=page, slot_stride=slot, head_stride=head)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    s["table"], s["num_pages"] = _table(case, g)
    fp8 = case["fp8"]
    if case["op"] == "append":
        T, H, Hkv, pad = case["T"], case["H"], case["Hkv"], case["pad"]
        lens, new = _lengths(case), _new(case)
        pos, seq = [], []
        for i, (n, c) in enumerate(zip(lens, new)):
            pos += range(n - c, n)
            seq += [i] * c
        pos = torch.tensor(pos + [-1] * pad, dtype=torch.int32)
        s["positions"] = pos.to(DEV)
        s["seq"] = torch.tensor(seq + [0] * pad, dtype=torch.int32).to(DEV)
        N = T + pad
        s["live"] = torch.arange(T, device=DEV)
        # the projections' one output row a token: queries, keys, values
        width = (H + Hkv + (Hkv if case["values"] else 0)) * D
        s["qkv"] = _randn(g, N, width).to(torch.bfloat16)
        angle = pos.clamp(min=0).double()[:, None] * \
            10000.0 ** (-torch.arange(0, case["rope"], 2, dtype=torch.float64) / max(1, case["rope"]))
        s["cos"], s["sin"] = (f(angle).float().contiguous().to(DEV) for f in (torch.cos, torch.sin))
        s["k"], s["k_scale"] = _pool_of(case, g, s["num_pages"], fp8)
        s["v"], s["v_scale"] = _pool_of(case, g, s["num_pages"], fp8) if case["values"] else (None, None)
        s["q_out"] = torch.zeros((N, H, D), device=DEV, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16)
        s["q_scale"] = torch.zeros((N, H, D // MX), device=DEV, dtype=torch.uint8) if fp8 else None
        if own:
            import sparse_attention_lightning_tcgen05_b200 as m
            s["desc"] = m.make_append_desc(
                _cache_desc(m, case, s), N, H, case["rope"],
                rope_style=m.DSA_ROPE_HALVES if case["split"] else m.DSA_ROPE_INTERLEAVED,
                q_dtype=m.DSA_KV_FP8_E4M3_E8M0_B32 if fp8 else m.DSA_KV_BF16,
                q_stride=width, k_stride=width, v_stride=width)
    elif case["op"] == "pool":
        s["k"], s["k_scale"] = _pool_of(case, g, s["num_pages"], fp8)
        first, last = zip(*_ranges(case))
        s["start"] = torch.tensor(first, dtype=torch.int32, device=DEV)
        s["positions"] = torch.tensor(last, dtype=torch.int32, device=DEV)
        S_pool = max(1, case["hi"] // case["block"])
        shape = (case["seqs"], case["Hkv"], S_pool, D)
        s["pooled"] = torch.zeros(shape, device=DEV, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16)
        s["pooled_scale"] = torch.zeros(shape[:-1] + (D // MX,), device=DEV, dtype=torch.uint8) if fp8 else None
        s["last"] = torch.zeros((case["seqs"], case["Hkv"]), device=DEV, dtype=torch.int32)
        if own:
            import sparse_attention_lightning_tcgen05_b200 as m
            s["desc"] = m.make_block_pool_desc(_cache_desc(m, case, s), case["block"], S_pool)
    else:
        H = case["H"]
        rows = _rows(case)
        T = len(rows)
        s["seq"] = torch.tensor([r[0] for r in rows], dtype=torch.int32).to(DEV)
        s["positions"] = torch.tensor([r[1] for r in rows], dtype=torch.int32).to(DEV)
        s["q"] = _randn(g, T, H, D).to(torch.bfloat16)
        s["k"], s["k_scale"] = _pool_of(case, g, s["num_pages"], fp8)
        s["v"], s["v_scale"] = _pool_of(case, g, s["num_pages"], fp8)
        s["sinks"] = _randn(g, H) if case["sinks"] else None
        s["scale"] = D ** -0.5
        s["out"] = torch.zeros((T, H, D), device=DEV, dtype=torch.bfloat16)
        s["lse"] = torch.zeros((T, H), device=DEV, dtype=torch.float32)
        if case["op"] == "blocks":
            # distinct visible blocks of every row, in any order; -1 at the
            # end where the row sees fewer (as an indexer's top-k gives them)
            Hb = case["Hkv"] if case["each"] else 1
            total = max(case["n"], -(-case["hi"] // case["block"]))
            seen = torch.div(s["positions"] + case["block"], case["block"], rounding_mode="floor")
            luck = torch.rand((T, Hb, total), generator=g, device=DEV)
            luck = luck.masked_fill(torch.arange(total, device=DEV) >= seen[:, None, None], -1.0)
            luck, at = luck.topk(case["n"], dim=-1)
            s["blocks"] = torch.where(luck >= 0, at, -1).to(torch.int32).contiguous()
        if own:
            import sparse_attention_lightning_tcgen05_b200 as m
            more = {}
            if case["op"] == "blocks":
                more = dict(block_size=case["block"], num_blocks=case["n"],
                            block_heads=case["Hkv"] if case["each"] else 1)
            s["desc"] = m.make_paged_attention_desc(_cache_desc(m, case, s), T, H, s["scale"],
                                                    window=case["window"], **more)
            s["bytes"] = m.dsa_paged_attention_workspace_size(s["desc"])
            s["workspace"] = torch.zeros(s["bytes"], dtype=torch.uint8, device=DEV)
    return s


# ---- the plain forms --------------------------------------------------------

def _rotate(x, cos, sin, split):
    """x [N, heads, D] fp32 with its leading 2 * cos.shape[1] features turned."""
    half = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    if split:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _quantize(x):
    """e4m3 values and e8m0 bytes of fp32 rows: per 32 features the least
    power of two that brings the largest magnitude to 448 or below."""
    b = x.unflatten(-1, (-1, MX))
    top = b.abs().amax(dim=-1).clamp(min=448.0 * 2.0 ** -127)
    m, e = torch.frexp(top)                           # top = m 2^e, 448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)
    data = torch.ldexp(b, -e[..., None]).flatten(-2).to(torch.float8_e4m3fn)
    return data, (e + 127).to(torch.uint8)


def _dequantize(data, scale):
    x = data.float().unflatten(-1, (-1, MX))
    return torch.ldexp(x, scale.to(torch.int32)[..., None] - 127).flatten(-2)


def _by_slot(pool, case):
    """A view [page, slot, head, feature]."""
    return pool.transpose(1, 2) if case["heads_first"] else pool


def _float(data, scale):
    return data.float() if scale is None else _dequantize(data, scale)


def _append_plain(s):
    case = s["case"]
    H, Hkv, ps = case["H"], case["Hkv"], case["page"]
    x = s["qkv"].float().unflatten(-1, (-1, D))
    q = _rotate(x[:, :H], s["cos"], s["sin"], case["split"])
    k = _rotate(x[:, H:H + Hkv], s["cos"], s["sin"], case["split"])
    v = x[:, H + Hkv:]
    pos = s["positions"].long()
    live = s["live"]                                  # padded tokens write nothing
    at, seq = pos[live], s["seq"].long()[live]
    page = s["table"].long()[seq, at // ps]
    if case["fp8"]:
        data, scale = _quantize(q[live])
        s["q_out"].view(torch.uint8)[live] = data.view(torch.uint8)
        s["q_scale"][live] = scale
    else:
        s["q_out"][live] = q[live].to(torch.bfloat16)
    _write(s["k"], s["k_scale"], case, page, at % ps, k[live])
    if case["values"]:
        _write(s["v"], s["v_scale"], case, page, at % ps, v[live])


def _write(pool, scale_pool, case, page, slot, rows):
    if scale_pool is None:
        _by_slot(pool, case)[page, slot] = rows.to(torch.bfloat16)
    else:
        data, scale = _quantize(rows)
        _by_slot(pool.view(torch.uint8), case)[page, slot] = data.view(torch.uint8)
        _by_slot(scale_pool, case)[page, slot] = scale


def _pool_plain(s):
    case = s["case"]
    r, ps = case["block"], case["page"]
    S_pool = s["pooled"].shape[2]
    b = torch.arange(S_pool, device=DEV)
    done = (s["positions"].long() + 1) // r           # complete blocks a sequence
    fresh = (b[None] < done[:, None]) & (b[None] >= (s["start"].long() // r)[:, None])
    seq, blk = fresh.nonzero(as_tuple=True)
    slot = blk[:, None] * r + torch.arange(r, device=DEV)
    page = s["table"].long()[seq[:, None], slot // ps]
    data = _by_slot(s["k"].view(torch.uint8) if case["fp8"] else s["k"], case)[page, slot % ps]
    if case["fp8"]:
        scale = _by_slot(s["k_scale"], case)[page, slot % ps]
        rows = _dequantize(data.view(torch.float8_e4m3fn), scale)
    else:
        rows = data.float()
    mean = rows.sum(dim=1) / r                        # [blocks, heads, D]
    if case["fp8"]:
        data, scale = _quantize(mean)
        s["pooled"].view(torch.uint8)[seq, :, blk] = data.view(torch.uint8)
        s["pooled_scale"][seq, :, blk] = scale
    else:
        s["pooled"][seq, :, blk] = mean.to(torch.bfloat16)
    s["last"][:] = (done - 1)[:, None]


def _attend(q, k, v, keep, sinks, scale):
    """q [T, Hkv, G, D], k and v [T, slots, Hkv, D], keep [T, Hkv or 1, slots]."""
    x = torch.einsum("tgid,tsgd->tgis", q, k) * scale
    x = x.masked_fill(~keep[:, :, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - base)
    total = p.sum(dim=-1, keepdim=True)
    lse = (base + torch.log(total)).flatten(1)
    if sinks is not None:
        total = total + torch.where(total > 0, torch.exp(sinks.view(1, q.shape[1], -1, 1) - base), 0.0)
    out = torch.einsum("tgis,tsgd->tgid", p, v)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.flatten(1, 2), lse


def _attention_plain(s):
    case = s["case"]
    Hkv, ps, window = case["Hkv"], case["page"], case["window"]
    q = s["q"].float().unflatten(1, (Hkv, -1))
    pos, seq = s["positions"].long(), s["seq"].long()
    if case["op"] == "dense":
        slot = torch.arange(_pages(case) * ps, device=DEV)[None, None]
        keep = slot <= pos[:, None, None]
        if window:
            keep = keep & (slot > pos[:, None, None] - window)
        page = s["table"].long()[seq]                 # [T, pages]
        k, v = (_float(_by_slot(_bytes(s[n]), case)[page].flatten(1, 2).view(s[n].dtype),
                       None if s[n + "_scale"] is None else
                       _by_slot(s[n + "_scale"], case)[page].flatten(1, 2)) for n in ("k", "v"))
    else:
        r = case["block"]
        inside = torch.arange(r, device=DEV)
        listed_slots = (s["blocks"].long()[..., None] * r + inside).flatten(2)
        keep = (s["blocks"] >= 0).repeat_interleave(r, dim=-1)
        keep = keep & (listed_slots <= pos[:, None, None] - window)
        recent = (pos[:, None] - torch.arange(window, device=DEV))[:, None].expand(-1, keep.shape[1], -1)
        slot = torch.cat([listed_slots, recent], dim=-1)           # [T, Hb, slots]
        keep = torch.cat([keep, recent >= 0], dim=-1)
        slot = torch.where(keep, slot, 0).expand(-1, Hkv, -1).transpose(1, 2)
        page = s["table"].long()[seq[:, None, None], slot // ps]
        head = torch.arange(Hkv, device=DEV)
        k, v = (_float(_by_slot(_bytes(s[n]), case)[page, slot % ps, head].view(s[n].dtype),
                       None if s[n + "_scale"] is None else
                       _by_slot(s[n + "_scale"], case)[page, slot % ps, head]) for n in ("k", "v"))
    out, lse = _attend(q, k, v, keep, s["sinks"], s["scale"])
    s["out"].copy_(out.to(torch.bfloat16))
    s["lse"].copy_(lse)


def _bytes(pool):
    return pool.view(torch.uint8) if pool.element_size() == 1 else pool


# ---- one pass ---------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if op == "append":
        if own:
            _append_own(s)
        else:
            _append_plain(s)
        return {"q": s["q_out"], "q_scale": _as_scale(s["q_scale"]), "k": s["k"],
                "k_scale": _as_scale(s["k_scale"]), "v": s["v"], "v_scale": _as_scale(s["v_scale"])}
    if op == "pool":
        if own:
            _pool_own(s)
        else:
            _pool_plain(s)
        return {"pooled": s["pooled"], "scale": _as_scale(s["pooled_scale"]), "last": s["last"]}
    if own:
        _attention_own(s)
    else:
        _attention_plain(s)
    return {"out": s["out"], "lse": s["lse"]}


def _as_scale(x):
    """The powers of two that the scale bytes stand for."""
    return None if x is None else x.view(torch.float8_e8m0fnu)


def _append_own(s):
    import sparse_attention_lightning_tcgen05_b200 as m
    case, x = s["case"], s["qkv"]
    H, Hkv = case["H"], case["Hkv"]
    m.dsa_cache_append(s["desc"], x if H else None, x[:, H * D:],
                       x[:, (H + Hkv) * D:] if case["values"] else None, s["cos"], s["sin"],
                       s["positions"], s["seq"], s["q_out"] if H else None, s["q_scale"] if H else None,
                       s["k"], s["k_scale"], s["v"], s["v_scale"], m.current_stream_handle())


def _pool_own(s):
    import sparse_attention_lightning_tcgen05_b200 as m
    m.dsa_block_pool(s["desc"], s["k"], s["k_scale"], s["start"], s["positions"], s["pooled"],
                     s["pooled_scale"], s["last"], m.current_stream_handle())


def _attention_own(s):
    import sparse_attention_lightning_tcgen05_b200 as m
    if s["case"]["op"] == "dense":
        m.dsa_paged_attention_forward(s["desc"], s["q"], s["k"], s["k_scale"], s["v"], s["v_scale"],
                                      s["sinks"], s["positions"], s["seq"], s["out"], s["lse"],
                                      s["workspace"], s["bytes"], m.current_stream_handle())
    else:
        m.dsa_block_attention_forward(s["desc"], s["q"], s["k"], s["k_scale"], s["v"], s["v_scale"],
                                      s["sinks"], s["positions"], s["seq"], s["blocks"], s["out"],
                                      s["lse"], s["workspace"], s["bytes"], m.current_stream_handle())


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    row = D + D // MX if case["fp8"] else 2 * D       # bytes of one cached head row
    if case["op"] == "append":
        T, H, Hkv = case["T"], case["H"], case["Hkv"]
        n = Hkv * (2 if case["values"] else 1)
        return {"bytes": T * ((H + n) * (2 * D + row) + 4 * case["rope"] + 8), "flops": T * (H + Hkv) * 3 * case["rope"]}
    if case["op"] == "pool":
        r = case["block"]
        blocks = sum(max(0, (last + 1) // r - first // r) for first, last in _ranges(case)) * case["Hkv"]
        return {"bytes": blocks * (r + 1) * row + case["seqs"] * (12 + 4 * case["Hkv"]), "flops": blocks * (r + 1) * D}
    H, Hkv, window = case["H"], case["Hkv"], case["window"]
    rows = _rows(case)
    if case["op"] == "dense":
        pairs = sum(min(p + 1, window or p + 1) for _, p in rows if p >= 0)
        slots = {}
        for q, p in rows:                             # the slots that a sequence's rows see
            if p >= 0:
                lo, hi = slots.get(q, (p + 1, p))
                slots[q] = (min(lo, max(0, p + 1 - window) if window else 0), max(hi, p))
        slots = sum(hi + 1 - lo for lo, hi in slots.values()) * Hkv
        extra = 0
    else:
        r, n = case["block"], case["n"]
        pairs, distinct = 0, {}
        for q, p in rows:
            if p >= 0:
                recent = min(window, p + 1)
                pairs += recent + min(n * r, p + 1 - recent)
                distinct[q] = min(p + 1, distinct.get(q, 0) + recent + n * r)
        slots = sum(distinct.values()) * Hkv
        extra = len(rows) * n * 4 * (Hkv if case["each"] else 1)
    return {"bytes": slots * 2 * row + len(rows) * H * (4 * D + 4) + extra, "flops": 4 * D * pairs * H}


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _append_exact(s)
    if case["op"] == "pool":
        return _pool_exact(s)
    return _attention_exact(s)


def _value64(pool, scale):
    """What every element of a pool stands for, in 64 bits."""
    x = pool.double()
    if scale is None:
        return x
    return x * torch.exp2(scale.double() - 127).repeat_interleave(MX, dim=-1)


def _turn64(x, angle_cos, angle_sin, case):
    """The rotation as a product of complex numbers."""
    x, half = x.double().clone(), case["rope"] // 2
    if half:
        w = torch.complex(angle_cos.double(), angle_sin.double())[:, None]
        re = slice(0, half) if case["split"] else slice(0, 2 * half, 2)
        im = slice(half, 2 * half) if case["split"] else slice(1, 2 * half, 2)
        z = torch.complex(x[..., re], x[..., im]) * w
        x[..., re], x[..., im] = z.real, z.imag
    return x


def _blocks64(x):
    """Rows over the powers of two that keep each 32 features within 448
    (unrounded), and those powers."""
    y = x.reshape(*x.shape[:-1], -1, MX)
    top = y.abs().max(dim=-1).values.clamp(min=448.0 * 2.0 ** -127)
    e = torch.ceil(torch.log2(top / 448.0))
    e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e).clamp(min=-127)
    return (y / torch.exp2(e)[..., None]).reshape(x.shape), torch.exp2(e)


def _append_exact(s):
    case = s["case"]
    H, Hkv, ps, fp8 = case["H"], case["Hkv"], case["page"], case["fp8"]
    got = {"q": s["q_out"].double(), "q_scale": None, "k": s["k"].double(), "k_scale": None, "v": None,
           "v_scale": None}
    x = s["qkv"].reshape(s["qkv"].shape[0], -1, D)
    live = [i for i, p in enumerate(s["positions"].tolist()) if p >= 0]
    q = _turn64(x[:, :H], s["cos"], s["sin"], case)[live]
    k = _turn64(x[:, H:H + Hkv], s["cos"], s["sin"], case)[live]
    v = x[:, H + Hkv:].double()[live]
    pos, seq = s["positions"][live].long(), s["seq"][live].long()
    page = s["table"][seq, pos // ps].long()

    def put(pool, scale_pool, rows):
        pool = pool.double()
        if not fp8:
            (pool.permute(0, 2, 1, 3) if case["heads_first"] else pool)[page, pos % ps] = rows
            return pool, None
        scales = torch.exp2(scale_pool.double() - 127)
        data, scale = _blocks64(rows)
        (pool.permute(0, 2, 1, 3) if case["heads_first"] else pool)[page, pos % ps] = data
        (scales.permute(0, 2, 1, 3) if case["heads_first"] else scales)[page, pos % ps] = scale
        return pool, scales

    if fp8:
        data, scale = _blocks64(q)
        got["q"][live] = data
        got["q_scale"] = torch.exp2(s["q_scale"].double() - 127)
        got["q_scale"][live] = scale
    else:
        got["q"][live] = q
    got["k"], got["k_scale"] = put(s["k"], s["k_scale"], k)
    if case["values"]:
        got["v"], got["v_scale"] = put(s["v"], s["v_scale"], v)
    return got


def _pool_exact(s):
    case = s["case"]
    r, ps = case["block"], case["page"]
    pooled = s["pooled"].double()
    scales = torch.exp2(s["pooled_scale"].double() - 127) if case["fp8"] else None
    for i, (first, last) in enumerate(_ranges(case)):
        lo, hi = first // r, (last + 1) // r
        if hi <= lo:
            continue
        pages = s["table"][i, lo * r // ps:(hi * r - 1) // ps + 1].long()
        keys = _value64(s["k"][pages], None if s["k_scale"] is None else s["k_scale"][pages])
        keys = (keys.permute(0, 2, 1, 3) if case["heads_first"] else keys).flatten(0, 1)
        off = lo * r - lo * r // ps * ps
        mean = keys[off:off + (hi - lo) * r].view(hi - lo, r, -1, D).mean(dim=1).transpose(0, 1)
        if case["fp8"]:
            pooled[i, :, lo:hi], scales[i, :, lo:hi] = _blocks64(mean)
        else:
            pooled[i, :, lo:hi] = mean
    return {"pooled": pooled, "scale": scales, "last": None}


def _attention_exact(s):
    case = s["case"]
    Hkv, ps, r, w = case["Hkv"], case["page"], case.get("block", 0), case["window"]
    G = case["H"] // Hkv
    T = s["q"].shape[0]
    out = torch.zeros((T, case["H"], D), dtype=torch.float64, device=DEV)
    lse = torch.full((T, case["H"]), -math.inf, dtype=torch.float64, device=DEV)
    lists = s["blocks"].tolist() if case["op"] == "blocks" else None
    cached = (None, None)
    for t, (i, p) in enumerate(_rows(case)):
        if p < 0:
            continue
        if cached[0] != i:                             # the sequence's keys and values, in order
            pages = s["table"][i].long()
            kv = []
            for n in ("k", "v"):
                y = _value64(s[n][pages], None if s[n + "_scale"] is None else s[n + "_scale"][pages])
                kv.append((y.permute(0, 2, 1, 3) if case["heads_first"] else y).flatten(0, 1).transpose(0, 1).contiguous())
            cached = (i, kv)
        k, v = cached[1]                               # [Hkv, slots, D]
        for g in range(Hkv if lists is not None and case["each"] else 1):
            heads = slice(g, g + 1) if lists is not None and case["each"] else slice(0, Hkv)
            if lists is None:
                at = slice(max(0, p + 1 - w) if w else 0, p + 1)
                kk, vv = k[heads, at], v[heads, at]
            else:
                slots = [b * r + j for b in lists[t][g] if b >= 0 for j in range(r) if b * r + j <= p - w]
                slots += range(max(0, p + 1 - w), p + 1)
                if not slots:
                    continue
                at = torch.tensor(slots, device=DEV)
                kk, vv = k[heads][:, at], v[heads][:, at]
            qq = s["q"][t].view(Hkv, G, D)[heads].double()
            x = torch.matmul(qq, kk.transpose(1, 2)) * s["scale"]
            e = torch.logsumexp(x, dim=-1)
            total = e
            if s["sinks"] is not None:
                total = torch.logaddexp(e, s["sinks"].double().view(Hkv, G)[heads])
            o = torch.matmul(torch.exp(x - total[..., None]), vv)
            out.view(T, Hkv, G, D)[t, heads] = o
            lse.view(T, Hkv, G)[t, heads] = e
    return {"out": out, "lse": lse}
