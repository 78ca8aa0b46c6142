"""The cases on which the paged 8-bit latent cache's operators are measured.

Five operators, as a serving program chains them:

  fork     rows take other rows' pages, keep some, give some back and get fresh ones for the tokens to
           come (mla_cache8_pages_update); pages that are shared and about to be written are copied
           (mla_cache8_pages_copy)
  compact  the pages in use move to the front of the pool (mla_cache8_pages_compact, mla_cache8_pages_copy)
  append   new tokens' keys rotated, quantised to e4m3 and written to their rows' pages
           (mla_cache8_append with tables)
  read     cached positions read back, in order over pages and context shards (mla_cache8_read with tables)
  decode   single-token attention over the pages; rows that share a long prefix attend to it together
           (mla_cache8_decode with tables, and with groups)

A pool is [P pages, page tokens, 512 latent + 64 rotary] e4m3 with one fp32 scale for each block of
tokens. tables [B, M] holds the page of each `page` tokens of a row (-1: none), refs [P] how many rows
hold a page (0: free). Under context parallelism position p of a row lives on shard
(p / interleave) mod cp, and each shard has a pool and tables of its own. Where `own` is false each
operator runs in its plain form: elementary torch operations in 32 bits (angles in 64), rounded once at
the end.
"""
import math

import torch

own = False

DEV = "cuda"
DV, DK = 512, 576    # latent dims (the values); with the rotary ones
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_EXP = -60        # smallest exponent of a block's scale
SCALE = 192 ** -0.5  # softmax scale of 128 + 64 dims a head
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # beam search over one sequence: 4 beams, each a token further, from the beams that were kept
        {"name": "fork_beams", "op": "fork", "b": 4, "m": 64, "p": 256, "page": 64, "block": 1, "held": 2000,
         "cp": 1, "shard": 0, "interleave": 1, "kind": "beams"},
        # a serving step: of 256 rows some end, some are cut back to the tokens that were accepted, new ones begin
        # behind a prompt that another row holds, most only go on
        {"name": "fork_serving", "op": "fork", "b": 256, "m": 128, "p": 16384, "page": 64, "block": 64, "held": 5000,
         "cp": 1, "shard": 0, "interleave": 1, "kind": "serving"},
        # a small pool, half of it in use here and there
        {"name": "compact_small", "op": "compact", "b": 13, "m": 40, "p": 384, "page": 64, "block": 1, "fill": 0.5},
        # a large pool after most of its sequences have ended
        {"name": "compact_pool", "op": "compact", "b": 64, "m": 256, "p": 16384, "page": 64, "block": 64, "fill": 0.33},
        # a decode step's tokens, one of each row
        {"name": "append_step", "op": "append", "b": 128, "n": 128, "cp": 1, "interleave": 1, "block": 1, "page": 64,
         "m": 32, "ragged": False, "dtype": "bf16"},
        # prompts of mixed lengths, 16385 tokens in all, blocks of 64
        {"name": "append_prompt", "op": "append", "b": 5, "n": 16385, "cp": 1, "interleave": 1, "block": 64,
         "page": 128, "m": 128, "ragged": True, "dtype": "bf16"},
        # a chunk of two sequences' context for the next prompt chunk
        {"name": "read_chunk", "op": "read", "b": 2, "n": 2047, "cp": 1, "interleave": 1, "block": 1, "page": 64,
         "m": 32, "ragged": True, "dtype": "bf16"},
        # long contexts gathered from four shards' pages into position order
        {"name": "read_long", "op": "read", "b": 8, "n": 262144, "cp": 4, "interleave": 16, "block": 64, "page": 64,
         "m": 256, "ragged": True, "dtype": "bf16"},
        # one sequence with a short context and 16 heads: latency
        {"name": "decode_token", "op": "decode", "b": 1, "h": 16, "cp": 1, "interleave": 1, "block": 1, "page": 64,
         "groups": 0, "prefix": 0, "own": 300},
        # a serving batch with nothing in common: 64 sequences of mixed lengths, 128 heads, blocks of 64
        {"name": "decode_serving", "op": "decode", "b": 64, "h": 128, "cp": 1, "interleave": 1, "block": 64,
         "page": 64, "groups": 0, "prefix": 0, "own": 16384},
        # 64 sequences behind two long prompts, 16 heads (a shard of a model's heads)
        {"name": "decode_prefix", "op": "decode", "b": 64, "h": 16, "cp": 1, "interleave": 1, "block": 64,
         "page": 64, "groups": 2, "prefix": 16384, "own": 1024},
        # 12 samples of one question over two shards, 40 heads, a prompt that ends inside a page
        {"name": "decode_samples", "op": "decode", "b": 12, "h": 40, "cp": 2, "interleave": 16, "block": 1,
         "page": 128, "groups": 1, "prefix": 6001, "own": 700},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fork", "compact", "append", "read", "decode", "decode"])
    page = rng.choice([32, 64, 64, 128, 256])
    block = rng.choice([1, 16, 64] if page >= 64 else [1, 16])
    cp = rng.choice([1, 1, 2, 4])
    interleave = rng.choice([1, 16, 64]) if cp > 1 else 1
    if op == "fork":
        b, m = _log(rng, 1, 256), _log(rng, 2, 128)
        while b * m > 20000:
            m = max(2, m // 2)
        p = min(16384 * 64 // page, b * m + _log(rng, 1, 512))
        return {"op": op, "b": b, "m": m, "p": p, "page": page, "block": block, "held": _log(rng, 1, m * page),
                "cp": cp, "shard": rng.randrange(cp), "interleave": interleave,
                "kind": rng.choice(["beams", "serving"])}
    if op == "compact":
        p = _log(rng, 2, 16384 * 64 // page)
        b = _log(rng, 1, 128)
        return {"op": op, "b": b, "m": max(1, min(512, -(-p // b))), "p": p, "page": page, "block": block,
                "fill": rng.choice([0.1, 0.33, 0.5, 0.7, 0.95])}
    if op in ("append", "read"):
        b = _log(rng, 1, 128)
        n = _log(rng, b, max(b + 1, 16385 if op == "append" else 200000))
        most = 2 * (n // b) + 64  # tokens of the longest row
        m = (most // cp + 2 * interleave + 64) // page + 2
        return {"op": op, "b": b, "n": n, "cp": cp, "interleave": interleave, "block": block, "page": page, "m": m,
                "ragged": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "bf16", "fp16"] if op == "append" else ["bf16", "bf16", "fp16", "fp32"])}
    h = rng.choice([8, 16, 16, 24, 32, 40, 64, 128])
    b = _log(rng, 1, 64)
    room = 64 * 128 * 16384 // (2 * b * max(h, 64))  # positions of a row
    groups = rng.choice([0, 1, max(1, b // 8), max(1, b // 3)])
    prefix = _log(rng, 1, max(2, min(room // 2, 32768))) if groups else 0
    return {"op": op, "b": b, "h": h, "cp": cp, "interleave": interleave, "block": block, "page": page,
            "groups": groups, "prefix": prefix, "own": _log(rng, 1, max(2, min(room // 2, 65536)))}


# ---- shared arithmetic of the cases ------------------------------------------


def _counts(case):
    """New (or read) tokens of each row on the host: even, or uneven when ragged."""
    b, n = case["b"], case["n"]
    if not case["ragged"]:
        return [n // b + (1 if i < n % b else 0) for i in range(b)]
    w = [1.0 + (i * 7 % 5) / 4 for i in range(b)]
    room = max(0, min(n, 2 * (n // b) if b > 1 else n))
    c = [min(room, int(n * x / sum(w))) for x in w]
    i = 0
    while sum(c) < n:  # the rest, to the first rows that still have room
        add = min(n - sum(c), max(0, room - c[i % b]) if i < b else n)
        c[i % b] += add
        i += 1
    return c


def _owner(pos, cp, interleave):
    """(shard, local index) of a position."""
    return (pos // interleave) % cp, pos // (interleave * cp) * interleave + pos % interleave


def _held(n, cp, shard, interleave):
    """How many of the first n positions a shard has."""
    whole, rest = n // (cp * interleave), n % (cp * interleave)
    return whole * interleave + (rest - shard * interleave).clamp(0, interleave)


def _group_counts(case):
    """Rows of each group: uneven, at least one each."""
    b, g = case["b"], max(1, case["groups"])
    c = [b // g + (1 if i < b % g else 0) for i in range(g)]
    if g > 1 and c[0] > 1:
        c[0], c[-1] = c[0] - 1, c[-1] + 1
    return c


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s (at least 2^-60)."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, k, MIN_EXP))


def _pool(g, p, page, block):
    """A filled pool: normalised latents with some louder tokens, rotary keys of about twice their size."""
    kv = torch.empty((p, page, DK), dtype=E4M3, device=DEV)
    scales = torch.empty((p, page // block), dtype=torch.float32, device=DEV)
    for i in range(0, p, 1024):
        n = min(1024, p - i)
        x = torch.randn((n, page, DK), generator=g, device=DEV)
        x[..., DV:] *= 2
        x *= torch.exp(0.3 * torch.randn((n, page, 1), generator=g, device=DEV))
        xb = x.bfloat16().float().unflatten(1, (page // block, block))
        s = _scale_of(xb.abs().amax((-1, -2)))
        kv[i:i + n], scales[i:i + n] = (xb / s[..., None, None]).flatten(1, 2).to(E4M3), s
    return kv, scales


def _uniform(g, n, lo, hi):
    """n whole numbers in [lo, hi]."""
    u = torch.rand((n,), generator=g, device=DEV, dtype=torch.float64)
    return (lo + (u * (hi - lo + 1)).long()).clamp(max=hi)


def _prepare_fork(case, s, g):
    b, m, p, page = case["b"], case["m"], case["p"], case["page"]
    spread = (case["cp"], case["shard"], case["interleave"])
    rows = torch.arange(b, device=DEV)
    # what rows hold before: beams about the same number of tokens, serving rows very different ones
    if case["kind"] == "beams":
        held = torch.full((b,), case["held"] * case["cp"], dtype=torch.long, device=DEV)
    else:
        held = _uniform(g, b, 0, 2 * case["held"] * case["cp"])
    local = _held(held, *spread).clamp(max=m * page)
    n = -(-local // page)
    over = (n.cumsum(0) - p).clamp(min=0)  # (as many as the pool has)
    n = (n - over).clamp(min=0)
    held = torch.where(over > 0, n * page * case["cp"], held)
    slot = torch.arange(m, device=DEV)[None]
    order = torch.randperm(p, generator=g, device=DEV)
    tables = torch.where(slot < n[:, None], order[((n.cumsum(0) - n)[:, None] + slot).clamp(max=p - 1)], -1)
    if case["kind"] == "beams":
        # groups of 4 beams that have the first three quarters in common; each goes on from one of its group's best two
        lead = rows // 4 * 4
        common = (slot < (n[lead] * 3 // 4)[:, None]) & (slot < n[:, None])
        tables = torch.where(common, tables[lead], tables)
        parents = torch.minimum(lead + 2 * _uniform(g, b, 0, 1), torch.tensor(b - 1, device=DEV))
        parents = torch.where(rows % 2 == 0, rows, parents)
        keeps, wants = held[parents], held[parents] + 1
    else:
        # ends, begins behind another row's prompt, cut back to what was accepted of 4 tokens, goes on by up to 4
        what = torch.rand((b,), generator=g, device=DEV)
        other = _uniform(g, b, 0, b - 1)
        parents = torch.where(what < 0.06, -1, torch.where(what < 0.12, other, rows))
        keeps = torch.where(what < 0.12, held[other] // 2, torch.where(what < 0.6, held, (held - 3).clamp(min=0)))
        wants = torch.where(what < 0.06, 0, keeps + 1 + _uniform(g, b, 0, 3))
    s["tables"] = tables.int()
    s["refs"] = torch.zeros((p,), dtype=torch.int32, device=DEV)
    used = s["tables"][s["tables"] >= 0].long()
    s["refs"].scatter_add_(0, used, torch.ones_like(used, dtype=torch.int32))
    s["parents"], s["keeps"], s["wants"] = parents.int(), keeps.int(), wants.int()
    s["cache"], s["scales"] = _pool(g, p, page, case["block"])
    # the tables that the next step uses (a program goes from one pair to the other and back)
    s["next"] = (torch.empty_like(s["tables"]), torch.empty_like(s["refs"]))
    s["copies"] = torch.empty((b, 2), dtype=torch.int32, device=DEV)
    s["missing"] = torch.empty((1,), dtype=torch.int32, device=DEV)


def _prepare_compact(case, s, g):
    b, m, p = case["b"], case["m"], case["p"]
    live = max(1, min(int(p * case["fill"]), b * m))
    # rows of uneven lengths, `live` pages in all
    u = torch.rand((b,), generator=g, device=DEV, dtype=torch.float64) + 0.2
    n = (u / u.sum() * live).long().clamp(max=m)
    slot = torch.arange(m, device=DEV)[None]
    order = torch.randperm(p, generator=g, device=DEV)
    s["tables"] = torch.where(slot < n[:, None], order[((n.cumsum(0) - n)[:, None] + slot).clamp(max=p - 1)], -1).int()
    # the last rows begin with the first one's pages
    k = min(int(n[0]), int(n[-1])) // 2
    if b > 1 and k:
        s["tables"][-1, :k] = s["tables"][0, :k]
    s["refs"] = torch.zeros((p,), dtype=torch.int32, device=DEV)
    used = s["tables"][s["tables"] >= 0].long()
    s["refs"].scatter_add_(0, used, torch.ones_like(used, dtype=torch.int32))
    s["cache"], s["scales"] = _pool(g, p, case["page"], case["block"])
    s["next"] = (torch.empty_like(s["tables"]), torch.empty_like(s["refs"]))
    s["copies"] = torch.empty((p // 2, 2), dtype=torch.int32, device=DEV)


def _inv_freq(rot, base=10000.0):
    """Radians a position of each pair."""
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    op, b = case["op"], case["b"]
    if op == "fork":
        _prepare_fork(case, s, g)
        return s
    if op == "compact":
        _prepare_compact(case, s, g)
        return s
    cp, il, page = case["cp"], case["interleave"], case["page"]
    if op == "decode":
        counts = _group_counts(case)
        first = [sum(counts[:i]) for i in range(len(counts))]
        lead = torch.tensor([f for f, c in zip(first, counts) for _ in range(c)], device=DEV)
        prefix, most = case["prefix"], case["prefix"] + case["own"]
        room = (most // (cp * il) + 1) * il
        m = -(-room // page)
        shared_pages = [int(_held(torch.tensor(prefix), cp, j, il)) // page for j in range(cp)]
        tables = []
        p = b * m + 3  # (pages that no row uses among them)
        for j in range(cp):
            t = torch.randperm(p, generator=g, device=DEV)[:b * m].view(b, m)
            if case["groups"]:  # whole pages of the prefix are the first row's; what ends inside a page is a copy of its own
                t = torch.where(torch.arange(m, device=DEV)[None] < shared_pages[j], t[lead], t)
            tables.append(t.int())
        s["cache"], s["scales"] = _pool(g, cp * p, page, case["block"])
        s["cache"], s["scales"] = s["cache"].view(cp, p, page, DK), s["scales"].view(cp, p, -1)
        s["q"] = torch.randn((b, case["h"], DK), generator=g, device=DEV).bfloat16()
        s["seq_lens"] = (prefix + _uniform(g, b, 1, case["own"])).int()
        if b == 1:
            s["seq_lens"].fill_(most)
        s["groups"] = torch.stack((lead, torch.tensor([c for c in counts for _ in range(c)], device=DEV)), 1).int()
        # the positions that rows have in common are those of the pages that they have in common
        whole = min((shared_pages[j] * page // il * cp + j) * il + shared_pages[j] * page % il for j in range(cp))
        s["shared"] = torch.full((b,), whole, dtype=torch.int32, device=DEV)
    else:
        m = case["m"]
        p = b * m + 3
        tables = [torch.randperm(p, generator=g, device=DEV)[:b * m].view(b, m).int() for _ in range(cp)]
        s["cache"], s["scales"] = _pool(g, cp * p, page, case["block"])
        s["cache"], s["scales"] = s["cache"].view(cp, p, page, DK), s["scales"].view(cp, p, -1)
        counts = _counts(case)
        s["cu"] = torch.tensor([0] + counts).cumsum(0).int().to(DEV)
        # positions at the end that no row uses: a round over the shards fills them unevenly
        most = torch.tensor([cp * m * page - (cp * il if cp > 1 else 0) - c for c in counts]).clamp(min=0).to(DEV)
        u = torch.rand((b,), generator=g, device=DEV, dtype=torch.float64)
        s["starts"] = torch.minimum((u * (most + 1)).long(), most).int()
        if op == "append":
            n = case["n"]
            s["latent"] = torch.randn((n, DV), generator=g, device=DEV).to(DTYPES[case["dtype"]])
            s["k_rope"] = (3 * torch.randn((n, 64), generator=g, device=DEV)).to(DTYPES[case["dtype"]])
            s["inv_freq"] = _inv_freq(64)
    s["tables"] = torch.stack(tables)
    s["caches"], s["scale_list"] = list(s["cache"].unbind(0)), list(s["scales"].unbind(0))
    s["table_list"] = list(s["tables"].unbind(0))
    return s


# ---- the plain forms ----------------------------------------------------------


def _copy_pages(s, copies):
    """Pages src -> dst of the pool, pairs of -1 left out."""
    real = copies[:, 0] >= 0
    src, dst = copies[real, 0].long(), copies[real, 1].long()
    bytes_ = s["cache"].view(torch.uint8)
    bytes_[dst] = bytes_[src]
    s["scales"][dst] = s["scales"][src]


def _plain_fork(s):
    case, tables, refs = s["case"], s["tables"].long(), s["refs"].long()
    (b, m), p, page = tables.shape, refs.shape[0], case["page"]
    spread = (case["cp"], case["shard"], case["interleave"])
    rows, slot = torch.arange(b, device=DEV), torch.arange(m, device=DEV)[None]
    parents = s["parents"].long()
    some = (parents >= 0) & (parents < b)
    keep = torch.where(some, _held(s["keeps"].long().clamp(min=0), *spread).clamp(max=m * page), 0)
    want = _held(s["wants"].long().clamp(min=0), *spread).clamp(max=m * page)
    n_keep = -(-keep // page)
    n_new = torch.maximum(n_keep, -(-want // page))
    old = torch.where(((tables >= 0) & (tables < p)).int().cumprod(1) > 0, tables, -1)
    taken = torch.where(slot < n_keep[:, None], old[parents.clamp(0, b - 1)], -1)
    taken = torch.where(some[:, None], taken, -1)
    # how many hold each page now
    bins = torch.zeros((p + 1,), dtype=torch.long, device=DEV)
    less = bins.scatter_add(0, old.flatten() + 1, torch.ones_like(old.flatten()))[1:]
    more = bins.scatter_add(0, taken.flatten() + 1, torch.ones_like(taken.flatten()))[1:]
    refs = refs - less + more
    # pages that are about to be written and that others hold as well
    at = (keep // page).clamp(max=m - 1)
    last = taken.gather(1, at[:, None])[:, 0]
    writes = (want > keep) & (keep % page > 0) & (last >= 0)
    slot_of = torch.where(writes, last, p)
    writers = torch.zeros((p + 1,), dtype=torch.long, device=DEV).scatter_add(0, slot_of, writes.long())
    latest = torch.full((p + 1,), -1, device=DEV).scatter_reduce(0, slot_of, rows, "amax")
    page_of = last.clamp(min=0)
    copied = writes & ((writers[page_of] < refs[page_of]) | (latest[page_of] != rows))
    # fresh pages, the lowest first, in the rows' order
    n_taken = (taken >= 0).sum(1)
    need = copied.long() + n_new - n_taken
    before = need.cumsum(0) - need
    free = torch.argsort((refs != 0).int(), stable=True)
    n_free = (refs == 0).sum()
    pool = torch.where(torch.arange(p, device=DEV) < n_free, free, -1)
    pool = torch.cat((pool, torch.full((b * (m + 1),), -1, device=DEV)))
    grown = (slot >= n_taken[:, None]) & (slot < n_new[:, None])
    new = torch.where(grown, pool[(before + copied)[:, None] + slot.clamp(min=0) - n_taken[:, None] * grown], taken)
    instead = pool[before]
    new = torch.where(copied[:, None] & (slot == at[:, None]), instead[:, None], new)
    refs = refs - torch.zeros((p,), dtype=torch.long, device=DEV).scatter_add(0, page_of, copied.long())
    # each page that was dealt has one holder
    dealt = torch.where(torch.arange(p, device=DEV) < need.sum(), pool[:p], -1)
    refs = refs + torch.zeros((p + 1,), dtype=torch.long, device=DEV).scatter_add(
        0, dealt + 1, torch.ones_like(dealt))[1:]
    s["next"][0].copy_(new)
    s["next"][1].copy_(refs)
    pair = copied & (instead >= 0)
    s["copies"].copy_(torch.where(pair[:, None], torch.stack((last, instead), 1), -1))
    s["missing"].copy_((need.sum() - n_free).clamp(min=0))
    _copy_pages(s, s["copies"])
    return *s["next"], s["copies"], s["missing"], s["cache"], s["scales"]


def _plain_compact(s):
    tables, refs = s["tables"].long(), s["refs"].long()
    p = refs.shape[0]
    live = refs > 0
    n = live.sum()
    here = torch.arange(p, device=DEV)
    goes, room = live & (here >= n), ~live & (here < n)
    k = goes.sum()
    src = torch.argsort((~goes).int(), stable=True)  # the pages that move, ascending, then the others
    dst = torch.argsort((~room).int(), stable=True)
    moved = here < k
    to = torch.scatter(here, 0, src, torch.where(moved, dst, src))
    s["next"][0].copy_(torch.where((tables >= 0) & (tables < p), to[tables.clamp(0, p - 1)], tables))
    s["next"][1].copy_(torch.zeros_like(refs).scatter_add(0, to, refs))
    pairs = torch.where(moved[:, None], torch.stack((src, dst), 1), -1)
    s["copies"].copy_(pairs[:p // 2])
    _copy_pages(s, s["copies"])
    return *s["next"], s["copies"], s["cache"], s["scales"]


def _positions(s, n):
    """Row and position of each of n packed tokens."""
    cu = s["cu"].long()
    row = torch.repeat_interleave(torch.arange(len(cu) - 1, device=DEV), cu[1:] - cu[:-1], output_size=n)
    return row, s["starts"].long()[row] + torch.arange(n, device=DEV) - cu[row]


def _plain_append(s):
    case, cache, scales = s["case"], s["cache"], s["scales"]
    cp, p, page, _ = cache.shape
    block, nb, il, b = case["block"], page // case["block"], case["interleave"], case["b"]
    row, pos = _positions(s, case["n"])
    angle = pos.double()[:, None] * s["inv_freq"]
    c, sn = angle.cos().float(), angle.sin().float()
    even, odd = s["k_rope"][:, 0::2].float(), s["k_rope"][:, 1::2].float()
    k = torch.stack((even * c - odd * sn, odd * c + even * sn), -1).flatten(-2)
    x = torch.cat((s["latent"].float(), k), -1)
    shard, loc = _owner(pos, cp, il)
    at = s["tables"].long()[shard, row, loc // page]
    # each block's scale: of its new tokens, and not below what the tokens that it already holds have
    ident = (shard * p + at) * nb + loc % page // block
    peak = torch.full((cp * p * nb,), -1.0, device=DEV).scatter_reduce_(0, ident, x.abs().amax(-1), "amax")
    peak = peak.view(cp, p, nb)
    new = torch.where(peak < 0, scales, _scale_of(peak.clamp(min=0)))
    bytes_ = cache.view(torch.uint8)
    if block > 1:
        j = torch.arange(cp, device=DEV)[:, None]
        held = _held(s["starts"].long()[None], cp, j, il)  # [cp, b] local tokens before
        slot = (held // page).clamp(max=s["tables"].shape[2] - 1)
        pg = s["tables"].long().gather(2, slot[..., None])[..., 0]
        first = held % page // block
        was, peaks = scales[j, pg, first], peak[j, pg, first]
        partly = (held % block > 0) & (peaks >= 0)
        grown = torch.where(partly, torch.maximum(_scale_of(peaks.clamp(min=0)), was), new[j, pg, first])
        new[j, pg, first] = grown
        # the earlier tokens of the blocks that grow
        ratio = torch.where(partly, was / grown, 1.0)[..., None, None]
        tok = first[..., None] * block + torch.arange(block, device=DEV)  # [cp, b, block]
        jj, bb = j[..., None].expand_as(tok), pg[..., None].expand_as(tok)
        codes = cache[jj, bb, tok].float()
        mine = (tok < (held % page)[..., None])[..., None]
        bytes_[jj, bb, tok] = torch.where(mine, (codes * ratio).to(E4M3).float(), codes).to(E4M3).view(torch.uint8)
    scales.copy_(new)
    y = x / new[shard, at, loc % page // block][:, None]
    bytes_[shard, at, loc % page] = y.to(E4M3).view(torch.uint8)
    return cache, scales


def _plain_read(s):
    case, cache = s["case"], s["cache"]
    row, pos = _positions(s, case["n"])
    shard, loc = _owner(pos, case["cp"], case["interleave"])
    at = s["tables"].long()[shard, row, loc // case["page"]]
    here = loc % case["page"]
    x = cache[shard, at, here].float() * s["scales"][shard, at, here // case["block"]][:, None]
    return x.to(DTYPES[case["dtype"]])


def _plain_decode(s):
    case, q = s["case"], s["q"].float()
    cp, b, m = s["tables"].shape
    il, t = case["interleave"], m * case["page"]
    j = torch.arange(cp, device=DEV)[:, None, None]
    kv = s["cache"][j, s["tables"].long()].float()  # [cp, b, m, page, dk]
    kv *= s["scales"][j, s["tables"].long()].repeat_interleave(case["block"], 3)[..., None]
    kv = kv.transpose(0, 1).reshape(b, cp * t, DK)
    loc = torch.arange(t, device=DEV)[None]
    pos = (loc // il * cp + torch.arange(cp, device=DEV)[:, None]) * il + loc % il
    see = (pos.reshape(1, -1) < s["seq_lens"].long()[:, None])[:, None]
    x = (q @ kv.transpose(1, 2) * SCALE).masked_fill(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top.clamp(min=-1e30))
    total = e.sum(-1, keepdim=True)
    o = (e @ kv[..., :DV]) / total.clamp(min=1e-30)
    return o.bfloat16(), (top + total.log())[..., 0]


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"fork": _plain_fork, "compact": _plain_compact, "append": _plain_append, "read": _plain_read,
                "decode": _plain_decode}[op](state)
    import decode_context_mla_dcp_gb300 as dcp
    if op == "fork":
        dcp.mla_cache8_pages_update(state["tables"], state["refs"], state["parents"], state["keeps"], state["wants"],
                                    page=case["page"], cp=case["cp"], shard=case["shard"],
                                    interleave=case["interleave"], out=state["next"], copies=state["copies"],
                                    missing=state["missing"])
        dcp.mla_cache8_pages_copy([state["cache"]], [state["scales"]], state["copies"])
        return *state["next"], state["copies"], state["missing"], state["cache"], state["scales"]
    if op == "compact":
        dcp.mla_cache8_pages_compact(state["tables"], state["refs"], out=state["next"], copies=state["copies"])
        dcp.mla_cache8_pages_copy([state["cache"]], [state["scales"]], state["copies"])
        return *state["next"], state["copies"], state["cache"], state["scales"]
    if op == "append":
        dcp.mla_cache8_append(state["latent"], state["k_rope"], state["caches"], state["scale_list"], state["starts"],
                              cu_new=state["cu"], block=case["block"], interleave=case["interleave"],
                              inv_freq=state["inv_freq"], tables=state["table_list"])
        return state["cache"], state["scales"]
    if op == "read":
        return dcp.mla_cache8_read(state["caches"], state["scale_list"], case["n"], starts=state["starts"],
                                   cu=state["cu"], block=case["block"], interleave=case["interleave"],
                                   dtype=DTYPES[case["dtype"]], tables=state["table_list"])
    shared = {"groups": state["groups"], "shared": state["shared"]} if case["groups"] else {}
    return dcp.mla_cache8_decode(state["q"], state["caches"], state["scale_list"], state["seq_lens"], SCALE,
                                 block=case["block"], interleave=case["interleave"], tables=state["table_list"],
                                 **shared)


# ---- what a pass cannot do without ----------------------------------------------


def _copies_for_work(case):
    """About how many pages a fork copies."""
    return case["b"] // 2 if case["kind"] == "beams" else case["b"] // 20


def work(case):
    op, b = case["op"], case["b"]
    if op in ("fork", "compact"):
        page = case["page"] * (DK + 4 / case["block"])
        lists = 8 * b * case["m"] + 8 * case["p"]  # tables and refs, read and written
        if op == "fork":
            return {"bytes": lists + 2 * _copies_for_work(case) * page, "flops": 0}
        live = max(1, min(int(case["p"] * case["fill"]), b * case["m"])) / case["p"]
        return {"bytes": lists + 2 * live * (1 - live) * case["p"] * page, "flops": 0}
    if op == "append":
        n = case["n"]
        return {"bytes": n * DK * 3 + 4 * max(1, n // case["block"]), "flops": 4 * n * DK}
    if op == "read":
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        return {"bytes": case["n"] * DK * (1 + size) + 4 * max(1, case["n"] // case["block"]),
                "flops": case["n"] * DK}
    mean = case["own"] if b == 1 else 0.5 * (case["own"] + 1)
    seen = b * mean + max(1, case["groups"]) * case["prefix"]  # a group's prefix is read once
    return {"bytes": seen * (DK + 4 / case["block"]) + b * case["h"] * (2 * DK + 2 * DV + 4),
            "flops": 2 * b * (mean + case["prefix"]) * case["h"] * (DK + DV)}


# ---- the definitions in 64 bits, and step by step on the host ---------------------


def _exact_fork(case, s):
    """One row after the other: releases, then copies and fresh pages."""
    b, m, p, page = case["b"], case["m"], case["p"], case["page"]
    refs = s["refs"].tolist()
    old = [[e for e in row if e >= 0] for row in s["tables"].tolist()]
    parents, keeps, wants = s["parents"].tolist(), s["keeps"].tolist(), s["wants"].tolist()
    mine = [0]  # local tokens before each position
    for x in range(max(keeps + wants + [0])):
        mine.append(mine[-1] + (x // case["interleave"] % case["cp"] == case["shard"]))
    new, plan = [], []
    for i in range(b):
        some = 0 <= parents[i] < b
        keep = min(mine[max(keeps[i], 0)], m * page) if some else 0
        want = min(mine[max(wants[i], 0)], m * page)
        new.append(list(old[parents[i]][:(keep + page - 1) // page]) if some else [])
        plan.append((keep, want))
    for i in range(b):
        for e in old[i]:
            refs[e] -= 1
        for e in new[i]:
            refs[e] += 1
    free = [e for e in range(p) if refs[e] == 0]
    writers = {}
    for i in range(b):
        keep, want = plan[i]
        if want > keep and keep % page and keep // page < len(new[i]):
            writers.setdefault(new[i][keep // page], []).append(i)
    others = {e: refs[e] - len(w) for e, w in writers.items()}
    copies, short = [[-1, -1] for _ in range(b)], 0

    def take():
        nonlocal short
        if free:
            e = free.pop(0)
            refs[e] = 1
            return e
        short += 1
        return -1

    for i in range(b):
        keep, want = plan[i]
        at = keep // page
        if want > keep and keep % page and at < len(new[i]):
            e = new[i][at]
            if others[e] > 0 or writers[e][-1] != i:
                refs[e] -= 1
                new[i][at] = take()
                if new[i][at] >= 0:
                    copies[i] = [e, new[i][at]]
        for _ in range(max((keep + page - 1) // page, (want + page - 1) // page) - len(new[i])):
            new[i].append(take())
    cache, scales = s["cache"].double(), s["scales"].double()
    for src, dst in copies:
        if src >= 0:
            cache[dst], scales[dst] = cache[src].clone(), scales[src].clone()
    put = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return put([r + [-1] * (m - len(r)) for r in new]), put(refs), put(copies), put([short]), cache, scales


def _exact_compact(case, s):
    refs, tables, p = s["refs"].tolist(), s["tables"].tolist(), case["p"]
    n = sum(r > 0 for r in refs)
    pairs = list(zip([e for e in range(n, p) if refs[e] > 0], [e for e in range(n) if refs[e] == 0]))
    to = dict(pairs)
    for a, z in pairs:
        refs[z], refs[a] = refs[a], 0
    cache, scales = s["cache"].double(), s["scales"].double()
    if pairs:
        a, z = torch.tensor(pairs, device=DEV).T
        cache[z], scales[z] = cache[a], scales[a]
    put = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    copies = put([list(x) for x in pairs] + [[-1, -1]] * (p // 2 - len(pairs))).view(p // 2, 2)
    return put([[to.get(e, e) for e in row] for row in tables]), put(refs), copies, cache, scales


def exact(case, seed):
    s = prepare(case, seed)
    op, b = case["op"], case["b"]
    if op == "fork":
        return _exact_fork(case, s)
    if op == "compact":
        return _exact_compact(case, s)
    cp, il, block, page = case["cp"], case["interleave"], case["block"], case["page"]
    tables = s["tables"].long()

    def places(i, pos):
        """Shard, page and token of positions of row i."""
        j = torch.div(pos, il, rounding_mode="floor").remainder(cp)
        at = pos // (cp * il) * il + pos.remainder(il)
        return j, tables[j, i, at // page], at % page

    if op == "decode":
        out = torch.zeros((b, case["h"], DV), dtype=torch.float64, device=DEV)
        lse = torch.full((b, case["h"]), -math.inf, dtype=torch.float64, device=DEV)
        for i, n in enumerate(s["seq_lens"].tolist()):
            j, e, at = places(i, torch.arange(n, device=DEV))
            k = s["cache"][j, e, at].double() * s["scales"][j, e, at // block].double()[:, None]
            x = s["q"][i].double() @ k.T * SCALE
            lse[i] = torch.logsumexp(x, 1)
            out[i] = torch.softmax(x, 1) @ k[:, :DV]
        return out, lse
    cu, starts = s["cu"].tolist(), s["starts"].tolist()
    if op == "read":
        rows = []
        for i in range(b):
            j, e, at = places(i, torch.arange(cu[i + 1] - cu[i], device=DEV) + starts[i])
            rows.append(s["cache"][j, e, at].double() * s["scales"][j, e, at // block].double()[:, None])
        return torch.cat(rows)
    cache, scales = s["cache"].double(), s["scales"].double()
    for i in range(b):
        if cu[i + 1] == cu[i]:
            continue
        pos = torch.arange(cu[i + 1] - cu[i], device=DEV) + starts[i]
        z = torch.polar(torch.ones((1, 32), dtype=torch.float64, device=DEV), pos.double()[:, None] * s["inv_freq"])
        w = torch.view_as_complex(s["k_rope"][cu[i]:cu[i + 1]].double().view(-1, 32, 2)) * z
        x = torch.cat((s["latent"][cu[i]:cu[i + 1]].double(), torch.view_as_real(w).flatten(1)), 1)
        j, e, at = places(i, pos)
        for shard in range(cp):
            mine = j == shard
            if not bool(mine.any()):
                continue
            # blocks in the order of the row's tokens on the shard
            which = e[mine] * (page // block) + at[mine] // block
            block_ids, back = torch.unique(which, return_inverse=True)
            need = torch.zeros((len(block_ids),), dtype=torch.float64, device=DEV)
            need.scatter_reduce_(0, back, x[mine].abs().amax(1), "amax")
            need = torch.exp2(torch.ceil(torch.log2(need / E4M3_MAX)).clamp(min=MIN_EXP))
            first, begin = int(e[mine][0]), int(at[mine][0])
            if begin % block:
                k = int((block_ids == int(which[0])).nonzero())
                old = scales[shard, first, begin // block].clone()
                need[k] = torch.maximum(need[k], old)
                part = slice(begin // block * block, begin)
                cache[shard, first, part] = (cache[shard, first, part] * (old / need[k])).float().to(E4M3).double()
            scales[shard].view(-1)[block_ids] = need
            cache[shard, e[mine], at[mine]] = (x[mine] / need[back][:, None]).float().to(E4M3).double()
    return cache, scales
