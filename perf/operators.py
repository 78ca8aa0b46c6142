"""The cases on which the 8-bit latent cache's operators are measured.

Four operators, as a serving program chains them for one layer and one step:

  rope    rotary positions on part of each query head (mla_rope)
  append  new tokens' keys rotated, quantised to e4m3 and written to the cache (mla_cache8_append)
  read    cached positions read back, in order over the context shards (mla_cache8_read)
  decode  single-token attention over the cache, with its log-sum-exp; optionally a sliding
          window with a few first tokens that stay visible (mla_cache8_decode)

The cache of a row is [T, 512 latent + 64 rotary] e4m3 with one fp32 scale for each block of
tokens; under context parallelism position p lives on shard (p / interleave) mod cp. Where `own`
is false each operator runs in its plain form: elementary torch operations in 32 bits (angles in
64), rounded once at the end.
"""
import math

import torch

own = False

DEV = "cuda"
DV = 512             # latent dims: the values
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_EXP = -60        # smallest exponent of a block's scale
SCALE = 192 ** -0.5  # softmax scale of 128 + 64 dims a head
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of one sequence, 16 heads (a shard of a model's heads): its rotary part, interleaved pairs
        {"name": "rope_token", "op": "rope", "n": 1, "h": 16, "d": 64, "start": 0, "rot": 64, "dtype": "bf16",
         "interleaved": True, "yarn": 1.0, "into": 0, "far": 4096},
        # a decode batch: halves, frequencies stretched for a long context, into the last 64 of 576 dims of the queries
        {"name": "rope_batch_into", "op": "rope", "n": 128, "h": 128, "d": 64, "start": 0, "rot": 64, "dtype": "bf16",
         "interleaved": False, "yarn": 40.0, "into": 576, "far": 163840},
        # a prompt's queries: 128 plain + 64 rotary dims a head, the plain ones copied
        {"name": "rope_prompt", "op": "rope", "n": 8192, "h": 64, "d": 192, "start": 128, "rot": 64, "dtype": "bf16",
         "interleaved": True, "yarn": 32.0, "into": 0, "far": 262144},
        # one token of one sequence: the smallest append
        {"name": "append_token", "op": "append", "b": 1, "n": 1, "cp": 1, "interleave": 1, "block": 1, "t": 4096,
         "ragged": False, "dtype": "bf16"},
        # speculative decoding: 256 requests x 4 tokens to verify, four context shards, blocks that already hold tokens
        {"name": "append_verify", "op": "append", "b": 256, "n": 1024, "cp": 4, "interleave": 16, "block": 16, "t": 512,
         "ragged": False, "dtype": "bf16"},
        # prompts of mixed lengths, 16385 tokens in all, blocks of 64
        {"name": "append_prompt", "op": "append", "b": 5, "n": 16385, "cp": 1, "interleave": 1, "block": 64, "t": 16448,
         "ragged": True, "dtype": "bf16"},
        # a chunk of two sequences' context for the next prompt chunk
        {"name": "read_chunk", "op": "read", "b": 2, "n": 2047, "cp": 1, "interleave": 1, "block": 1, "t": 2048,
         "ragged": True, "dtype": "bf16"},
        # long contexts gathered from four shards into position order
        {"name": "read_long", "op": "read", "b": 8, "n": 262144, "cp": 4, "interleave": 16, "block": 64, "t": 16384,
         "ragged": True, "dtype": "bf16"},
        # one sequence with a short context and 16 heads: latency
        {"name": "decode_short", "op": "decode", "b": 1, "h": 16, "cp": 1, "interleave": 1, "block": 1, "t": 200,
         "ragged": False, "window": 0, "sinks": 0},
        # 8 sequences x 4096 tokens, 128 heads
        {"name": "decode_batch", "op": "decode", "b": 8, "h": 128, "cp": 1, "interleave": 1, "block": 1, "t": 4096,
         "ragged": False, "window": 0, "sinks": 0},
        # a serving batch: 64 sequences of mixed lengths, 128 heads, blocks of 64
        {"name": "decode_serving", "op": "decode", "b": 64, "h": 128, "cp": 1, "interleave": 1, "block": 64, "t": 16384,
         "ragged": True, "window": 0, "sinks": 0},
        # 16 sequences of up to 64K tokens on four shards, 64 heads, the last 4096 tokens and the first 4 visible
        {"name": "decode_window", "op": "decode", "b": 16, "h": 64, "cp": 4, "interleave": 1, "block": 1, "t": 16384,
         "ragged": True, "window": 4096, "sinks": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "decode"])
    if op == "rope":
        rot = rng.choice([32, 64, 64, 128])
        start = rng.choice([0, 64, 128, 512])
        d = start + rot + rng.choice([0, 0, 32])
        h = rng.choice([1, 7, 16, 40, 64, 128])
        n = _log(rng, 1, max(2, 8192 * 64 * 192 // (h * d)))
        return {"op": op, "n": min(n, 30000), "h": h, "d": d, "start": start, "rot": rot,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "interleaved": rng.random() < 0.5,
                "yarn": rng.choice([1.0, 4.0, 40.0]), "into": d + rng.choice([64, 512]) if rng.random() < 0.4 else 0,
                "far": _log(rng, 100, 1000000)}
    cp = rng.choice([1, 1, 2, 4, 8])
    interleave = rng.choice([1, 16, 64]) if cp > 1 else 1
    block = rng.choice([1, 1, 16, 64])
    if op == "append":
        b = _log(rng, 1, 256)
        n = _log(rng, b, max(b + 1, 16385))
        most = 2 * (n // b) + 64  # tokens of the longest row
        t = (most // cp + 2 * interleave + 64) // 64 * 64 + 64
        return {"op": op, "b": b, "n": n, "cp": cp, "interleave": interleave, "block": block, "t": t,
                "ragged": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    if op == "read":
        b = _log(rng, 1, 64)
        n = _log(rng, b, 200000)
        t = (2 * (n // b) // cp + 2 * interleave + 64) // 64 * 64 + 64
        return {"op": op, "b": b, "n": n, "cp": cp, "interleave": interleave, "block": block, "t": t,
                "ragged": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    h = rng.choice([8, 16, 24, 32, 64, 128])
    b = _log(rng, 1, 64)
    t = _log(rng, 1, max(2, 64 * 128 * 16384 // (2 * b * max(h, 64) * cp)))
    t = min(t, 131072 // cp)
    whole = max(block, interleave)  # caches are allocated in whole blocks and whole rounds over the shards
    t = -(-t // whole) * whole
    window = rng.choice([0, 0, _log(rng, 1, max(2, t * cp))])
    return {"op": op, "b": b, "h": h, "cp": cp, "interleave": interleave, "block": block, "t": t,
            "ragged": rng.random() < 0.6, "window": window, "sinks": rng.choice([0, 4, 64]) if window else 0}


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


def _inv_freq(rot, yarn, base=10000.0, original=4096):
    """Radians a position, and the factor on cos and sin: stretched over long wavelengths (YaRN) for yarn > 1."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-i / rot)
    if yarn == 1.0:
        return f, 1.0
    edge = [rot * math.log(original / (x * 2 * math.pi)) / (2 * math.log(base)) for x in (32.0, 1.0)]
    lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
    keep = 1 - ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f / yarn * (1 - keep) + f * keep, 0.1 * math.log(yarn) + 1.0


def _quantise(x, block):
    """[.., T, D] floats -> e4m3 and one power-of-two scale for each block of tokens: the cache's format."""
    t = x.shape[-2]
    xb = x.unflatten(-2, (t // block, block))
    s = _scale_of(xb.abs().amax((-1, -2)))
    return (xb / s[..., None, None]).flatten(-3, -2).to(E4M3), s


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s (at least 2^-60)."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, k, MIN_EXP))


def _cache(g, cp, b, t, dk, block):
    """A filled cache: normalised latents with some louder tokens, rotary keys of about twice their size."""
    kv = torch.empty((cp, b, t, dk), dtype=E4M3, device=DEV)
    scales = torch.empty((cp, b, t // block), dtype=torch.float32, device=DEV)
    for j in range(cp):
        for i in range(b):
            x = torch.randn((t, dk), generator=g, device=DEV)
            x[:, DV:] *= 2
            x *= torch.exp(0.3 * torch.randn((t, 1), generator=g, device=DEV))
            kv[j, i], scales[j, i] = _quantise(x.bfloat16().float(), block)
    return kv, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rope":
        x = torch.randn((case["n"], case["h"], case["d"]), generator=g, device=DEV).to(DTYPES[case["dtype"]])
        f, s["mscale"] = _inv_freq(case["rot"], case["yarn"])
        s["x"], s["inv_freq"] = x, f.to(DEV)
        s["positions"] = torch.randint(0, case["far"], (case["n"],), generator=g, device=DEV)
        if case["into"]:  # the queries' buffer, whose first dims another operator has written
            s["buffer"] = torch.randn((case["n"], case["h"], case["into"]), generator=g, device=DEV).to(x.dtype)
            s["out"] = s["buffer"][..., case["into"] - case["d"]:]
        else:
            s["buffer"] = s["out"] = torch.empty_like(x)
        return s
    cp, b, t, block = case["cp"], case["b"], case["t"], case["block"]
    dk = DV + 64
    s["cache"], s["scales"] = _cache(g, cp, b, t, dk, block)
    s["caches"], s["scale_list"] = list(s["cache"].unbind(0)), list(s["scales"].unbind(0))
    if case["op"] == "decode":
        s["q"] = torch.randn((b, case["h"], dk), generator=g, device=DEV).bfloat16()
        # lengths of a serving batch: from a few tokens to the whole cache
        if case["ragged"]:
            u = torch.rand((b,), generator=g, device=DEV)
            s["seq_lens"] = (1 + u * (cp * t - 1)).int()
        else:
            s["seq_lens"] = torch.full((b,), cp * t - (1 if cp * t > 1 else 0), dtype=torch.int32, device=DEV)
        return s
    counts = _counts(case)
    cu = torch.tensor([0] + counts).cumsum(0)
    s["cu"] = cu.int().to(DEV)
    # positions at the end that no row uses: a round over the shards fills them unevenly
    most = torch.tensor([cp * t - (cp * case["interleave"] if cp > 1 else 0) - c for c in counts]).clamp(min=0).to(DEV)
    u = torch.rand((b,), generator=g, device=DEV, dtype=torch.float64)
    s["starts"] = torch.minimum((u * (most + 1)).long(), most).int()
    if case["op"] == "append":
        n = case["n"]
        s["latent"] = torch.randn((n, DV), generator=g, device=DEV).to(DTYPES[case["dtype"]])
        s["k_rope"] = (3 * torch.randn((n, 64), generator=g, device=DEV)).to(DTYPES[case["dtype"]])
        f, s["mscale"] = _inv_freq(64, 1.0)
        s["inv_freq"] = f.to(DEV)
    return s


# ---- the plain forms ----------------------------------------------------------


def _rotate(x, pos, inv_freq, mscale, interleaved):
    """x [.., n, h, rot] fp32 rotated by each position's angles."""
    ang = pos.double()[:, None] * inv_freq
    c, s = (ang.cos() * mscale).float()[:, None], (ang.sin() * mscale).float()[:, None]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _plain_rope(s):
    case, x = s["case"], s["x"]
    lo, hi = case["start"], case["start"] + case["rot"]
    r = _rotate(x[..., lo:hi].float(), s["positions"], s["inv_freq"], s["mscale"], case["interleaved"])
    s["out"][..., lo:hi] = r.to(x.dtype)
    if case["d"] > case["rot"]:
        s["out"][..., :lo], s["out"][..., hi:] = x[..., :lo], x[..., hi:]
    return s["buffer"]


def _positions(s, n):
    """Row and position of each of n packed tokens."""
    cu = s["cu"].long()
    row = torch.repeat_interleave(torch.arange(len(cu) - 1, device=DEV), cu[1:] - cu[:-1], output_size=n)
    return row, s["starts"].long()[row] + torch.arange(n, device=DEV) - cu[row]


def _plain_append(s):
    case, cache, scales = s["case"], s["cache"], s["scales"]
    cp, b, t, dk = cache.shape
    block, nb, il = case["block"], scales.shape[2], case["interleave"]
    row, pos = _positions(s, case["n"])
    k = _rotate(s["k_rope"].float()[:, None], pos, s["inv_freq"], s["mscale"], True)[:, 0]
    x = torch.cat((s["latent"].float(), k), -1)
    shard, loc = _owner(pos, cp, il)
    # each block's scale: of its new tokens, and not below what the tokens that it already holds have
    ident = (shard * b + row) * nb + loc // block
    peak = torch.full((cp * b * nb,), -1.0, device=DEV).scatter_reduce_(0, ident, x.abs().amax(-1), "amax")
    peak = peak.view(cp, b, nb)
    j = torch.arange(cp, device=DEV)[:, None]
    start = s["starts"].long()[None]
    held = start // (il * cp) * il + (start % (il * cp) - j * il).clamp(0, il)  # [cp, b] local tokens before
    first, partly = held // block, held % block > 0
    here = (torch.arange(nb, device=DEV) == first[..., None]) & partly[..., None]
    new = _scale_of(peak.clamp(min=0))
    new = torch.where(here, torch.maximum(new, scales), new)
    new = torch.where(peak < 0, scales, new)
    # the earlier tokens of the blocks that grow
    bytes_ = cache.view(torch.uint8)
    if block > 1:
        at = first.clamp(max=nb - 1)
        ratio = (scales.gather(2, at[..., None]) / new.gather(2, at[..., None]))[..., None]
        tok = at[..., None] * block + torch.arange(block, device=DEV)  # [cp, b, block]
        jj, bb = j[..., None].expand_as(tok), torch.arange(b, device=DEV)[None, :, None].expand_as(tok)
        was = cache[jj, bb, tok]
        redone = torch.where((tok < held[..., None])[..., None], (was.float() * ratio).to(E4M3).float(), was.float())
        bytes_[jj, bb, tok] = redone.to(E4M3).view(torch.uint8)
    scales.copy_(new)
    y = x / new[shard, row, loc // block][:, None]
    bytes_[shard, row, loc] = y.to(E4M3).view(torch.uint8)
    return cache, scales


def _plain_read(s):
    case, cache = s["case"], s["cache"]
    row, pos = _positions(s, case["n"])
    shard, loc = _owner(pos, case["cp"], case["interleave"])
    x = cache[shard, row, loc].float() * s["scales"][shard, row, loc // case["block"]][:, None]
    return x.to(DTYPES[case["dtype"]])


def _visible(case, seq_lens):
    """[b, cp * t] truth values: which cached tokens a row attends to."""
    t, cp, il = case["t"], case["cp"], case["interleave"]
    loc = torch.arange(t, device=DEV)[None]
    pos = (loc // il * cp + torch.arange(cp, device=DEV)[:, None]) * il + loc % il
    pos, end = pos.reshape(1, -1), seq_lens.long()[:, None]
    see = pos < end
    return see & ((pos >= end - case["window"]) | (pos < case["sinks"])) if case["window"] else see


def _plain_decode(s):
    case, q = s["case"], s["q"].float()
    kv = s["cache"].float() * s["scales"].repeat_interleave(case["block"], 2)[..., None]
    kv = kv.transpose(0, 1).flatten(1, 2)  # [b, cp * t, dk]
    see = _visible(case, s["seq_lens"])[:, None]
    x = (q @ kv.transpose(1, 2) * SCALE).masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = (p @ kv[..., :DV]) / total.clamp(min=1e-30)
    return o.bfloat16(), (m + total.log())[..., 0]


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "decode": _plain_decode}[op](state)
    import decode_context_mla_dcp_gb300 as dcp
    if op == "rope":
        dcp.mla_rope(state["x"], state["positions"], state["inv_freq"], start=case["start"],
                     interleaved=case["interleaved"], mscale=state["mscale"], out=state["out"])
        return state["buffer"]
    if op == "append":
        dcp.mla_cache8_append(state["latent"], state["k_rope"], state["caches"], state["scale_list"], state["starts"],
                              cu_new=state["cu"], block=case["block"], interleave=case["interleave"],
                              inv_freq=state["inv_freq"], mscale=state["mscale"])
        return state["cache"], state["scales"]
    if op == "read":
        return dcp.mla_cache8_read(state["caches"], state["scale_list"], case["n"], starts=state["starts"],
                                   cu=state["cu"], block=case["block"], interleave=case["interleave"],
                                   dtype=DTYPES[case["dtype"]])
    return dcp.mla_cache8_decode(state["q"], state["caches"], state["scale_list"], state["seq_lens"], SCALE,
                                 block=case["block"], interleave=case["interleave"], window=case["window"],
                                 sinks=case["sinks"])


# ---- what a pass cannot do without ----------------------------------------------


def _lengths_for_work(case):
    """Mean visible tokens of a row over all shards."""
    whole = case["cp"] * case["t"]
    if not case["ragged"]:
        n = max(1, whole - 1)
        return float(min(n, case["window"] + case["sinks"]) if case["window"] else n)
    if not case["window"]:
        return 0.5 * (whole + 1)
    w = min(whole, case["window"] + case["sinks"])
    return w * (1 - w / whole) + 0.5 * w * w / whole  # lengths below the window are seen whole


def work(case):
    op, dk = case["op"], DV + 64
    if op == "rope":
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        return {"bytes": 2 * case["n"] * case["h"] * case["d"] * size + 8 * case["n"],
                "flops": 3 * case["n"] * case["h"] * case["rot"]}
    if op == "append":
        n = case["n"]
        return {"bytes": n * dk * 3 + 4 * max(1, n // case["block"]), "flops": 4 * n * dk}
    if op == "read":
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        return {"bytes": case["n"] * dk * (1 + size) + 4 * max(1, case["n"] // case["block"]),
                "flops": case["n"] * dk}
    seen = _lengths_for_work(case) * case["b"]
    return {"bytes": seen * (dk + 4 / case["block"]) + case["b"] * case["h"] * (2 * dk + 2 * DV + 4),
            "flops": 2 * seen * case["h"] * (dk + DV)}


# ---- the definitions in 64 bits ---------------------------------------------------


def _turned(x, pos, inv_freq, mscale, interleaved):
    """The rotation as a product of complex numbers, 64-bit parts."""
    z = torch.polar(torch.full_like(inv_freq, mscale)[None].expand(len(pos), -1), pos.double()[:, None] * inv_freq)
    half = x.shape[-1] // 2
    re, im = (x[..., ::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    w = torch.complex(re.contiguous(), im.contiguous()) * z[:, None]
    return torch.view_as_real(w).flatten(-2) if interleaved else torch.cat((w.real, w.imag), -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, b = case["op"], case.get("b", 0)
    if op == "rope":
        x = s["x"].double()
        lo, hi = case["start"], case["start"] + case["rot"]
        x[..., lo:hi] = _turned(x[..., lo:hi], s["positions"], s["inv_freq"], s["mscale"], case["interleaved"])
        return torch.cat((s["buffer"][..., :case["into"] - case["d"]].double(), x), -1) if case["into"] else x
    cp, il, block = case["cp"], case["interleave"], case["block"]
    cu = s["cu"].tolist() if "cu" in s else None
    if op == "read":
        rows = []
        for i in range(b):
            pos = torch.arange(cu[i + 1] - cu[i], device=DEV) + int(s["starts"][i])
            j, at = torch.div(pos, il, rounding_mode="floor").remainder(cp), pos // (cp * il) * il + pos.remainder(il)
            rows.append(s["cache"][j, i, at].double() * s["scales"][j, i, at // block].double()[:, None])
        return torch.cat(rows)
    if op == "append":
        cache, scales = s["cache"].double(), s["scales"].double()
        for i in range(b):
            n, start = cu[i + 1] - cu[i], int(s["starts"][i])
            if not n:
                continue
            pos = torch.arange(n, device=DEV) + start
            k = _turned(s["k_rope"][cu[i]:cu[i + 1], None].double(), pos, s["inv_freq"], s["mscale"], True)[:, 0]
            x = torch.cat((s["latent"][cu[i]:cu[i + 1]].double(), k), 1)
            for j in range(cp):
                mine = torch.div(pos, il, rounding_mode="floor").remainder(cp) == j
                if not bool(mine.any()):
                    continue
                at = (pos // (cp * il) * il + pos.remainder(il))[mine]
                xs, lo = x[mine], int(at[0])
                first, last = lo // block, int(at[-1]) // block
                need = torch.zeros((last - first + 1,), dtype=torch.float64, device=DEV)
                need.scatter_reduce_(0, at // block - first, xs.abs().amax(1), "amax")
                need = torch.exp2(torch.ceil(torch.log2(need / E4M3_MAX)).clamp(min=MIN_EXP))
                if lo % block:
                    old = scales[j, i, first].clone()
                    need[0] = torch.maximum(need[0], old)
                    part = slice(first * block, lo)
                    cache[j, i, part] = (cache[j, i, part] * (old / need[0])).float().to(E4M3).double()
                scales[j, i, first:last + 1] = need
                cache[j, i, at] = (xs / need[at // block - first][:, None]).float().to(E4M3).double()
        return cache, scales
    out = torch.zeros((b, case["h"], DV), dtype=torch.float64, device=DEV)
    lse = torch.full((b, case["h"]), -math.inf, dtype=torch.float64, device=DEV)
    for i in range(b):
        end = int(s["seq_lens"][i])
        pos = torch.arange(end, device=DEV)
        if case["window"]:
            pos = pos[(pos >= end - case["window"]) | (pos < case["sinks"])]
        if not len(pos):
            continue
        j, at = torch.div(pos, il, rounding_mode="floor").remainder(cp), pos // (cp * il) * il + pos.remainder(il)
        k = s["cache"][j, i, at].double() * s["scales"][j, i, at // block].double()[:, None]
        x = s["q"][i].double() @ k.T * SCALE
        lse[i] = torch.logsumexp(x, 1)
        out[i] = torch.softmax(x, 1) @ k[:, :DV]
    return out, lse
