"""The paged cache's operators on the GPU against their plain forms (oracle/pages.py, oracle/cache8.py). Tables, counts
and copied bytes are whole numbers and have to be equal."""
import random

import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from oracle import cache8
from oracle import pages as ref
from .test_gpu_cache8 import check_decode

pytestmark = pytest.mark.gpu

DEV = "cuda"


def ints(x, *shape):
    t = torch.tensor(x, dtype=torch.int32, device=DEV)
    return t.view(shape) if shape else t


def make_tables(r, B, M, P, fill=0.7, shared=0.3):
    """Random rows of distinct pages, some of which begin with another row's; and the counts."""
    order = r.sample(range(P), P)
    tables, at = [], 0
    for b in range(B):
        n = min(r.randint(0, M), max(0, int(P * fill) - at))
        row = order[at:at + n]
        at += n
        if b and r.random() < shared:
            other = [e for e in tables[r.randrange(b)] if e >= 0]
            row = (other[:r.randint(0, len(other))] + row)[:M]
        tables.append(row + [-1] * (M - len(row)))
    refs = [0] * P
    for row in tables:
        for e in row:
            if e >= 0:
                refs[e] += 1
    return tables, refs


def check_update(tables, refs, parents, keeps, wants, page, **kw):
    """Both forms, in place and into other tensors, against the plain one."""
    B, M, P = len(tables), len(tables[0]), len(refs)
    want = ref.update(tables, refs, parents, keeps, wants, page, **kw)
    rows = [ints(x, B) for x in (parents, keeps, wants)]
    t, f = ints(tables, B, M), ints(refs)
    out = (torch.full_like(t, 77), torch.full_like(f, 77))
    got = dcp.mla_cache8_pages_update(t, f, *rows, page=page, out=out, **kw)
    assert got[0] is out[0] and got[1] is out[1]
    assert t.tolist() == tables and f.tolist() == refs  # (the inputs are as they were)
    for g in (got, dcp.mla_cache8_pages_update(t, f, *rows, page=page, **kw)):
        assert g[0].tolist() == want[0]
        assert g[1].tolist() == want[1]
        assert g[2].tolist() == want[2]
        assert g[3].tolist() == [want[3]]
    assert g[0] is t and g[1] is f
    return want


@pytest.mark.parametrize("B,M,P,page,cp,interleave", [
    (1, 1, 1, 32, 1, 1), (1, 1, 5, 64, 1, 1), (2, 3, 9, 64, 1, 1), (4, 40, 200, 64, 1, 1), (17, 7, 100, 128, 2, 1),
    (33, 300, 3000, 32, 1, 1), (64, 20, 900, 64, 4, 16), (257, 9, 1500, 256, 1, 1), (5, 1000, 4000, 32, 3, 64),
    (1500, 3, 3000, 64, 1, 1)])
def test_update_random(B, M, P, page, cp, interleave):
    for seed in range(4):
        r = random.Random(1000 * B + seed)
        tables, refs = make_tables(r, B, M, P)
        for e in r.sample(range(P), P // 10):
            refs[e] += 1  # pages that the program keeps besides
        most = M * page * cp
        parents = [r.choice([b, b, b, -1, r.randrange(B), r.randrange(B)]) for b in range(B)]
        keeps = [r.randint(0, most) if r.random() < 0.5 else r.randint(0, min(most, 3 * page)) for _ in range(B)]
        wants = [max(0, k + r.choice([0, 1, 4, -3, page, 2 * page])) for k in keeps]
        check_update(tables, refs, parents, keeps, wants, page, cp=cp, shard=seed % cp, interleave=interleave)


def test_update_beams():
    """Beams that descend from two of four rows, over several steps, each state from the one before."""
    r = random.Random(5)
    tables, refs = [[-1] * 6 for _ in range(8)], [0] * 40
    lens = [0] * 8
    tables, refs, _, _ = check_update(tables, refs, list(range(8)), lens, [150] * 8, 64)
    lens = [150] * 8
    for _ in range(12):
        parents = [4 * (b // 4) + r.randrange(4) for b in range(8)]
        tables, refs, copies, missing = check_update(tables, refs, parents, [lens[p] for p in parents],
                                                     [lens[p] + 7 for p in parents], 64)
        lens = [lens[p] + 7 for p in parents]
        assert missing == 0
        held = [0] * 40
        for row in tables:
            for e in row:
                held[e] += e >= 0
        assert held == refs
        # no row writes where another can see it
        for b in range(8):
            e = tables[b][(lens[b] - 1) // 64]
            assert refs[e] == 1 or (lens[b] - 7) % 64 == 0


@pytest.mark.parametrize("P", [1, 2, 3, 8])
def test_update_when_the_pool_runs_out(P):
    tables = [[0, -1, -1], [0, -1, -1], [-1, -1, -1]]
    refs = [2] + [0] * (P - 1)
    check_update(tables, refs, [0, 1, 0], [40, 40, 30], [100, 192, 31], 64)


def test_update_takes_bad_values():
    """Parents outside the rows, negative and far positions, entries that are no page."""
    tables = [[0, 9, 1], [1 << 30, 2, -1], [3, -5, 4], [4, 2, 1]]
    refs = [1, 1, 1, 1, 1, 0]
    check_update(tables, refs, [4, -7, 2, (1 << 31) - 1], [64, 5, 190, 3], [-5, 1, (1 << 31) - 1, 3], 64)
    check_update(tables, refs, [1, 0, 2, 3], [190, 190, -(1 << 31), 64], [0, 0, 0, 500], 64)


def test_update_of_a_large_table():
    """More entries and pages than a warp's turn: every page of a full pool changes hands."""
    B, M = 40, 1200
    P = B * M
    tables = [list(range(b * M, (b + 1) * M)) for b in range(B)]
    refs = [1] * P
    most = M * 32
    check_update(tables, refs, [(b + 1) % B for b in range(B)], [most - 5] * B, [most] * B, 32)
    check_update(tables, refs, [0] * B, [most - 5] * B, [most] * B, 32)
    check_update(tables, refs, [b if b % 2 else -1 for b in range(B)], [most // 2 + 1] * B, [most] * B, 32)


def test_update_of_a_pool_that_shared_memory_does_not_hold():
    """262,144 pages are kept on chip; and more rows than are."""
    r = random.Random(3)
    for B, M, P in ((50, 60, 300_001), (20_000, 2, 50_000), (20, 60, 150_000)):
        tables, refs = make_tables(r, B, M, P, 0.5)
        parents = [r.choice([b, b, -1, r.randrange(B)]) for b in range(B)]
        keeps = [r.randint(0, M * 32) for _ in range(B)]
        check_update(tables, refs, parents, keeps, [k + r.choice([0, 1, 40]) for k in keeps], 32)


def test_update_of_no_rows():
    t, f = torch.empty((0, 4), dtype=torch.int32, device=DEV), ints([0, 2, 0])
    e = torch.empty((0,), dtype=torch.int32, device=DEV)
    t2, f2, copies, missing = dcp.mla_cache8_pages_update(t, f, e, e, e, page=64)
    assert f2.tolist() == [0, 2, 0] and copies.shape == (0, 2) and missing.tolist() == [0]


def check_compact(tables, refs):
    B, M, P = len(tables), len(tables[0]), len(refs)
    want = ref.compact(tables, refs)
    pairs = want[2] + [[-1, -1]] * (P // 2 - len(want[2]))
    t, f = ints(tables, B, M), ints(refs)
    out = (torch.full_like(t, 77), torch.full_like(f, 77))
    got = dcp.mla_cache8_pages_compact(t, f, out=out)
    assert t.tolist() == tables and f.tolist() == refs
    for g in (got, dcp.mla_cache8_pages_compact(t, f)):
        assert g[0].tolist() == want[0]
        assert g[1].tolist() == want[1]
        assert g[2].tolist() == pairs
    assert g[0] is t and g[1] is f


@pytest.mark.parametrize("B,M,P", [(1, 1, 1), (1, 1, 2), (2, 3, 9), (13, 40, 384), (33, 300, 9001), (300, 5, 70000)])
@pytest.mark.parametrize("fill", [0.0, 0.3, 0.5, 0.9, 1.0])
def test_compact(B, M, P, fill):
    r = random.Random(B * P)
    tables, refs = make_tables(r, B, M, P, fill)
    for e in r.sample(range(P), P // 20):
        refs[e] += 1
    check_compact(tables, refs)


def test_compact_leaves_what_is_no_page():
    check_compact([[7, -1, 5], [99, -3, 6], [2, 7, 1 << 30]], [0, 0, 0, 0, 0, 1, 0, 2])


def make_pools(g, pools, P, page, dk, block):
    kv = [torch.randint(0, 256, (P, page, dk), generator=g, device=DEV, dtype=torch.uint8) for _ in range(pools)]
    return kv, [torch.rand((P, page // block), generator=g, device=DEV) for _ in range(pools)]


@pytest.mark.parametrize("pools,P,page,dk,block", [
    (1, 3, 32, 576, 1), (2, 9, 64, 512, 16), (5, 40, 128, 576, 128), (1, 5, 4096, 576, 64), (3, 700, 32, 512, 32),
    (128, 4, 32, 576, 16), (1, 33, 256, 576, 1)])
def test_copy(pools, P, page, dk, block):
    g = torch.Generator(device=DEV)
    g.manual_seed(P)
    r = random.Random(P)
    kv, sc = make_pools(g, pools, P, page, dk, block)
    some = r.sample(range(P), P // 2 * 2)
    half = len(some) // 2
    pairs = [[r.choice(some[:half]), d] if r.random() < 0.7 else [-1, -1] for d in some[half:]]
    pairs += [[-1, 0], [0, -1], [P, 0], [0, P], [(1 << 31) - 1, -(1 << 31)]]
    want = [x.clone() for x in kv + sc]
    for a, b in pairs:
        if 0 <= a < P and 0 <= b < P:
            for x in want:
                x[b] = x[a]
    if pools == 2:  # e4m3 as well as codes
        kv = [x.view(torch.float8_e4m3fn) for x in kv]
    dcp.mla_cache8_pages_copy(kv, sc, ints(pairs, len(pairs), 2))
    for x, y in zip(kv + sc, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_copy_past_32_bits():
    """Pages whose bytes lie past 2^32."""
    P, page = 130000, 64
    kv = torch.zeros((P, page, 576), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((P, 1), device=DEV)
    kv[P - 1], sc[P - 1] = 7, 3.0
    kv[5], sc[5] = 9, 4.0
    dcp.mla_cache8_pages_copy([kv], [sc], ints([[P - 1, 0], [5, P - 2]], 2, 2))
    assert bool((kv[0] == 7).all()) and bool((kv[P - 2] == 9).all())
    assert sc[0] == 3 and sc[P - 2] == 4 and int(kv[1:5].sum()) == 0 and int(kv[P - 3].sum()) == 0


def test_update_and_copy_in_a_graph_on_another_stream():
    """A captured step, replayed: each replay goes on from the state that the last one left."""
    r = random.Random(9)
    B, M, P, page = 6, 8, 64, 32
    tables, refs = make_tables(r, B, M, P, 0.4)
    parents, keeps = [0, 0, 2, 2, 4, -1], [33, 33, 40, 41, 64, 0]
    wants = [k + 1 for k in keeps]
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    kv, sc = make_pools(g, 2, P, page, 576, 16)
    plain = [x.clone() for x in kv + sc]
    t, f = ints(tables, B, M), ints(refs)
    rows = [ints(x, B) for x in (parents, keeps, wants)]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        _, _, copies, missing = dcp.mla_cache8_pages_update(t, f, *rows, page=page)
        dcp.mla_cache8_pages_copy(kv, sc, copies)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        tables, refs, pairs, short = ref.update(tables, refs, parents, keeps, wants, page)
        for a, b in pairs:
            if a >= 0:
                for x in plain:
                    x[b] = x[a]
        assert t.tolist() == tables and f.tolist() == refs and copies.tolist() == pairs and missing.tolist() == [short]
    for x, y in zip(kv + sc, plain):
        assert torch.equal(x, y)


# ---- tokens in pages ------------------------------------------------------------------


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def make_paged(g, cp, B, M, page, dk, block, spare=3):
    """Pools of finite codes, with tables of distinct pages in random order."""
    P = B * M + spare
    kv = [(randn(g, P, page, dk) * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(cp)]
    sc = [torch.exp2(torch.randint(-8, 3, (P, page // block), generator=g, device=DEV).float()) for _ in range(cp)]
    tb = [torch.randperm(P, generator=g, device=DEV)[:B * M].view(B, M).int() for _ in range(cp)]
    return kv, sc, tb


def as_rows(kv, sc, tb):
    """The same rows, one after the other."""
    rows = [c.view(torch.uint8)[t.long()].flatten(1, 2) for c, t in zip(kv, tb)]
    return [r.view(torch.float8_e4m3fn) for r in rows], [s[t.long()].flatten(1, 2) for s, t in zip(sc, tb)]


APPENDS = [
    # B, counts, starts, cp, interleave, block, page, M, dk, dtype
    (1, [1], [0], 1, 1, 1, 32, 1, 576, torch.bfloat16),
    (1, [1], [31], 1, 1, 32, 32, 2, 576, torch.bfloat16),
    (3, [4, 0, 90], [60, 5, 0], 1, 1, 1, 32, 4, 576, torch.float16),
    (3, [4, 0, 90], [60, 5, 0], 1, 1, 16, 64, 2, 576, torch.bfloat16),
    (2, [131, 64], [1, 127], 1, 1, 128, 128, 2, 512, torch.bfloat16),
    (4, [300, 17, 1, 200], [13, 100, 255, 0], 4, 16, 64, 64, 2, 576, torch.bfloat16),
    (3, [90, 5, 0], [13, 44, 7], 3, 5, 2, 32, 2, 576, torch.bfloat16),
    (2, [50, 60], [100, 30], 1, 1, 8, 64, 2, 576, torch.bfloat16),  # past the last page
    (2, [5000, 17], [60, 5000], 1, 1, 64, 4096, 2, 576, torch.bfloat16),
    (700, None, None, 1, 1, 16, 32, 3, 512, torch.bfloat16),
    (300, None, None, 2, 1, 32, 64, 2, 576, torch.float16),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"B{c[0]}cp{c[3]}i{c[4]}b{c[5]}p{c[6]}M{c[7]}d{c[8]}")
def test_paged_append_and_read_are_those_of_the_rows(case):
    """The contiguous forms have tests against 64 bits; over pages the same codes, scales and numbers, and no page is
    touched besides."""
    B, counts, starts, cp, il, block, page, M, dk, dtype = case
    r = random.Random(B)
    counts = counts or [r.choice([0, 1, 2, 7, 40]) for _ in range(B)]
    starts = starts or [r.randrange(M * page * cp - 40) for _ in range(B)]
    g = torch.Generator(device=DEV)
    g.manual_seed(B + page)
    n = sum(counts)
    kv, sc, tb = make_paged(g, cp, B, M, page, dk, block)
    if cp == 3:  # a shard that is not held
        kv[1] = sc[1] = tb[1] = None
    held = [j for j in range(cp) if kv[j] is not None]
    pick = lambda x: [x[j] for j in held]
    rows, rscales = as_rows(pick(kv), pick(sc), pick(tb))
    full = lambda x: [x[held.index(j)] if j in held else None for j in range(cp)]
    rows, rscales = full(rows), full(rscales)
    before = [None if c is None else c.view(torch.uint8).clone() for c in kv]
    latent = (randn(g, n + 1, 512) * torch.exp2(torch.randint(-9, 9, (n + 1, 1), generator=g, device=DEV).float())).to(dtype)
    rope = randn(g, n + 1, 64).to(dtype) if dk == 576 else None
    inv_freq = dcp.mla_rope_inv_freq(64)[0] if dk == 576 else None
    cu = ints([0] + counts).cumsum(0).int()
    lens = ints(starts)
    kw = dict(cu_new=cu, block=block, interleave=il, inv_freq=inv_freq, mscale=1.25)
    dcp.mla_cache8_append(latent, rope, rows, rscales, lens, **kw)
    dcp.mla_cache8_append(latent, rope, kv, sc, lens, tables=tb, **kw)
    got, gscales = as_rows(pick(kv), pick(sc), pick(tb))
    for a, b, c, d in zip(got, pick(rows), gscales, pick(rscales)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(c, d)
    for j in held:
        spare = torch.ones((kv[j].shape[0],), dtype=torch.bool, device=DEV)
        spare[tb[j].long().flatten()] = False
        assert torch.equal(kv[j].view(torch.uint8)[spare], before[j][spare])
    for out_dtype in (torch.bfloat16, torch.float16, torch.float32):
        a, b = (torch.full((n + 1, dk), 7.0, dtype=out_dtype, device=DEV) for _ in range(2))
        kw = dict(starts=lens, cu=cu, block=block, interleave=il)
        dcp.mla_cache8_read(rows, rscales, n + 1, out=a, **kw)
        dcp.mla_cache8_read(kv, sc, n + 1, out=b, tables=tb, **kw)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("block", [1, 16])
def test_tokens_without_a_page(block):
    """They are not written and not read; entries that are no page may be any number."""
    g = torch.Generator(device=DEV)
    g.manual_seed(block)
    page, dk = 32, 576
    kv, sc, _ = make_paged(g, 1, 1, 4, page, dk, block, 0)
    tb = [ints([[2, -1, 0, 4], [1 << 30, 1, -(1 << 31), 3]], 2, 4)]
    n = 2 * 128
    latent, rope = randn(g, n, 512).bfloat16(), randn(g, n, 64).bfloat16()
    lens = ints([0, 0])
    dcp.mla_cache8_append(latent, rope, kv, sc, lens, block=block, tables=tb)
    out = torch.full((n, dk), 7.0, device=DEV)
    dcp.mla_cache8_read(kv, sc, n, block=block, out=out, tables=tb)
    x = torch.cat((latent, rope), 1).double().view(2, 4, page, dk)
    got = out.double().view(2, 4, page, dk)
    for b, i in ((0, 0), (0, 2), (1, 1), (1, 3)):
        # half a step of e4m3, or of its subnormals (2^-10 of a scale that is at most 2 / 448 of a block's peak)
        peak = x[b, i].abs().amax()
        assert ((got[b, i] - x[b, i]).abs() <= torch.maximum(2.0 ** -4 * x[b, i].abs(), 2.0 ** -10 * peak * 2 / 448)).all()
    for b, i in ((0, 1), (0, 3), (1, 0), (1, 2)):
        assert (got[b, i] == 7).all()


def test_pages_past_32_bits():
    """Tokens whose bytes, and whose numbers, lie far into a pool of 8 GB."""
    P, page = 230000, 64
    kv = [torch.zeros((P, page, 576), dtype=torch.uint8, device=DEV)]
    sc = [torch.ones((P, 1), device=DEV)]
    tb = [ints([[P - 1, 116509], [3, P - 2]], 2, 2)]
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    latent, rope = randn(g, 200, 512).bfloat16(), randn(g, 200, 64).bfloat16()
    dcp.mla_cache8_append(latent, rope, kv, sc, ints([0, 20]), block=64, tables=tb)
    got = dcp.mla_cache8_read(kv, sc, 200, starts=ints([0, 20]), block=64, tables=tb, dtype=torch.float32).double()
    x = torch.cat((latent, rope), 1).double()
    # half a step of e4m3, or of its subnormals: 2^-10 of the block's scale, which is the one that 5 sigma need or, where
    # row 1 begins inside a block that holds tokens, the 1 that stands there (a scale never shrinks)
    assert ((got - x).abs() <= torch.clamp(2.0 ** -4 * x.abs(), min=2.0 ** -10)).all()
    touched = kv[0].view(P, -1).any(1).nonzero()[:, 0].tolist()
    assert touched == [3, 116509, P - 2, P - 1]


# ---- attention over pages ----------------------------------------------------------------
# The tolerances are those of test_gpu_cache8.py (derived there): the kernel is the same one, and how a row is cut into
# segments, and whether some of them are of a prefix, changes the order of fp32 sums only.

SCALE = 192 ** -0.5


def make_pool(g, P, page, dk, block):
    x = randn(g, P, page, dk) * torch.exp(0.4 * randn(g, P, page, 1))
    s = torch.exp2(torch.randint(-8, -6, (P, page // block), generator=g, device=DEV).float())
    s = s * (1 + 0.5 * torch.rand((P, page // block), generator=g, device=DEV))  # not only powers of two
    return (x / s.repeat_interleave(block, 1)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


def check_paged(q, kv, sc, tb, lens, cp, il, block, window, sinks, out, lse, base_e=True, held=None, rows=None,
                scale=SCALE):
    """Each row's visible tokens that have a page, one after the other, as a cache of one row and one shard."""
    P, page, dk = next(c.shape for c in kv if c is not None)
    for b in (range(q.shape[0]) if rows is None else rows):
        toks = []
        for p in cache8.visible(max(int(lens[b]), 0), window, sinks):
            j, t = cache8.place(p, cp, il)
            if (held is None or j in held) and t < tb[j].shape[1] * page:
                toks.append((j, t))
        codes, us = torch.zeros((0, dk), device=DEV), torch.zeros((0,), device=DEV)
        if toks:
            j, t = torch.tensor(toks, device=DEV).T
            parts, scales = [], []
            for k in range(cp):
                at = t[j == k]
                if not len(at):
                    continue
                e = tb[k][b, at // page].long()
                ok = (e >= 0) & (e < P)
                parts.append(kv[k][e[ok], at[ok] % page].float())
                scales.append(sc[k][e[ok], at[ok] % page // block])
            codes, us = torch.cat(parts), torch.cat(scales)
        n = codes.shape[0]
        check_decode(q[b:b + 1], [codes[None]], [us[None]], [n], scale, 1, 1, 1, 0, 0, out[b:b + 1], lse[b:b + 1],
                     base_e)


DECODES = [
    # H, dk, cp, interleave, block, page, M, lengths, window, sinks
    (16, 576, 1, 1, 1, 32, 1, [1, 0, 32], 0, 0),
    (16, 576, 1, 1, 1, 32, 7, [0, 1, 31, 32, 33, 127, 128, 129, 199, 224], 0, 0),
    (64, 576, 1, 1, 1, 64, 5, [0, 1, 127, 128, 129, 256, 257, 300], 0, 0),
    (32, 576, 1, 1, 16, 64, 5, [0, 5, 128, 299], 0, 0),
    (128, 576, 1, 1, 64, 128, 9, [1030, 0, 999, 64], 0, 0),
    (128, 512, 1, 1, 1, 256, 3, [700, 3, 513], 0, 0),
    (16, 512, 1, 1, 128, 1024, 1, [700, 3, 513], 0, 0),
    (32, 512, 2, 1, 4, 64, 5, [600, 3, 513], 0, 0),
    (8, 576, 2, 16, 16, 64, 3, [259, 100, 16, 17], 0, 0),
    (24, 576, 4, 1, 1, 32, 3, [360, 1, 2, 3, 0], 0, 0),
    (65, 576, 3, 7, 8, 64, 5, [700, 41], 0, 0),
    (48, 576, 16, 1, 2, 32, 2, [640, 7, 600], 0, 0),
    (64, 576, 1, 1, 1, 64, 8, [500, 130, 129, 100, 0], 128, 0),
    (64, 576, 1, 1, 1, 32, 30, [900, 600, 40], 300, 4),
    (16, 576, 1, 1, 16, 128, 8, [900, 600, 404, 403], 400, 3),
    (128, 576, 2, 1, 1, 64, 8, [1000, 700, 9], 333, 8),
    (32, 576, 4, 16, 32, 32, 10, [1200, 900, 77, 0], 100, 130),
    (64, 512, 1, 1, 1, 64, 11, [700, 640], 1, 0),
    (64, 576, 1, 1, 1, 64, 11, [700, 640], 5, 1000),
    (64, 576, 1, 1, 1, 512, 2, [900, 640], 130, 131),
    (16, 576, 1, 1, 1, 64, 8, [10000, -5, 499], 0, 0),  # beyond the table, negative
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"H{c[0]}d{c[1]}cp{c[2]}i{c[3]}b{c[4]}p{c[5]}M{c[6]}w{c[8]}s{c[9]}")
def test_paged_decode(case):
    H, dk, cp, il, block, page, M, lengths, window, sinks = case
    g = torch.Generator(device=DEV)
    g.manual_seed(H + M + window)
    B = len(lengths)
    P = B * M + 2
    kv, sc = map(list, zip(*[make_pool(g, P, page, dk, block) for _ in range(cp)]))
    tb = [torch.randperm(P, generator=g, device=DEV)[:B * M].view(B, M).int() for _ in range(cp)]
    q = randn(g, B, H, dk).bfloat16()
    lens = ints(lengths)
    # what no row sees may hold anything: NaN codes, NaN scales where a whole block is unseen, entries that are no page
    for j in range(cp):
        seen = torch.zeros((P, page), dtype=torch.bool, device=DEV)
        for b, n in enumerate(lengths):
            for p in cache8.visible(max(n, 0), window, sinks):
                k, t = cache8.place(p, cp, il)
                if k == j and t < M * page:
                    seen[int(tb[j][b, t // page]), t % page] = True
        kv[j].view(torch.uint8)[~seen] = 0x7F
        sc[j][~seen.view(P, -1, block).any(2)] = float("nan")
        used = seen.any(1)[tb[j].long()]
        tb[j] = torch.where(used, tb[j], torch.randint(-2, 2, (B, M), generator=g, device=DEV).int() * (1 << 29))
    kw = dict(block=block, interleave=il, window=window, sinks=sinks, lse_base_e=H % 3 != 0)
    status = torch.zeros((1,), dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, tables=tb, status=status, **kw)
    assert int(status) == 0
    check_paged(q, kv, sc, tb, lens, cp, il, block, window, sinks, out, lse, kw["lse_base_e"])
    again = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, tables=tb, flags=dcp.DCP_FLAG_PDL, **kw)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("H,B,M,page,cp", [(16, 1, 700, 64, 1), (128, 1, 200, 64, 1), (64, 2, 70, 128, 2),
                                           (128, 37, 6, 128, 1), (32, 600, 13, 32, 1)])
def test_paged_decode_is_that_of_the_rows(H, B, M, page, cp):
    """Bit for bit, where tiles begin at the same tokens (no window)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    P = B * M + 1
    kv, sc = map(list, zip(*[make_pool(g, P, page, 576, 16) for _ in range(cp)]))
    tb = [torch.randperm(P, generator=g, device=DEV)[:B * M].view(B, M).int() for _ in range(cp)]
    rows, rscales = as_rows(kv, sc, tb)
    q = randn(g, B, H, 576).bfloat16()
    lens = (torch.rand((B,), generator=g, device=DEV) * cp * M * page).int()
    lens[0] = cp * M * page
    a = dcp.mla_cache8_decode(q, rows, rscales, lens, SCALE, block=16)
    b = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=16, tables=tb)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("loud", [1.0, 40.0])
def test_paged_decode_of_tokens_without_a_page(H, page, loud):
    """Anywhere in a row: its first tiles, its last, all of them, a few. (Loud keys give scores far from zero.)"""
    g = torch.Generator(device=DEV)
    g.manual_seed(H + page)
    n = 1024
    M, B = n // page, 8
    P = B * M
    kv, sc = make_pool(g, P, page, 576, 1)
    sc *= loud
    tb = torch.randperm(P, generator=g, device=DEV).view(B, M).int()
    slot = torch.arange(M, device=DEV)
    bad = torch.rand((B, M), generator=g, device=DEV) < 0.4
    bad[0] = slot < M - 1          # the last page alone
    bad[1] = slot >= 1             # the first alone
    bad[2] = True
    bad[3] = (slot * page >= 200) & (slot * page < 700)
    bad[4] = False
    bad[5, :max(1, 512 // page)] = True
    tb = torch.where(bad, ints([-1, P, 1 << 30, -(1 << 31)])[torch.randint(0, 4, (B, M), generator=g, device=DEV)], tb)
    q = randn(g, B, H, 576).bfloat16()
    lens = ints([n, n - 3, n, 1000, n, n, 900, 40])
    for kw in ({}, dict(window=300, sinks=5)):
        out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, tables=[tb], **kw)
        check_paged(q, [kv], [sc], [tb], lens, 1, 1, 1, kw.get("window", 0), kw.get("sinks", 0), out, lse)
        assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()
    groups, shared = dcp.mla_cache8_groups([B], [512])
    same = roomy(tb, 1, page)
    same[:, :512 // page] = tb[5, :512 // page]
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, tables=[same], groups=groups, shared=shared)
    check_paged(q, [kv], [sc], [same], lens, 1, 1, 1, 0, 0, out, lse)


def roomy(t, cp, page):
    """Tables with room for the 1024 tiles from which on groups are used: entries of -1 behind the others."""
    B, M = t.shape
    more = max(0, -(-1024 * 128 // (B * cp * page)) - M)
    return torch.cat((t, torch.full((B, more), -1, dtype=torch.int32, device=DEV)), 1)


GROUPS = [
    # H, cp, interleave, block, page, rows of the groups, their shared positions, most tokens of a row's own
    (16, 1, 1, 1, 64, [2], [128], 1),
    (16, 1, 1, 1, 64, [4], [1000], 300),
    (16, 1, 1, 64, 64, [9, 1, 3], [1500, 700, 129], 200),
    (16, 1, 1, 1, 32, [1, 1, 1, 1], [300, 0, 400, 128], 100),
    (8, 1, 1, 1, 64, [20], [640], 130),
    (1, 1, 1, 1, 64, [70], [513], 20),
    (40, 1, 1, 1, 128, [5, 2], [900, 1111], 500),
    (100, 1, 1, 16, 64, [3, 6], [777, 640], 150),
    (24, 2, 1, 1, 64, [4, 3], [1000, 300], 100),
    (16, 4, 16, 16, 32, [6], [3000], 70),
    (48, 3, 5, 1, 64, [2, 2, 4], [500, 2000, 100], 90),
    (16, 1, 1, 1, 64, [2] * 20, [256] * 20, 300),
    (12, 1, 1, 1, 64, [3, 1] * 90, [256, 0] * 90, 150),
    (32, 1, 1, 1, 256, [300], [384], 64),
    (64, 1, 1, 1, 64, [3], [600], 100),      # (groups make no difference)
    (20, 1, 1, 1, 64, [3, 4], [100, 127], 300),  # shorter than a tile
    (16, 1, 1, 1, 64, [6], [1 << 30], 300),  # beyond every row
    (16, 16, 1, 1, 32, [5], [4000], 300),
]


@pytest.mark.parametrize("case,dk", [(c, 576) for c in GROUPS] + [(c, 512) for c in GROUPS if c[0] in (16, 40, 100)],
                         ids=lambda c: c if isinstance(c, int) else
                         f"H{c[0]}cp{c[1]}i{c[2]}b{c[3]}p{c[4]}g{len(c[5])}n{sum(c[5])}s{c[6][0]}")
def test_groups(case, dk):
    """Rows behind shared prefixes; among them rows of nothing of their own, of no token, and shorter than the prefix
    (with pages of their own)."""
    H, cp, il, block, page, counts, shared, most = case
    B = sum(counts)
    r = random.Random(B + H)
    lens, first, alone = [], [], []
    for n, s in zip(counts, shared):
        f = len(lens)
        for i in range(n):
            base = s if s < 1 << 29 else 400
            kind = r.random() if n > 2 else 1.0
            cut = kind < 0.12 and s < 1 << 29
            lens.append(r.randint(0, max(base - 1, 0)) if cut else base + (0 if kind < 0.25 else r.randint(1, most)))
            first.append(f)
            alone.append(cut)
    g = torch.Generator(device=DEV)
    g.manual_seed(B * H)
    M = -(-(max(lens) // (cp * il) + 1) * il // page) + 1
    P = B * M + 1
    kv, sc = map(list, zip(*[make_pool(g, P, page, dk, block) for _ in range(cp)]))
    tb = [torch.randperm(P, generator=g, device=DEV)[:B * M].view(B, M).int() for _ in range(cp)]
    tb = [roomy(t, cp, page) for t in tb]
    for j in range(cp):
        for b in range(B):
            s = shared[[b >= sum(counts[:k]) and b < sum(counts[:k + 1]) for k in range(len(counts))].index(True)]
            if b == first[b] or alone[b] or s >= 1 << 29:
                continue
            have = ref.share(s, cp, j, il)
            whole = have // page
            tb[j][b, :whole] = tb[j][first[b], :whole]
            if have % page:  # the page that the prefix ends in: a copy, as the step of the tables leaves it
                a, z = int(tb[j][first[b], whole]), int(tb[j][b, whole])
                n = have % page
                kv[j].view(torch.uint8)[z, :n] = kv[j].view(torch.uint8)[a, :n]
                sc[j][z, :-(-n // block)] = sc[j][a, :-(-n // block)]
    q = randn(g, B, H, dk).bfloat16()
    n = ints(lens)
    groups, common = dcp.mla_cache8_groups(counts, shared)
    kw = dict(block=block, interleave=il, lse_base_e=H % 3 != 0, tables=tb)
    status = torch.zeros((1,), dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, kv, sc, n, SCALE, groups=groups, shared=common, status=status, **kw)
    assert int(status) == 0
    check_paged(q, kv, sc, tb, n, cp, il, block, 0, 0, out, lse, kw["lse_base_e"],
                rows=range(B) if B < 60 else list(range(0, B, 7)) + [B - 1])
    plain = dcp.mla_cache8_decode(q, kv, sc, n, SCALE, **kw)
    # two results within 2^-8 of one value each, and the sums' orders
    assert ((out.float() - plain[0].float()).abs() <= 2.0 ** -6 * plain[0].float().abs().amax(-1, keepdim=True)).all()
    if H % 64 == 0:
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    again = dcp.mla_cache8_decode(q, kv, sc, n, SCALE, groups=groups, shared=common, flags=dcp.DCP_FLAG_PDL, **kw)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_groups_of_a_long_prefix():
    """Prefixes that are cut over many CTAs, offset by one long row alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    H, page, counts, shared = 16, 64, [30, 1, 33], [12000, 0, 7000]
    B = sum(counts)
    own = torch.randint(1, 400, (B,), generator=g, device=DEV).tolist()
    own[30] = 20000
    lens = [s + own[i] for i, s in enumerate([12000] * 30 + [0] + [7000] * 33)]
    M = -(-20000 // page)
    P = 2 * M + B * 8
    kv, sc = make_pool(g, P + 320, page, 576, 64)
    free = iter(torch.randperm(P + 320, generator=g, device=DEV).tolist())
    take = lambda n: [next(free) for _ in range(n)]
    heads = {0: take(12000 // page), 30: take(M), 31: take(7000 // page)}
    tb = []
    for i in range(B):
        row = list(heads[0 if i < 30 else 30 if i == 30 else 31])
        row += take(-(-lens[i] // page) - len(row))
        tb.append(row + [-1] * (M - len(row)))
    # (a page of the prefix's last, partial page is the row's own, with tokens of its own: shared ends at whole pages)
    groups, common = dcp.mla_cache8_groups(counts, [s // page * page for s in shared])
    q, n, tb = randn(g, B, H, 576).bfloat16(), ints(lens), [ints(tb, B, M)]
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], n, SCALE, block=64, tables=tb, groups=groups, shared=common)
    check_paged(q, [kv], [sc], tb, n, 1, 1, 64, 0, 0, out, lse, rows=[0, 1, 7, 29, 30, 31, 40, 63])


def test_groups_that_break_the_rules_read_nothing_out_of_place():
    """Whatever stands in groups and shared, rows that are grouped rightly keep their results."""
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    B, M, page, H = 12, 8, 64, 16
    P = B * M
    kv, sc = make_pool(g, P, page, 576, 1)
    tb = roomy(torch.randperm(P, generator=g, device=DEV).view(B, M).int(), 1, page)
    tb[1:4, :4] = tb[0, :4]
    q, lens = randn(g, B, H, 576).bfloat16(), ints([400, 300, 256, 500, 100, 512, 0, 17, 129, 300, 64, 511])
    groups, shared = dcp.mla_cache8_groups([4] + [1] * 8, [256] + [0] * 8)
    for b, (first, count, common) in enumerate([(-1, 9, 200), (3, 4, 100), (4, 100, 256), (1 << 30, 2, 128),
                                                (4, -5, 300), (-(1 << 31), 1 << 30, 256), (11, 3, 999),
                                                ((1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1)], start=4):
        groups[b, 0], groups[b, 1], shared[b] = first, count, common
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, tables=[tb], groups=groups, shared=shared)
    check_paged(q, [kv], [sc], [tb], lens, 1, 1, 1, 0, 0, out, lse, rows=range(4))


def test_paged_decode_partials_of_shards_merge_to_the_whole():
    """Each shard alone, with a prefix, then the merge: the whole."""
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    cp, B, H, page, M = 4, 6, 16, 64, 4
    kv, sc = map(list, zip(*[make_pool(g, B * M, page, 576, 1) for _ in range(cp)]))
    tb = [roomy(torch.randperm(B * M, generator=g, device=DEV).view(B, M).int(), cp, page) for _ in range(cp)]
    for t in tb:
        t[1:, :2] = t[0, :2]
    q, lens = randn(g, B, H, 576).bfloat16(), ints([600, 512, 1000, 700, 513, 3])
    groups, shared = dcp.mla_cache8_groups([B], [512])
    kw = dict(groups=groups, shared=shared)
    whole, wl = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, tables=tb, **kw)
    check_paged(q, kv, sc, tb, lens, cp, 1, 1, 0, 0, whole, wl)
    srcs, lses = [], []
    for j in range(cp):
        only = lambda x: [x[k] if k == j else None for k in range(cp)]
        o, l = dcp.mla_cache8_decode(q, only(kv), only(sc), lens, SCALE, tables=only(tb), **kw)
        check_paged(q, kv, sc, tb, lens, cp, 1, 1, 0, 0, o, l, held=[j])
        srcs.append(o)
        lses.append(l)
    outs, louts = dcp.merge(srcs, lses, True, seq_lens=lens)
    # each partial is rounded to bf16 (2^-9 of itself), and so is the merged one
    merged = torch.cat(outs, 1).double()
    size = torch.stack(srcs).double().abs().amax(0)
    assert ((merged - whole.double()).abs() <= 2.0 ** -7 * torch.maximum(size, whole.double().abs())).all()
    assert ((torch.cat(louts, 1) - wl).abs() <= 1e-4).all()


def test_a_serving_run():
    """Prompt, fork, decode steps in a captured graph, an end, a compaction: every step's attention against 64 bits over
    what the tables say, and the tables against the plain form."""
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    B, M, P, page, H, block = 6, 360, 60, 64, 16, 16  # (room for 1024 tiles: groups are used)
    tables, refs = [[-1] * M for _ in range(B)], [0] * P
    t, f = ints(tables, B, M), ints(refs)
    kv = torch.zeros((P, page, 576), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    sc = torch.ones((P, page // block), device=DEV)
    inv_freq, _ = dcp.mla_rope_inv_freq(64)
    rows = [ints([0] * B) for _ in range(3)]

    def plan(parents, keeps, wants):
        nonlocal tables, refs
        for x, y in zip(rows, (parents, keeps, wants)):
            x.copy_(ints(y))
        tables, refs, _, short = ref.update(tables, refs, parents, keeps, wants, page)
        assert short == 0

    def step():
        _, _, copies, missing = dcp.mla_cache8_pages_update(t, f, *rows, page=page)
        dcp.mla_cache8_pages_copy([kv], [sc], copies)
        return missing

    # a prompt of 300 tokens in row 0, one of 77 in row 4
    plan(list(range(B)), [0] * B, [300, 0, 0, 0, 77, 0])
    step()
    latent, rope = randn(g, 377, 512).bfloat16(), randn(g, 377, 64).bfloat16()
    dcp.mla_cache8_append(latent, rope, [kv], [sc], ints([0] * B), cu_new=ints([0, 300, 300, 300, 300, 377, 377]),
                          block=block, inv_freq=inv_freq, tables=[t])
    # rows 0 to 3 go on from row 0, each with tokens of its own; row 5 from row 4
    lens = [300, 300, 300, 300, 77, 77]
    n = ints(lens)
    groups, shared = dcp.mla_cache8_groups([4, 2], [300, 77])
    q = torch.empty((B, H, 576), dtype=torch.bfloat16, device=DEV)
    new, pe = torch.empty((B, 512), dtype=torch.bfloat16, device=DEV), torch.empty((B, 64), dtype=torch.bfloat16, device=DEV)
    plan([0, 0, 0, 0, 4, 4], lens, [x + 1 for x in lens])
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        missing = step()
        dcp.mla_rope(q[..., 512:], n, inv_freq, out=q[..., 512:])
        dcp.mla_cache8_append(new, pe, [kv], [sc], n, block=block, inv_freq=inv_freq, tables=[t])
        n.add_(1)
        out, lse = dcp.mla_cache8_decode(q, [kv], [sc], n, SCALE, block=block, tables=[t], groups=groups, shared=shared)
    for i in range(70):
        q.copy_(randn(g, B, H, 576))
        new.copy_(randn(g, B, 512))
        pe.copy_(randn(g, B, 64))
        if i:
            plan(list(range(B)), lens, [x + 1 for x in lens])
        graph.replay()
        torch.cuda.synchronize()
        lens = [x + 1 for x in lens]
        assert t.tolist() == tables and f.tolist() == refs and n.tolist() == lens and int(missing) == 0
        if i % 23 == 0 or i == 69:
            check_paged(q, [kv], [sc], [t], n, 1, 1, block, 0, 0, out, lse)
    # rows 0 and 3 end, and the pool shrinks to what is in use
    plan([-1, 1, 2, -1, 4, 5], lens, [0 if b in (0, 3) else x for b, x in enumerate(lens)])
    step()
    before = dcp.mla_cache8_decode(q, [kv], [sc], n, SCALE, block=block, tables=[t])
    _, _, copies = dcp.mla_cache8_pages_compact(t, f)
    dcp.mla_cache8_pages_copy([kv], [sc], copies)
    tables, refs, _ = ref.compact(tables, refs)
    assert t.tolist() == tables and f.tolist() == refs
    used = sum(r > 0 for r in refs)
    assert max(max(r) for r in tables) == used - 1
    after = dcp.mla_cache8_decode(q, [kv[:used]], [sc[:used]], n, SCALE, block=block, tables=[t])
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert (after[0][0] == 0).all() and (after[1][3] == -float("inf")).all()


@pytest.mark.parametrize("B,H,M,grouped", [(1, 16, 3, False), (8, 16, 40, True), (8, 128, 40, False)])
def test_paged_decode_after_waits_that_gave_up(B, H, M, grouped):
    """As for the rows: a wait that runs out sets the status, and the next call is right."""
    g = torch.Generator(device=DEV)
    g.manual_seed(B)
    page = 64
    kv, sc = make_pool(g, B * M, page, 576, 1)
    tb = [torch.randperm(B * M, generator=g, device=DEV).view(B, M).int()]
    if grouped:
        tb = [roomy(tb[0], 1, page)]
        tb[0][1:, :8] = tb[0][0, :8]
    q = randn(g, B, H, 576).bfloat16()
    lens = torch.full((B,), M * page - 5, dtype=torch.int32, device=DEV)
    groups, shared = dcp.mla_cache8_groups([B], [512])
    kw = dict(groups=groups, shared=shared) if grouped else {}
    status = torch.zeros((1,), dtype=torch.int32, device=DEV)
    dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, tables=tb, status=status, flags=dcp.DCP_MLA_FLAG_TEST_STALL, **kw)
    torch.cuda.synchronize()
    assert int(status) == 1
    status.zero_()
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, tables=tb, status=status, **kw)
    check_paged(q, [kv], [sc], tb, lens, 1, 1, 1, 0, 0, out, lse, rows=[0, B - 1])
    assert int(status) == 0


def test_paged_decode_far_into_a_pool():
    """Pages whose bytes lie past 2^32 and past 2^33."""
    P, page = 240000, 64
    kv = torch.zeros((P, page, 576), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    sc = torch.zeros((P, page // 16), device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    at = [P - 1, 116509, 3, 233017, 120000, P - 7]
    x, s = make_pool(g, len(at), page, 576, 16)
    for i, e in enumerate(at):
        kv.view(torch.uint8)[e], sc[e] = x.view(torch.uint8)[i], s[i]
    tb = [ints([[P - 1, 116509, 3], [233017, 120000, P - 7]], 2, 3)]
    q, lens = randn(g, 2, 16, 576).bfloat16(), ints([190, 180])
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, block=16, tables=tb)
    check_paged(q, [kv], [sc], tb, lens, 1, 1, 16, 0, 0, out, lse)


def test_paged_calls_of_no_rows():
    kv, sc = torch.zeros((4, 64, 576), dtype=torch.uint8, device=DEV), torch.ones((4, 64), device=DEV)
    none, zero = torch.empty((0,), dtype=torch.int32, device=DEV), ints([0])
    tb = [torch.empty((0, 3), dtype=torch.int32, device=DEV)]
    latent, rope = (torch.empty((0, w), dtype=torch.bfloat16, device=DEV) for w in (512, 64))
    dcp.mla_cache8_append(latent, rope, [kv], [sc], none, cu_new=zero, tables=tb)
    assert dcp.mla_cache8_read([kv], [sc], 0, tables=tb).shape == (0, 576)
    q = torch.empty((0, 16, 576), dtype=torch.bfloat16, device=DEV)
    groups, shared = dcp.mla_cache8_groups([], [])
    for kw in ({}, dict(groups=groups, shared=shared)):
        out, lse = dcp.mla_cache8_decode(q, [kv], [sc], none, SCALE, tables=tb, **kw)
        assert out.shape == (0, 16, 512) and lse.shape == (0, 16)


def grouped_batch(g, B, H, prefix, own, page=64, block=1, dk=576):
    """One group behind `prefix` positions (whole pages), with room for groups to be used: pool, tables, q, lengths."""
    M = -(-(prefix + max(own)) // page)
    P = B * M
    kv, sc = make_pool(g, P, page, dk, block)
    tb = roomy(torch.randperm(P, generator=g, device=DEV).view(B, M).int(), 1, page)
    tb[1:, :prefix // page] = tb[0, :prefix // page]
    return kv, sc, tb, randn(g, B, H, dk).bfloat16(), ints([prefix + n for n in own])


def test_groups_take_what_a_call_may_bring():
    """A workspace of just the size, full of NaN; outputs given; q with odd strides; another stream; bits that stay."""
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    B, H = 7, 24
    kv, sc, tb, q, lens = grouped_batch(g, B, H, 640, [1, 0, 130, 200, 127, 128, 300], block=16)
    groups, shared = dcp.mla_cache8_groups([B], [640])
    kw = dict(block=16, tables=[tb], groups=groups, shared=shared)
    want = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, **kw)
    check_paged(q, [kv], [sc], [tb], lens, 1, 1, 16, 0, 0, *want)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    size = dcp.dcp_mla_cache8_decode_paged_workspace_bytes(1, B, H, 64, tb.shape[1], 0, 0, True, sms)
    assert size > dcp.dcp_mla_cache8_decode_paged_workspace_bytes(1, B, H, 64, tb.shape[1], 0, 0, False, sms)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    wide = torch.zeros((B, H + 1, 600), dtype=torch.bfloat16, device=DEV)
    odd = wide[:, 1:, 2:578]  # heads and rows on 4-byte boundaries only
    odd.copy_(q)
    out, lse = torch.full((B, H, 512), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((B, H), 7.0, device=DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = dcp.mla_cache8_decode(odd, [kv], [sc], lens, SCALE, out=out, lse=lse, workspace=ws, stream=stream, **kw)
    stream.synchronize()
    assert got[0] is out and got[1] is lse
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(dcp.DcpError):
        dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, workspace=ws[:size - 256], **kw)


@pytest.mark.parametrize("loud", [(1.0, 30.0), (30.0, 1.0), (0.01, 30.0), (60.0, 60.0)])
def test_groups_whose_prefix_and_rows_lie_far_apart(loud):
    """Scores of the prefix and of the rows' own tokens of very different sizes: the join's weights."""
    g = torch.Generator(device=DEV)
    g.manual_seed(12)
    B, H = 9, 16
    kv, sc, tb, q, lens = grouped_batch(g, B, H, 1280, [300, 5, 0, 129, 64, 1, 200, 256, 17])
    common = tb[0, :20].long()
    sc *= loud[1]
    sc[common] *= loud[0] / loud[1]
    groups, shared = dcp.mla_cache8_groups([B], [1280])
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, tables=[tb], groups=groups, shared=shared)
    check_paged(q, [kv], [sc], [tb], lens, 1, 1, 1, 0, 0, out, lse)


def test_groups_keep_nan_to_its_row_and_head():
    """Heads of several rows stand in one block: a NaN or an infinity in one row's q stays there; one in a token of the
    prefix reaches every row, one behind it its own row alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(13)
    B, H = 6, 16
    kv, sc, tb, q, lens = grouped_batch(g, B, H, 640, [100, 200, 1, 50, 300, 128])
    groups, shared = dcp.mla_cache8_groups([B], [640])
    kw = dict(tables=[tb], groups=groups, shared=shared)
    want = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE, **kw)
    bad = q.clone()
    bad[1, 3, 17], bad[4, 15, 570] = float("nan"), float("inf")
    out, lse = dcp.mla_cache8_decode(bad, [kv], [sc], lens, SCALE, **kw)
    hit = torch.zeros((B, H), dtype=torch.bool, device=DEV)
    hit[1, 3] = hit[4, 15] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
    own = sc.clone()
    own[tb[3, 10].long(), 5] = float("nan")  # position 645 of row 3
    out, lse = dcp.mla_cache8_decode(q, [kv], [own], lens, SCALE, **kw)
    rows = torch.arange(B, device=DEV) == 3
    assert out[rows].isnan().all() and torch.equal(out[~rows], want[0][~rows]) and torch.equal(lse[~rows], want[1][~rows])
    all_ = sc.clone()
    all_[tb[0, 2].long(), 5] = float("nan")  # position 133 of the prefix
    out, lse = dcp.mla_cache8_decode(q, [kv], [all_], lens, SCALE, **kw)
    assert out.isnan().all() and lse.isnan().all()


def test_two_graphs_over_one_workspace_in_turn():
    """Two captured calls that share a workspace, replayed one after the other, in either order."""
    g = torch.Generator(device=DEV)
    g.manual_seed(14)
    B, H = 5, 16
    kv, sc, tb, q, lens = grouped_batch(g, B, H, 640, [100, 200, 1, 50, 300])
    groups, shared = dcp.mla_cache8_groups([B], [640])
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.empty((dcp.dcp_mla_cache8_decode_paged_workspace_bytes(1, B, H, 64, tb.shape[1], 0, 0, True, sms),),
                     dtype=torch.uint8, device=DEV)
    calls = [(q, lens), (randn(g, B, H, 576).bfloat16(), lens - 30)]
    want = [dcp.mla_cache8_decode(a, [kv], [sc], n, SCALE, tables=[tb], groups=groups, shared=shared) for a, n in calls]
    graphs, got = [], []
    for a, n in calls:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(dcp.mla_cache8_decode(a, [kv], [sc], n, SCALE, tables=[tb], groups=groups, shared=shared,
                                             workspace=ws))
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("seed", range(20))
def test_paged_decode_random(seed):
    """Random sizes: heads, shards, blocks, pages, windows or groups, pages that are missing."""
    r = random.Random(seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    H, dk = r.choice([1, 7, 16, 20, 32, 48, 64, 100, 128]), r.choice([576, 576, 512])
    cp, page = r.choice([1, 1, 2, 5]), r.choice([32, 64, 128, 512])
    il, block = r.choice([1, 16, 24]) if cp > 1 else 1, r.choice([1, 8, 32])
    B, M = r.choice([1, 3, 10, 40]), r.randint(1, 6)
    most = min(M * page, 900) * cp
    lens = [r.choice([0, 1, r.randint(0, most), r.randint(0, most), most + 50]) for _ in range(B)]
    P = B * M + 1
    kv, sc = map(list, zip(*[make_pool(g, P, page, dk, block) for _ in range(cp)]))
    tb = [torch.randperm(P, generator=g, device=DEV)[:B * M].view(B, M).int() for _ in range(cp)]
    kw = {}
    window = sinks = 0
    if r.random() < 0.4:
        window, sinks = r.randint(1, most), r.choice([0, 3, 200])
        kw = dict(window=window, sinks=sinks)
    else:
        counts = []
        while sum(counts) < B:
            counts.append(min(r.randint(1, 6), B - sum(counts)))
        common = [r.randint(0, most) // (page * cp * il) * (page * cp * il) for _ in counts]
        groups, shared = dcp.mla_cache8_groups(counts, common)
        tb = [roomy(t, cp, page) for t in tb]
        for b in range(B):
            first, s = int(groups[b, 0]), int(shared[b])
            if lens[b] >= s:
                for j in range(cp):
                    n = ref.share(s, cp, j, il) // page
                    tb[j][b, :n] = tb[j][first, :n]
        kw = dict(groups=groups, shared=shared)
    if r.random() < 0.3:  # (the same entry in every row, so that prefixes stay common)
        for t in tb:
            t[:, r.randrange(M)] = r.choice([-1, P, 1 << 30])
    q = randn(g, B, H, dk).bfloat16()
    out, lse = dcp.mla_cache8_decode(q, kv, sc, ints(lens), SCALE, block=block, interleave=il, tables=tb, **kw)
    check_paged(q, kv, sc, tb, ints(lens), cp, il, block, window, sinks, out, lse)
