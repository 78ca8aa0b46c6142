"""The paged cache's operators on the GPU against their plain forms (oracle/pages.py, oracle/cache8.py). Tables, counts
and copied bytes are whole numbers and have to be equal."""
import random

import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from oracle import cache8
from oracle import pages as ref

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
