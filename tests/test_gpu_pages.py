"""The paged cache's operators on the GPU against their plain forms (oracle/pages.py, oracle/cache8.py). Tables, counts
and copied bytes are whole numbers and have to be equal."""
import random

import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
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
