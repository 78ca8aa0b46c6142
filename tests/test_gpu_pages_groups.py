"""Groups of rows over pages whose first rows have ended or have been cut back: the rows that go on keep their prefix."""
import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from .test_gpu_pages import DEV, SCALE, check_paged, ints, make_pool, randn, roomy

pytestmark = pytest.mark.gpu


def make_group(g, B, H, cp, page, prefix, own, block=1):
    """One group behind `prefix` positions (whole pages of each shard): pools, tables, q, lengths."""
    share = prefix // cp
    assert share % page == 0
    M = -(-(prefix + max(own)) // (cp * page)) + 1
    P = B * M
    kv, sc = map(list, zip(*[make_pool(g, P, page, 576, block) for _ in range(cp)]))
    tb = [torch.randperm(P, generator=g, device=DEV).view(B, M).int() for _ in range(cp)]
    for t in tb:
        t[1:, :share // page] = t[0, :share // page]
    return kv, sc, [roomy(t, cp, page) for t in tb], randn(g, B, H, 576).bfloat16(), [prefix + n for n in own]


@pytest.mark.parametrize("B,H,cp,page,ended,cut", [
    (5, 16, 1, 64, [0], []),            # the first row has ended
    (5, 16, 1, 64, [], [0]),            # it has been cut back
    (6, 24, 1, 32, [0, 2], [1, 4]),
    (9, 16, 2, 64, [0, 1], [2]),
    (45, 8, 1, 64, list(range(34)), []),  # more than a warp looks at in one turn
    (40, 16, 1, 128, list(range(39)), []),
    (4, 16, 1, 64, [0, 1, 2, 3], []),   # nobody is left
])
def test_a_group_outlives_its_first_rows(B, H, cp, page, ended, cut):
    g = torch.Generator(device=DEV)
    g.manual_seed(B * H + page)
    prefix = 10 * 128 * cp
    kv, sc, tb, q, lens = make_group(g, B, H, cp, page, prefix, [(37 * b) % 300 for b in range(B)])
    # what the step of the tables leaves of a row that has ended, and of one that keeps 100 positions a shard
    for b in ended:
        lens[b] = 0
        for t in tb:
            t[b] = -1
    for b in cut:
        lens[b] = 100 * cp
        for t in tb:
            t[b, -(-100 // page):] = -1
    n = ints(lens)
    groups, shared = dcp.mla_cache8_groups([B], [prefix])
    out, lse = dcp.mla_cache8_decode(q, kv, sc, n, SCALE, tables=tb, groups=groups, shared=shared)
    check_paged(q, kv, sc, tb, n, cp, 1, 1, 0, 0, out, lse)


def test_a_beam_that_ends_in_a_step():
    """Four rows forked from one, the first of which ends in the next step of the tables, in place."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    B, H, page, M, P = 4, 16, 64, 600, 64
    kv, sc = make_pool(g, P, page, 576, 1)
    tables, refs = torch.full((B, M), -1, dtype=torch.int32, device=DEV), torch.zeros(P, dtype=torch.int32, device=DEV)
    update = lambda parents, keeps, wants: dcp.mla_cache8_pages_update(tables, refs, ints(parents), ints(keeps),
                                                                       ints(wants), page=page)
    update([0, -1, -1, -1], [0] * 4, [1300, 0, 0, 0])
    _, _, copies, _ = update([0, 0, 0, 0], [1300] * 4, [1301] * 4)
    dcp.mla_cache8_pages_copy([kv], [sc], copies)
    _, _, copies, missing = update([-1, 1, 2, 3], [0, 1301, 1301, 1301], [0, 1302, 1302, 1302])
    dcp.mla_cache8_pages_copy([kv], [sc], copies)
    assert int(missing) == 0 and (tables[0] == -1).all()
    groups, shared = dcp.mla_cache8_groups([B], [1280])
    q, n = randn(g, B, H, 576).bfloat16(), ints([0, 1302, 1302, 1302])
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], n, SCALE, tables=[tables], groups=groups, shared=shared)
    check_paged(q, [kv], [sc], [tables], n, 1, 1, 1, 0, 0, out, lse)
    assert (out[0] == 0).all() and (out[1:] != 0).any(-1).all()
