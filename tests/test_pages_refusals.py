"""What the calls on pages refuse, on the host, and what their plain forms (oracle/pages.py) say of small cases that can
be worked out by hand. Nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from decode_context_mla_dcp_gb300 import build as dcp_build
from oracle import pages as ref

A = 1 << 20  # an aligned address that is never dereferenced
NULL, SHAPE, BLOCK, CP, ALIGN = range(-201, -206, -1)
WS, PAGE, ALIAS = -208, -211, -212


@pytest.fixture(scope="module", autouse=True)
def built():
    dcp_build.build()


def refused(code, fn, base, **change):
    with pytest.raises(dcp.DcpError) as e:
        fn(**{**base, **change})
    assert e.value.status == code
    assert dcp.dcp_mla_cache8_strerror(code) in str(e.value)


UPDATE = dict(tables=A, refs=2 * A, parents=A, keeps=A, wants=A, B=4, M=8, P=16, page=64, tables_out=A,
              refs_out=2 * A, copies=A, missing=A, workspace=A, workspace_bytes=1 << 40, stream=0)
COMPACT = dict(tables=A, refs=2 * A, B=4, M=8, P=16, tables_out=A, refs_out=2 * A, copies=A, workspace=A,
               workspace_bytes=1 << 40, stream=0)
COPY = dict(kv_ptrs=[A], scale_ptrs=[2 * A], pools=1, P=16, page=64, Dk=576, block=16, copies=A, n=4, stream=0)

TABLES = [(SHAPE, dict(B=-1)), (SHAPE, dict(B=65536)), (SHAPE, dict(M=0)), (SHAPE, dict(P=0)),
          (SHAPE, dict(P=1 << 31)), (SHAPE, dict(B=65535, M=1 << 15)), (SHAPE, dict(M=1 << 31)),
          (NULL, dict(tables=None)), (NULL, dict(refs=None)), (NULL, dict(tables_out=None)),
          (NULL, dict(refs_out=None)), (NULL, dict(copies=None)), (ALIGN, dict(tables=A + 1)),
          (ALIGN, dict(refs=A + 2)), (ALIGN, dict(copies=A + 4)), (WS, dict(workspace=None)),
          (WS, dict(workspace=A + 128)), (WS, dict(workspace_bytes=100)),
          # one in place and the other not; outputs that overlap inputs or each other
          (ALIAS, dict(tables_out=4 * A)), (ALIAS, dict(refs_out=4 * A)),
          (ALIAS, dict(tables_out=A + 64, refs_out=4 * A)), (ALIAS, dict(tables_out=4 * A, refs_out=2 * A + 32)),
          (ALIAS, dict(tables_out=2 * A, refs_out=4 * A)), (ALIAS, dict(tables_out=4 * A, refs_out=A)),
          (ALIAS, dict(tables_out=4 * A, refs_out=4 * A)), (ALIAS, dict(refs=A, refs_out=A))]


@pytest.mark.parametrize("code,change", TABLES + [
    (PAGE, dict(page=16)), (PAGE, dict(page=48)), (PAGE, dict(page=8192)), (PAGE, dict(page=0)),
    (CP, dict(cp=0)), (CP, dict(cp=17)), (CP, dict(cp=2, shard=2)), (CP, dict(shard=-1)), (CP, dict(interleave=0)),
    (CP, dict(interleave=(1 << 24) + 1)), (NULL, dict(parents=None)), (NULL, dict(keeps=None)),
    (NULL, dict(wants=None)), (NULL, dict(missing=None)), (ALIGN, dict(parents=A + 2)), (ALIGN, dict(missing=A + 2))])
def test_update(code, change):
    refused(code, dcp.dcp_mla_pages_update, UPDATE, **change)


@pytest.mark.parametrize("code,change", TABLES)
def test_compact(code, change):
    refused(code, dcp.dcp_mla_pages_compact, COMPACT, **change)


@pytest.mark.parametrize("code,change", [
    (SHAPE, dict(n=-1)), (SHAPE, dict(n=1 << 31)), (SHAPE, dict(n=1 << 29, page=4096)), (SHAPE, dict(P=0)), (SHAPE, dict(Dk=640)), (SHAPE, dict(pools=0)),
    (SHAPE, dict(pools=129, kv_ptrs=[A] * 129, scale_ptrs=[A] * 129)), (BLOCK, dict(block=3)), (BLOCK, dict(block=0)),
    (BLOCK, dict(block=256, page=256)), (PAGE, dict(page=16)), (PAGE, dict(page=96)), (PAGE, dict(page=32, block=64)),
    (NULL, dict(kv_ptrs=[None])), (NULL, dict(scale_ptrs=[None])), (NULL, dict(copies=None)),
    (ALIGN, dict(kv_ptrs=[A + 8])), (ALIGN, dict(scale_ptrs=[A + 2])), (ALIGN, dict(copies=A + 4)),
    (ALIAS, dict(pools=2, kv_ptrs=[A, A], scale_ptrs=[A, 2 * A])),
    (ALIAS, dict(pools=2, kv_ptrs=[A, 3 * A], scale_ptrs=[2 * A, 2 * A]))])
def test_copy(code, change):
    refused(code, dcp.dcp_mla_pages_copy, COPY, **change)


def test_copy_of_no_pairs_is_nothing():
    dcp.dcp_mla_pages_copy(**{**COPY, "n": 0, "copies": None})


PAGED = dict(latent=A, latent_row=512, k_rope=A, rope_row=64, dtype=0, N=4, B=2, Dk=576, cu_new=A, seq_lens=A,
             kv_ptrs=[A], scale_ptrs=[2 * A], table_ptrs=[A], cp=1, P=8, page=64, M=4, stream=0)
READ = dict(kv_ptrs=[A], scale_ptrs=[A], table_ptrs=[A], cp=1, B=2, P=8, page=64, M=4, Dk=576, block=1, interleave=1,
            starts=A, cu=A, N=4, out=A, out_row=576, dtype=0, stream=0)
DTYPE = -206
POOLS = [(SHAPE, dict(B=-1)), (SHAPE, dict(B=65536)), (SHAPE, dict(P=-1)), (SHAPE, dict(P=1 << 31)),
         (SHAPE, dict(M=0)), (SHAPE, dict(M=1 << 25)), (SHAPE, dict(B=65535, M=1 << 16)), (PAGE, dict(page=16)),
         (PAGE, dict(page=65)), (PAGE, dict(page=8192)), (PAGE, dict(page=32, block=64)), (BLOCK, dict(block=3)),
         (CP, dict(cp=0)), (CP, dict(cp=17, kv_ptrs=[A] * 17, scale_ptrs=[A] * 17, table_ptrs=[A] * 17)),
         (CP, dict(interleave=0)), (NULL, dict(table_ptrs=[None])),
         (NULL, dict(kv_ptrs=[None], scale_ptrs=[None])), (NULL, dict(scale_ptrs=[None])),
         (ALIGN, dict(table_ptrs=[A + 2])), (ALIGN, dict(kv_ptrs=[A + 8])), (ALIGN, dict(scale_ptrs=[A + 2])),
         (SHAPE, dict(Dk=640))]


@pytest.mark.parametrize("code,change", POOLS + [
    (SHAPE, dict(N=-1)), (SHAPE, dict(cu_new=None, N=3)), (SHAPE, dict(B=0)), (DTYPE, dict(dtype=2)),
    (NULL, dict(latent=None)), (NULL, dict(k_rope=None)), (NULL, dict(seq_lens=None)), (ALIGN, dict(latent_row=516)),
    (CP, dict(cp=2, kv_ptrs=[A, A], scale_ptrs=[A, 2 * A], table_ptrs=[A, A]))])
def test_paged_append(code, change):
    refused(code, dcp.dcp_mla_cache8_append_paged, PAGED, **change)


@pytest.mark.parametrize("code,change", POOLS + [
    (SHAPE, dict(N=-1)), (SHAPE, dict(cu=None, N=3)), (DTYPE, dict(dtype=5)), (NULL, dict(out=None)),
    (ALIGN, dict(out=A + 8)), (ALIGN, dict(out_row=580)), (ALIGN, dict(starts=A + 2))])
def test_paged_read(code, change):
    refused(code, dcp.dcp_mla_cache8_read_paged, READ, **change)


DECODE = dict(q=A, q_row=576 * 16, q_head=576, kv_ptrs=[A], scale_ptrs=[A], table_ptrs=[A], seq_lens=A, cp=1, B=2, H=16,
              Dk=576, Dv=512, P=8, page=64, M=40, block=1, interleave=1, window=0, sinks=0, scale=1.0, lse_base_e=True,
              workspace=A, workspace_bytes=1 << 40, out=A, lse=A, stream=0)
FLAGS, WINDOW = -207, -209


@pytest.mark.parametrize("code,change", POOLS + [
    (SHAPE, dict(H=0)), (SHAPE, dict(H=1025)), (SHAPE, dict(Dv=256)), (WINDOW, dict(window=-1)),
    (WINDOW, dict(sinks=4)), (WINDOW, dict(groups=A, shared=A, window=4)), (FLAGS, dict(flags=2)),
    (NULL, dict(q=None)), (NULL, dict(out=None)), (NULL, dict(seq_lens=None)), (NULL, dict(groups=A)),
    (NULL, dict(shared=A)), (ALIGN, dict(q=A + 2)), (ALIGN, dict(q_row=577)), (ALIGN, dict(out=A + 8)),
    (ALIGN, dict(groups=A + 4, shared=A)), (ALIGN, dict(groups=A, shared=A + 2)), (ALIGN, dict(status=A + 2)),
    (SHAPE, dict(B=65535, M=32767, page=64, cp=16, kv_ptrs=[A] * 16, scale_ptrs=[A] * 16, table_ptrs=[A] * 16))])
def test_paged_decode(code, change):
    refused(code, dcp.dcp_mla_cache8_decode_paged, DECODE, **change)


def test_paged_decode_workspace_bytes():
    ws = dcp.dcp_mla_cache8_decode_paged_workspace_bytes
    rows = dcp.dcp_mla_cache8_decode_workspace_bytes
    assert ws(1, 8, 16, 64, 100, 0, 0, False, 152) == rows(1, 8, 16, 6400, 0, 0, 152) > 0
    # up to three tiles a row: no row is split
    assert ws(1, 8, 16, 64, 4, 0, 0, False, 152) == ws(1, 8, 16, 64, 6, 0, 0, False, 152) == 0
    assert ws(1, 8, 16, 64, 7, 0, 0, False, 152) > 0 == ws(3, 8, 16, 64, 2, 0, 0, False, 152)
    # with groups a place for each row's own part and for each set of a group's heads, in blocks of 64
    assert ws(1, 8, 16, 64, 256, 0, 0, True, 152) >= (152 + 16) * 64 * 513 * 4
    assert ws(1, 2, 16, 64, 1024, 0, 0, True, 152) < ws(1, 4, 16, 64, 1024, 0, 0, True, 152)  # blocks of 32, of 64
    # groups make no difference with whole blocks of 64 heads, many rows, one, or fewer than 1024 tiles of room
    for B, H, M in ((8, 64, 1024), (8, 128, 1024), (2049, 16, 1024), (1, 16, 4096), (8, 16, 254)):
        assert ws(1, B, H, 64, M, 0, 0, True, 152) == ws(1, B, H, 64, M, 0, 0, False, 152)
    assert ws(1, 8, 16, 64, 256, 0, 0, True, 152) == ws(4, 8, 16, 64, 64, 0, 0, True, 152) != \
        ws(1, 8, 16, 64, 256, 0, 0, False, 152)
    assert ws(1, 0, 16, 64, 100, 0, 0, True, 152) == 0
    for bad in (dict(page=16), dict(page=96), dict(M=0), dict(M=1 << 26), dict(B=-1), dict(H=0), dict(sms=0)):
        a = {**dict(B=8, H=16, page=64, M=100, sms=152), **bad}
        assert ws(1, a["B"], a["H"], a["page"], a["M"], 0, 0, True, a["sms"]) == -1


def test_groups_on_the_host():
    groups, shared = dcp.mla_cache8_groups([2, 0, 1, 3], [40, 7, 0, 9], device="cpu")
    assert groups.tolist() == [[0, 2], [0, 2], [2, 1], [3, 3], [3, 3], [3, 3]]
    assert shared.tolist() == [40, 40, 0, 9, 9, 9] and groups.dtype == shared.dtype == torch.int32
    assert dcp.mla_cache8_groups([], [], device="cpu")[0].shape == (0, 2)
    for bad in (([1], []), ([-1], [0]), ([1], [-1]), ([1], [1 << 31])):
        with pytest.raises(ValueError):
            dcp.mla_cache8_groups(*bad, device="cpu")


def test_decode_wrapper_checks_groups():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    kv, sc, t = torch.zeros((4, 64, 576), dtype=torch.uint8), torch.ones((4, 64)), i32(2, 3)
    q = torch.zeros((2, 4, 576), dtype=torch.bfloat16)
    call = lambda tables=[t], **k: dcp.mla_cache8_decode(q, [kv], [sc], i32(2), 1.0, tables=tables, **k)
    with pytest.raises(ValueError, match="CUDA"):
        call(groups=i32(2, 2), shared=i32(2))
    for kw in (dict(groups=i32(2, 2)), dict(shared=i32(2)), dict(groups=i32(3, 2), shared=i32(2)),
               dict(groups=i32(2, 2).long(), shared=i32(2)), dict(groups=i32(2, 2), shared=i32(3)),
               dict(groups=i32(2, 2), shared=i32(2), window=5), dict(tables=None, groups=i32(2, 2), shared=i32(2)),
               dict(groups=i32(2, 4)[:, ::2], shared=i32(2)), dict(tables=[None]), dict(tables=[t.long()])):
        with pytest.raises(ValueError):
            call(**kw)


def test_paged_calls_of_nothing():
    dcp.dcp_mla_cache8_decode_paged(**{**DECODE, "B": 0, "workspace": None})
    dcp.dcp_mla_cache8_append_paged(**{**PAGED, "N": 0})
    dcp.dcp_mla_cache8_append_paged(**{**PAGED, "P": 0})
    dcp.dcp_mla_cache8_read_paged(**{**READ, "N": 0, "out": None})


def test_workspace_bytes():
    up, co = dcp.dcp_mla_pages_update_workspace_bytes, dcp.dcp_mla_pages_compact_workspace_bytes
    assert up(4, 100, 50, True) >= up(4, 100, 50, False) + 4 * 100 * 4
    assert up(20000, 1, 300000, False) >= 20000 * 16 + 300000 * 12 and co(100000) >= 2 * 12500
    for bad in ((-1, 1, 1), (65536, 1, 1), (1, 0, 1), (1, 1, 0), (65535, 1 << 15, 1)):
        assert up(*bad, False) == -1
    assert co(0) == co(1 << 31) == -1
    assert up(16384, 100, 262144, False) == 0 < up(16385, 100, 262144, False)
    assert up(1, 1, 262145, False) > 0 and up(1, 1, 1, True) > 0
    assert up(0, 4, 8, True) == 0


def test_wrappers():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    t, r, row = i32(2, 4), i32(8), i32(2)
    up = lambda t=t, r=r, a=row, b=row, c=row, page=64, **k: dcp.mla_cache8_pages_update(t, r, a, b, c, page=page, **k)
    with pytest.raises(ValueError, match="CUDA"):
        up()
    with pytest.raises(ValueError, match="CUDA"):
        dcp.mla_cache8_pages_compact(t, r)
    for kw in (dict(t=t.long()), dict(t=i32(4, 2).T), dict(t=row), dict(r=r.long()), dict(r=t), dict(r=i32(0)),
               dict(t=i32(2, 0)), dict(a=i32(3)), dict(b=row.long()), dict(c=None), dict(page=16), dict(page=100),
               dict(page=1 << 33), dict(cp=0), dict(cp=2, shard=2), dict(interleave=0), dict(out=(t, i32(9))),
               dict(out=(t.long(), r))):
        with pytest.raises(ValueError):
            up(**kw)
    kv, sc = torch.zeros((4, 64, 576), dtype=torch.uint8), torch.ones((4, 4))
    pairs = i32(3, 2)
    copy = dcp.mla_cache8_pages_copy
    with pytest.raises(ValueError, match="CUDA"):
        copy([kv], [sc], pairs)
    for c, s, p in [([], [], pairs), ([kv], [sc, sc], pairs), ([kv[..., :500]], [sc], pairs), ([kv[0]], [sc], pairs),
                    ([kv], [sc[:3]], pairs), ([kv], [torch.ones((4, 5))], pairs), ([kv, kv[:3]], [sc, sc], pairs),
                    ([kv[:, ::2]], [sc[:, ::2]], pairs), ([kv], [sc], pairs.long()), ([kv], [sc], i32(3, 3)),
                    ([kv], [sc], i32(2, 3).T), ([kv] * 129, [sc] * 129, pairs)]:
        with pytest.raises(ValueError):
            copy(c, s, p)
    with pytest.raises(TypeError):
        copy([kv.float()], [sc], pairs)
    with pytest.raises(TypeError):
        copy([kv], [sc.double()], pairs)


def test_wrappers_check_tables():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    kv, sc, t = torch.zeros((4, 64, 576), dtype=torch.uint8), torch.ones((4, 64)), i32(2, 3)
    lat, pe, lens = torch.zeros((2, 512), dtype=torch.bfloat16), torch.zeros((2, 64), dtype=torch.bfloat16), i32(2)
    kv48, sc48 = torch.zeros((4, 48, 576), dtype=torch.uint8), torch.ones((4, 48))
    calls = (lambda c, s, tables, **k: dcp.mla_cache8_append(lat, pe, c, s, lens, tables=tables, **k),
             lambda c, s, tables, **k: dcp.mla_cache8_read(c, s, 2, tables=tables, **k))
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call([kv], [sc], [t])
        for c, s, tables, kw in [([kv], [sc], [], {}), ([kv], [sc], [t, t], {}), ([kv], [sc], [None], {}),
                                 ([kv, None], [sc, None], [t, t], {}), ([kv], [sc], [t.long()], {}),
                                 ([kv], [sc], [lens], {}), ([kv], [sc], [i32(3, 2).T], {}),
                                 ([kv, kv.clone()], [sc, sc.clone()], [t, i32(2, 4)], {}), ([kv48], [sc48], [t], {}),
                                 ([kv], [sc], [i32(2, 0)], {}),
                                 ([kv[:, :32].contiguous()], [torch.ones((4, 1))], [t], dict(block=64))]:
            with pytest.raises(ValueError):
                call(c, s, tables, **kw)
    with pytest.raises(ValueError, match="seq_lens"):  # rows are the tables', not the pool's
        dcp.mla_cache8_append(lat, pe, [kv], [sc], i32(4), tables=[t])


# ---- the plain forms, by hand ---------------------------------------------------------


def test_a_fork_shares_whole_pages_and_copies_the_one_that_is_written():
    # row 0: 70 tokens on pages 3, 5; row 1 becomes its twin, and both write their next token
    t, r, c, m = ref.update([[3, 5, -1], [-1, -1, -1]], [0, 0, 0, 1, 0, 1], [0, 0], [70, 70], [71, 71], 64)
    assert (t, r, c, m) == ([[3, 0, -1], [3, 5, -1]], [1, 0, 0, 2, 0, 1], [[5, 0], [-1, -1]], 0)
    # only row 1 writes: row 0 keeps the page
    t, r, c, m = ref.update([[3, 5, -1], [-1, -1, -1]], [0, 0, 0, 1, 0, 1], [0, 0], [70, 70], [70, 71], 64)
    assert (t, r, c, m) == ([[3, 5, -1], [3, 0, -1]], [1, 0, 0, 2, 0, 1], [[-1, -1], [5, 0]], 0)
    # at a page's end nothing is copied
    t, r, c, m = ref.update([[3, -1], [-1, -1]], [0, 0, 0, 1], [0, 0], [64, 64], [65, 65], 64)
    assert (t, r, c, m) == ([[3, 0], [3, 1]], [1, 1, 0, 2], [[-1, -1], [-1, -1]], 0)


def test_rows_end_and_their_pages_are_dealt_in_the_same_step():
    t, r, c, m = ref.update([[0, 1], [2, -1]], [1, 1, 1], [-1, 1], [0, 64], [0, 128], 64)
    assert (t, r, c, m) == ([[-1, -1], [2, 0]], [1, 0, 1], [[-1, -1]] * 2, 0)
    # rows change places
    t, r, c, m = ref.update([[0, 1], [2, -1]], [1, 1, 1], [1, 0], [64, 100], [64, 100], 64)
    assert (t, r, c, m) == ([[2, -1], [0, 1]], [1, 1, 1], [[-1, -1]] * 2, 0)


def test_a_pool_that_runs_out():
    t, r, c, m = ref.update([[0, -1, -1]], [1, 0], [0], [10], [190], 64)
    assert (t, r, c, m) == ([[0, 1, -1]], [1, 1], [[-1, -1]], 1)


def test_compaction_by_hand():
    t, r, c = ref.compact([[5, 1], [5, -1]], [0, 1, 0, 0, 0, 2])
    assert (t, r, c) == ([[0, 1], [0, -1]], [2, 1, 0, 0, 0, 0], [[5, 0]])
