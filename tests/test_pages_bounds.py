"""Sizes and addresses at the limits of the calls on pages, on the host. Nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from .test_pages_refusals import A, ALIAS, COMPACT, COPY, DECODE, SHAPE, UPDATE, WS, built, refused  # noqa: F401


@pytest.mark.parametrize("M,page", [(1 << 26, 32), (1 << 19, 4096), (1 << 25, 64), ((1 << 31) - 2, 32),
                                    ((1 << 31) - 32, 64), ((1 << 31) - 129, 32)])
def test_a_row_has_room_for_less_than_2_31_tokens(M, page):
    """One row of M pages: loops over its entries count in 32 bits."""
    refused(SHAPE, dcp.dcp_mla_pages_update, UPDATE, B=1, M=M, page=page, tables=1 << 40, tables_out=1 << 40)
    if M >= 1 << 26:  # whatever the page
        refused(SHAPE, dcp.dcp_mla_pages_compact, COMPACT, B=1, M=M, tables=1 << 40, tables_out=1 << 40)
        for in_place in (False, True):
            assert dcp.dcp_mla_pages_update_workspace_bytes(1, M, 16, in_place) == -1


def test_the_wrapper_refuses_rows_of_2_31_tokens():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="2\\^31"):
        dcp.mla_cache8_pages_update(i32(1, 1 << 19), i32(8), i32(1), i32(1), i32(1), page=4096)
    assert dcp.dcp_mla_pages_update_workspace_bytes(1, (1 << 26) - 1, 16, False) == 0


# the step of the tables and the compaction with every buffer in a place of its own
APART = dict(tables=A, refs=2 * A, parents=3 * A, keeps=4 * A, wants=5 * A, tables_out=6 * A, refs_out=7 * A,
             copies=8 * A, missing=9 * A, workspace=10 * A)


@pytest.mark.parametrize("change", [
    dict(copies=A), dict(copies=A + 120), dict(copies=6 * A - 8), dict(copies=2 * A + 56), dict(copies=7 * A),
    dict(copies=3 * A), dict(copies=4 * A + 8), dict(copies=5 * A), dict(missing=A), dict(missing=7 * A + 60),
    dict(missing=4 * A), dict(missing=8 * A + 28), dict(tables_out=3 * A), dict(tables_out=4 * A - 124),
    dict(refs_out=5 * A), dict(tables_out=A, refs_out=2 * A, copies=A + 64),
    dict(tables_out=A, refs_out=2 * A, wants=A + 4), dict(tables_out=A, refs_out=2 * A, workspace=4 * A),
    dict(tables_out=A, refs_out=2 * A, workspace=8 * A)])
def test_an_update_that_would_write_over_what_it_takes(change):
    refused(ALIAS, dcp.dcp_mla_pages_update, {**UPDATE, **APART}, **change)


@pytest.mark.parametrize("change", [
    dict(copies=A), dict(copies=2 * A + 56), dict(copies=6 * A + 120), dict(copies=7 * A), dict(copies=10 * A),
    dict(workspace=A), dict(workspace=2 * A), dict(workspace=6 * A), dict(workspace=7 * A)])
def test_a_compaction_that_would_write_over_what_it_takes(change):
    apart = {k: APART[k] for k in ("tables", "refs", "tables_out", "refs_out", "copies", "workspace")}
    refused(ALIAS, dcp.dcp_mla_pages_compact, {**COMPACT, **apart}, **change)


POOL, ROOM = 16 * 64 * 576, 16 * 4 * 4  # bytes of COPY's pool and of its scales


@pytest.mark.parametrize("kv,scales", [
    ([A, A + 64 * 576], [4 * A, 5 * A]), ([A + POOL - 16, A], [4 * A, 5 * A]), ([A, 2 * A], [4 * A, 4 * A + 16]),
    ([A, 2 * A], [4 * A + ROOM - 4, 4 * A]), ([A, 2 * A, 3 * A, A + POOL // 2 // 16 * 16], [5 * A, 6 * A, 7 * A, 8 * A])])
def test_pools_that_overlap(kv, scales):
    refused(ALIAS, dcp.dcp_mla_pages_copy, COPY, pools=len(kv), kv_ptrs=kv, scale_ptrs=scales)


def test_pools_side_by_side():
    dcp.dcp_mla_pages_copy(**{**COPY, "n": 0, "pools": 2, "kv_ptrs": [A, A + POOL], "scale_ptrs": [4 * A + ROOM, 4 * A]})


SHARDS = lambda cp: dict(cp=cp, kv_ptrs=[A] * cp, scale_ptrs=[A] * cp, table_ptrs=[A] * cp)
TILES = [(2048, 16, 1 << 15), (40, 1, (1 << 25) - 1), (65, 1, 1 << 24)]  # rows, shards, pages of 64


@pytest.mark.parametrize("B,cp,M", TILES)
def test_groups_with_room_for_more_tiles_than_can_be_counted_twice(B, cp, M):
    """Groups make no difference there: what a call without them takes, one with them takes too."""
    ws = dcp.dcp_mla_cache8_decode_paged_workspace_bytes
    size = ws(cp, B, 16, 64, M, 0, 0, False, 152)
    assert size == ws(cp, B, 16, 64, M, 0, 0, True, 152) > 0
    assert ws(cp, B // 2, 16, 64, M, 0, 0, True, 152) > size  # (where they are used there are more places)
    for kw in ({}, dict(groups=A, shared=A)):
        with pytest.raises(dcp.DcpError) as e:
            dcp.dcp_mla_cache8_decode_paged(**{**DECODE, **SHARDS(cp), **kw, "B": B, "M": M, "workspace": None})
        assert e.value.status in (WS, -10)  # (without a GPU the workspace is not come to)


@pytest.mark.parametrize("B,cp,M", [(2 * B + 2, cp, M) for B, cp, M in TILES if 2 * B * M < 1 << 31] + [(63, 16, 1 << 22)])
def test_tiles_that_cannot_be_counted(B, cp, M):
    refused(SHAPE, dcp.dcp_mla_cache8_decode_paged, DECODE, **SHARDS(cp), B=B, M=M)
    for grouped in (False, True):
        assert dcp.dcp_mla_cache8_decode_paged_workspace_bytes(cp, B, 16, 64, M, 0, 0, grouped, 152) == -1
    assert dcp.dcp_mla_cache8_decode_workspace_bytes(cp, B, 16, M * 64, 0, 0, 152) == -1
    rows = dict(q=A, q_row=576 * 16, q_head=576, kv_ptrs=[A] * cp, scale_ptrs=[A] * cp, seq_lens=A, cp=cp, B=B, H=16,
                Dk=576, Dv=512, T=M * 64, block=1, interleave=1, window=0, sinks=0, scale=1.0, lse_base_e=True,
                workspace=A, workspace_bytes=1 << 40, out=A, lse=A, stream=0)
    refused(SHAPE, dcp.dcp_mla_cache8_decode, rows)


def test_the_messages_of_pages():
    seen = {dcp.dcp_mla_cache8_strerror(c) for c in (-211, -212, -213)}
    assert len(seen) == 3 and "cluster of 16" in dcp.dcp_mla_cache8_strerror(-213)
    assert dcp.dcp_mla_cache8_strerror(-214) not in seen
