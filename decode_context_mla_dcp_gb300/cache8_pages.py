"""The pages of an 8-bit latent cache from torch tensors (include/dcp_mla_pages.h).

A paged cache is a pool [P, page, Dk] e4m3 (or uint8 codes) with scales
[P, page / block], and, for each context shard, tables [B, M] int32 (the page of
each ``page`` tokens of a row; -1: none) and refs [P] int32 (how many rows hold a
page; 0: free). Tables and refs are the same for all layers. It starts as tables
of -1 and refs of 0, and a serving step chains

    wants = torch.where(parents < 0, 0, lens + 1)  # (a row ends with parents -1, lens 0 and wants 0)
    tables, refs, copies, missing = mla_cache8_pages_update(tables, refs, parents, lens, wants, page=64)
    mla_cache8_pages_copy(caches_of_all_layers, scales_of_all_layers, copies)
    mla_cache8_append(latent, k_pe, [cache], [scale], lens, tables=[tables], ...)
    out, lse = mla_cache8_decode(q, [cache], [scale], wants, scale, tables=[tables], ...)

Streams, errors and what a call allocates: as in cache8.py. Nothing is read back to
the host, so that a step can be captured into a graph (``missing`` tells a program
that looks at it that the pool ran out; rows then lack pages, and one whose copy could
not be made has lost the tokens that it kept in that page: a program that wants to go
back keeps the state before, with ``out``).
"""
from __future__ import annotations

import ctypes

from . import _binding as _b
from . import cache8 as _c

_ROOM: dict = {}  # sizes of a call -> bytes of workspace


def _tables_refs(tables, refs, torch):
    """(device index, B, M, P) of a pair of tables and counts."""
    index = tables.get_device()
    if tables.dtype != torch.int32 or tables.dim() != 2 or not tables.is_contiguous():
        raise ValueError("tables must be a contiguous int32 tensor [B, M]")
    if refs.dtype != torch.int32 or refs.dim() != 1 or not refs.is_contiguous() or refs.get_device() != index:
        raise ValueError("refs must be a contiguous int32 tensor [P] on the tables' device")
    B, M = tables.shape
    return index, B, M, refs.shape[0]


def _outputs(out, tables, refs, index):
    """The pair that the call writes."""
    if out is None:
        return tables, refs
    t, r = out
    torch = _c._torch
    if t.shape != tables.shape or r.shape != refs.shape or t.dtype != torch.int32 or r.dtype != torch.int32 or \
            t.get_device() != index or r.get_device() != index or not (t.is_contiguous() and r.is_contiguous()):
        raise ValueError("out must be contiguous int32 tensors like tables and refs, on their device")
    return t, r


def _pairs(copies, n, index):
    torch = _c._torch
    if copies is None:
        return torch.empty((n, 2), dtype=torch.int32, device=_c._cuda(index))
    if copies.shape != (n, 2) or copies.dtype != torch.int32 or copies.get_device() != index or \
            not copies.is_contiguous():
        raise ValueError(f"copies must be a contiguous int32 tensor [{n}, 2] on the tables' device")
    return copies


def _space(workspace, key, ask, index):
    """(address, bytes, what keeps them) of the workspace."""
    if workspace is None:
        size = _ROOM.get(key)
        if size is None:
            if len(_ROOM) > 4096:
                _ROOM.clear()
            size = _ROOM[key] = ask()
        if size <= 0:
            return None, size, None
        torch = _c._torch
        workspace = torch.empty((size,), dtype=torch.uint8, device=_c._cuda(index))
        return workspace.data_ptr(), size, workspace
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the tables' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def mla_cache8_groups(rows, shared, device="cuda"):
    """The groups of a batch for mla_cache8_decode, from the host: rows[g] consecutive
    rows of the batch begin with the same shared[g] positions, in the same pages (a row
    alone is a group of 1). Worth it where shared is long beside the rows' own tokens
    (dcp_mla_pages.h says how long). Returns (groups int32 [B, 2], shared int32 [B])."""
    import torch
    rows, shared = [int(n) for n in rows], [int(n) for n in shared]
    if len(rows) != len(shared) or min(rows + shared, default=0) < 0 or max(shared, default=0) >= 1 << 31:
        raise ValueError("rows and shared must be counts of the same groups")
    pairs, common, first = [], [], 0
    for n, s in zip(rows, shared):
        pairs += [(first, n)] * n
        common += [s] * n
        first += n
    return torch.tensor(pairs, dtype=torch.int32, device=device).view(first, 2), \
        torch.tensor(common, dtype=torch.int32, device=device)


def mla_cache8_pages_update(tables, refs, parents, keeps, wants, *, page: int, cp: int = 1, shard: int = 0,
                            interleave: int = 1, out=None, copies=None, missing=None, workspace=None, stream=None):
    """Rows take over other rows' pages, are cut back, end, begin and grow, all at once.

    Row b keeps the first keeps[b] positions of what row parents[b] held (b itself to
    go on; -1: nothing, and with wants[b] 0 the row ends) and gets pages for wants[b]
    positions (all int32 [B]; positions of the whole sequence, of which shard ``shard``
    of ``cp`` has its part; keeps[b] is a length of row parents[b]). Pages are
    shared, not copied, but for one that row b is about to write (wants[b] > keeps[b])
    behind kept tokens while another row holds it: row b gets a fresh one in its place
    and copies[b] = (old, new), for mla_cache8_pages_copy; other rows of copies are -1.
    Fresh pages are the free ones with the lowest numbers, dealt in row order; where
    they run out the entry is -1 and missing counts it (where that was to be a copy, the
    row has let go of the old page and of its tokens there). out: None changes tables and
    refs in place, or a pair of other tensors of their shapes. copies: int32 [B, 2],
    missing: int32 [1] (allocated when not given). Returns (tables, refs, copies,
    missing)."""
    lib, torch = _c._ready()
    index, B, M, P = _tables_refs(tables, refs, torch)
    if M < 1 or P < 1:
        raise ValueError("tables need a column and refs an entry")
    if page < _b.DCP_MLA_PAGE_MIN or page > _b.DCP_MLA_PAGE_MAX or page & (page - 1):
        raise ValueError(f"page must be a power of two in [{_b.DCP_MLA_PAGE_MIN}, {_b.DCP_MLA_PAGE_MAX}]")
    if M * page >= 1 << 31:
        raise ValueError("M * page must be below 2^31")
    if not 1 <= cp <= _b.DCP_MLA_CACHE8_CP_MAX or not 0 <= shard < cp or not 1 <= interleave <= 1 << 24:
        raise ValueError("cp must be in [1, 16], shard in [0, cp) and interleave in [1, 2^24]")
    rows = [_c._ints(name, t, B, index) for name, t in (("parents", parents), ("keeps", keeps), ("wants", wants))]
    if None in rows:
        raise ValueError("parents, keeps and wants are required")
    new_tables, new_refs = _outputs(out, tables, refs, index)
    raw, inside = _c._on(index, stream)
    if inside is not None:
        with inside:
            return mla_cache8_pages_update(tables, refs, parents, keeps, wants, page=page, cp=cp, shard=shard,
                                           interleave=interleave, out=out, copies=copies, missing=missing,
                                           workspace=workspace)
    copies = _pairs(copies, B, index)
    if missing is None:
        missing = torch.empty((1,), dtype=torch.int32, device=_c._cuda(index))
    elif missing.dtype != torch.int32 or missing.numel() != 1 or missing.get_device() != index:
        raise ValueError("missing must be an int32 tensor of one entry on the tables' device")
    place = new_refs.data_ptr() == refs.data_ptr()
    room, size, workspace = _space(workspace, (B, M, P, place),
                                   lambda: lib.dcp_mla_pages_update_workspace_bytes(B, M, P, place), index)
    rc = lib.dcp_mla_pages_update(tables.data_ptr(), refs.data_ptr(), *rows, B, M, P, page, cp, shard, interleave,
                                  new_tables.data_ptr(), new_refs.data_ptr(), copies.data_ptr(), missing.data_ptr(),
                                  room, size, raw)
    if rc:
        _b._check8(rc)
    return new_tables, new_refs, copies, missing


def mla_cache8_pages_compact(tables, refs, *, out=None, copies=None, workspace=None, stream=None):
    """Move the pages in use to the front of the pool, so that its end can be given up.

    With n pages in use, those at n and beyond go, ascending, to the free ones below n:
    tables and refs are changed (in place, or into the pair ``out``), and copies
    (int32 [P // 2, 2], allocated when not given) lists (page, new place), then -1: the
    tokens move with mla_cache8_pages_copy. Returns (tables, refs, copies)."""
    lib, torch = _c._ready()
    index, B, M, P = _tables_refs(tables, refs, torch)
    if M < 1 or P < 1:
        raise ValueError("tables need a column and refs an entry")
    new_tables, new_refs = _outputs(out, tables, refs, index)
    raw, inside = _c._on(index, stream)
    if inside is not None:
        with inside:
            return mla_cache8_pages_compact(tables, refs, out=out, copies=copies, workspace=workspace)
    copies = _pairs(copies, P // 2, index)
    room, size, workspace = _space(workspace, P, lambda: lib.dcp_mla_pages_compact_workspace_bytes(P), index)
    rc = lib.dcp_mla_pages_compact(tables.data_ptr(), refs.data_ptr(), B, M, P, new_tables.data_ptr(),
                                   new_refs.data_ptr(), copies.data_ptr(), room, size, raw)
    if rc:
        _b._check8(rc)
    return new_tables, new_refs, copies


def mla_cache8_pages_copy(caches, scales, copies, *, stream=None) -> None:
    """Copy pages, codes and scales, inside each of several pools (the layers).

    caches: up to 128 pools [P, page, Dk] of one shape, scales: as many [P, page /
    block], of which no two overlap. copies: int32 [n, 2], (from, to) as mla_cache8_pages_update and
    mla_cache8_pages_compact give them; a pair with an entry outside [0, P) is passed
    over. No page may be the target of two pairs, or of one and the source of
    another."""
    lib, torch = _c._ready()
    pools = len(caches)
    if not 1 <= pools <= _b.DCP_MLA_PAGES_POOLS_MAX or len(scales) != pools:
        raise ValueError(f"need 1 to {_b.DCP_MLA_PAGES_POOLS_MAX} pools and as many scale tensors")
    first, sfirst = caches[0], scales[0]
    index, shape, sshape = first.get_device(), first.shape, sfirst.shape
    if len(shape) != 3 or shape[2] not in (512, 576) or len(sshape) != 2 or sshape[0] != shape[0] or sshape[1] < 1 or \
            shape[1] % sshape[1]:
        raise ValueError("pools must be [P, page, 512 or 576], and their scales [P, page / block]")
    P, page, dk = shape
    kv, sc = (ctypes.c_void_p * pools)(), (ctypes.c_void_p * pools)()
    for j in range(pools):
        c, s = caches[j], scales[j]
        if (c.dtype != torch.float8_e4m3fn and c.dtype != torch.uint8) or s.dtype != torch.float32:
            raise TypeError("pools must be float8_e4m3fn (or uint8 codes) and scales float32")
        if c.shape != shape or s.shape != sshape or c.get_device() != index or s.get_device() != index or \
                not (c.is_contiguous() and s.is_contiguous()):
            raise ValueError("pools and scales must be contiguous, of one shape each, and on one device")
        kv[j], sc[j] = c.data_ptr(), s.data_ptr()
    if copies.dim() != 2 or copies.shape[1] != 2 or copies.dtype != torch.int32 or copies.get_device() != index or \
            not copies.is_contiguous():
        raise ValueError("copies must be a contiguous int32 tensor [n, 2] on the pools' device")
    raw, inside = _c._on(index, stream)
    if inside is not None:
        with inside:
            return mla_cache8_pages_copy(caches, scales, copies)
    if P == 0 or page == 0:
        return
    rc = lib.dcp_mla_pages_copy(kv, sc, pools, P, page, dk, page // sshape[1], copies.data_ptr(), copies.shape[0],
                                raw)
    if rc:
        _b._check8(rc)
