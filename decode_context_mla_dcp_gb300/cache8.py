"""The 8-bit latent cache from torch tensors: rotary positions, the quantising
append, the read-back and single-token attention (include/dcp_mla_cache8.h).

A row's cache is [T, 512 latent + 64 rotary] e4m3 (or 512 alone) with one fp32
scale for each ``block`` consecutive tokens. Under context parallelism position
p is held by shard (p / interleave) mod cp; calls take one cache and one scale
tensor per shard, None for a shard that this device does not hold ("[DCP]
Optimize shared Output, Query, and Indexer/Top-K via peer memory", sglang
#32851, commit notes on the interleaved KV shards). A serving step chains them:

    mla_rope(q_pe, positions, inv_freq, out=q[..., 512:])
    mla_cache8_append(latent, k_pe, caches, scales, seq_lens, inv_freq=inv_freq)
    out, lse = mla_cache8_decode(q, caches, scales, seq_lens + 1, scale)

Streams: everything runs on ``stream`` (default: the current stream of the
tensors' device); what a call allocates is allocated for that stream. Wrong
arguments raise ValueError, TypeError or DcpError before anything is launched.
A batch of no rows is nothing to do; a cache of no tokens (T = 0) is refused, for
its tensor has no address.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

from . import _binding as _b

_torch = None
_DTYPES: dict = {}  # torch dtype -> library dtype
_SMS: dict = {}
_ROOM: dict = {}  # sizes of a decode -> bytes of workspace


def _ready():
    """The library and torch (imported on first use)."""
    global _torch
    if _torch is None:
        import torch
        _DTYPES.update({torch.bfloat16: _b.DCP_DTYPE_BF16, torch.float16: _b.DCP_DTYPE_F16,
                        torch.float32: _b.DCP_DTYPE_F32})
        _torch = torch
    return _b._lib or _b.load(), _torch


# A small call's time is its host time, and most of that is looking at tensors: the
# checks use what is cheapest to ask (device indices, not device objects; shape[0],
# not len()).


def _on(index: int, stream):
    """(raw stream, context) on CUDA device ``index``: the stream to launch on, and
    what to be inside of while allocating and launching (None where that is the
    present state)."""
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        # (the raw handle: building a torch.cuda.Stream for it costs as much as a launch)
        return _torch._C._cuda_getCurrentRawStream(index), \
            None if _torch._C._cuda_getDevice() == index else _torch.cuda.device(index)
    cuda = _torch.cuda
    if isinstance(stream, int):
        raw = stream
        stream = cuda.default_stream(index) if raw == 0 else cuda.ExternalStream(raw, device=index)
    else:
        raw = int(stream.cuda_stream)
        if stream.device.index != index:
            raise ValueError("the stream is on another device than the tensors")
    both = contextlib.ExitStack()
    both.enter_context(cuda.device(index))
    both.enter_context(cuda.stream(stream))
    return raw, both


def _sms(index: int) -> int:
    n = _SMS.get(index)
    if n is None:
        n = _SMS[index] = int(_torch.cuda.get_device_properties(index).multi_processor_count)
    return n


def _cuda(index: int):
    return _torch.device("cuda", index)


def _ints(name, t, n, index):
    """The address of a contiguous int32 tensor of n entries (None for None)."""
    if t is None:
        return None
    if t.dtype != _torch.int32 or t.dim() != 1 or t.shape[0] != n or t.get_device() != index or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on the caches' device")
    return t.data_ptr()


def _shards(caches, scales, block, interleave):
    """Check the shards' tensors; (device index, B, T, Dk, cache pointers, scale pointers)."""
    cp = len(caches)
    if cp < 1 or cp > _b.DCP_MLA_CACHE8_CP_MAX or len(scales) != cp:
        raise ValueError(f"need 1 to {_b.DCP_MLA_CACHE8_CP_MAX} caches (None for a shard that is not held) and as "
                         "many scale tensors")
    if block < 1 or block > _b.DCP_MLA_CACHE8_BLOCK_MAX or block & (block - 1):
        raise ValueError(f"block must be a power of two, at most {_b.DCP_MLA_CACHE8_BLOCK_MAX}")
    if interleave < 1 or interleave > 1 << 24:  # (here, for ctypes drops an int's high bits)
        raise ValueError("interleave must be in [1, 2^24]")
    shape = None
    kv, sc = (ctypes.c_void_p * cp)(), (ctypes.c_void_p * cp)()
    e4m3, codes, f32 = _torch.float8_e4m3fn, _torch.uint8, _torch.float32
    for j in range(cp):
        c, s = caches[j], scales[j]
        if c is None or s is None:
            if c is not s:
                raise ValueError("a shard has both a cache and scales, or neither")
            continue
        if shape is None:
            index, shape = c.get_device(), c.shape
            if len(shape) != 3 or shape[2] not in (512, 576):
                raise ValueError("a cache must be [B, T, 512] or [B, T, 576]")
            B, T, dk = shape
            sshape = (B, -(-T // block))
        elif c.shape != shape:
            raise ValueError("the caches must have one shape")
        if (c.dtype != e4m3 and c.dtype != codes) or s.dtype != f32:
            raise TypeError("caches must be float8_e4m3fn (or uint8 codes) and scales float32")
        if s.shape != sshape or c.get_device() != index or s.get_device() != index:
            raise ValueError("shards must be on one device, and scales [B, ceil(T / block)]")
        if not (c.is_contiguous() and s.is_contiguous()):
            raise ValueError("caches and scales must be contiguous")
        # (tensors of no rows have no address, and NULL is a shard that is not held: one that is never read stands in)
        kv[j], sc[j] = (c.data_ptr(), s.data_ptr()) if B else (256 * (j + 1), 256 * (j + 1))
    if shape is None:
        raise ValueError("no shard is held here")
    return index, B, T, dk, kv, sc


def _tables(tables, caches, page, block, index):
    """Check a paged cache's tables; (B, M, table pointers)."""
    cp = len(caches)
    if len(tables) != cp:
        raise ValueError("need a table for each cache (None for a shard that is not held)")
    if page < _b.DCP_MLA_PAGE_MIN or page > _b.DCP_MLA_PAGE_MAX or page & (page - 1) or page % block:
        raise ValueError(f"a page must be a power of two in [{_b.DCP_MLA_PAGE_MIN}, {_b.DCP_MLA_PAGE_MAX}] and a "
                         "multiple of block")
    shape, i32 = None, _torch.int32
    tb = (ctypes.c_void_p * cp)()
    for j in range(cp):
        t = tables[j]
        if t is None or caches[j] is None:
            if t is not caches[j]:
                raise ValueError("a shard has both a cache and tables, or neither")
            continue
        if shape is None:
            shape = t.shape
        if len(shape) != 2 or t.shape != shape or t.dtype != i32 or t.get_device() != index or not t.is_contiguous():
            raise ValueError("tables must be contiguous int32 tensors [B, M] of one shape on the caches' device")
        tb[j] = t.data_ptr()
    B, M = shape
    if M < 1 or M * page >= 1 << 31:
        raise ValueError("tables need a column, and M * page must be below 2^31")
    return B, M, tb


def mla_rope_inv_freq(rot: int = 64, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                      original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                      mscale: float = 1.0, mscale_all_dim: float = 0.0, device="cuda"):
    """Radians per position of each rotated pair, and the factor for cos and sin.

    scaling "none": base^(-2i / rot). "linear": divided by ``factor``. "yarn":
    pairs that turn more than ``beta_fast`` times over ``original_len`` positions
    keep their frequency, those below ``beta_slow`` turns are divided by
    ``factor``, those between are blended linearly over the pair index; the
    factor is (0.1 mscale ln(factor) + 1) / (0.1 mscale_all_dim ln(factor) + 1).
    Returns (float64 tensor [rot / 2] on ``device``, float), for mla_rope and
    mla_cache8_append."""
    import torch
    if rot < 2 or rot % 2 or base <= 0 or factor < 1 or original_len < 1:
        raise ValueError("rot must be even and positive, base positive, factor >= 1, original_len >= 1")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-i / rot)
    amp = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if base == 1:
            raise ValueError("base must not be 1 with yarn")
        at = [rot * math.log(original_len / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (beta_fast, beta_slow)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        keep = 1 - ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / factor * (1 - keep) + f * keep
        amp = (0.1 * mscale * math.log(factor) + 1) / (0.1 * mscale_all_dim * math.log(factor) + 1)
    elif scaling != "none":
        raise ValueError("scaling must be 'none', 'linear' or 'yarn'")
    return f.to(device), amp


def _meet(gap, n, h, d, row, head, orow, ohead) -> bool:
    """Whether x [n, h, d] and out, ``gap`` elements behind it, may share elements: if
    their spans do, unless they are different dims of the same heads."""
    if gap < 0:
        gap, row, head, orow, ohead = -gap, orow, ohead, row, head
    if gap >= (n - 1) * row + (h - 1) * head + d:
        return False
    step = math.gcd(row if n > 1 else 0, head if h > 1 else 0)
    return (n > 1 and row != orow) or (h > 1 and head != ohead) or step == 0 or not d <= gap % step <= step - d


def _folded(n, h, d, row, head) -> bool:
    """Whether [n, h, d] with strides (row, head, 1) has two elements in one place."""
    if n > 1 and row < d or h > 1 and head < d:
        return True
    if n <= 1 or h <= 1 or head >= (n - 1) * row + d or row >= (h - 1) * head + d:
        return False
    # heads and rows interlock: a row i further meets the head whose place is next below or above its own
    if n > h:
        n, h, row, head = h, n, head, row
    return any(i * row % head < d and i * row // head < h or
               head - i * row % head < d and i * row // head + 1 < h for i in range(1, n))


def mla_rope(x, positions, inv_freq, *, start: int = 0, interleaved: bool = True, mscale: float = 1.0, out=None,
             stream=None):
    """Rotary positions on dims [start, start + 2 len(inv_freq)) of every head.

    x: CUDA bf16, fp16 or fp32 [N, H, D] (unit stride along D). positions: int32
    or int64 [N]. inv_freq: float64 [rot / 2] (mla_rope_inv_freq). ``interleaved``
    pairs dims (2i, 2i + 1), otherwise (i, i + rot / 2). out: None allocates
    [N, H, D]; x itself rotates in place; another tensor or view (unit stride
    along D, not overlapping x) also receives the dims that are not rotated.
    What is written must not share elements between rows or heads (an expanded x
    cannot be rotated in place). Returns out."""
    lib, torch = _ready()
    if x.dim() != 3:
        raise ValueError("x must be [N, H, D]")
    n, h, d = x.shape
    row, head, unit = x.stride()
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise TypeError("x must be bf16, fp16 or fp32")
    index = x.get_device()
    if unit != 1 and d > 1:
        raise ValueError("x needs unit stride along D")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous() or \
            inv_freq.get_device() != index:
        raise ValueError("inv_freq must be a contiguous float64 tensor on x's device")
    wide = positions.dtype == torch.int64
    if not (wide or positions.dtype == torch.int32) or positions.dim() != 1 or positions.shape[0] != n or \
            positions.get_device() != index or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int32 or int64 tensor [N] on x's device")
    if start < 0 or start > d:
        raise ValueError("start must be in [0, D]")
    src = x.data_ptr()
    if out is not None:
        dst, orow, ohead = src, row, head
        if out is not x:
            orow, ohead, unit = out.stride() if out.dim() == 3 else (0, 0, 0)
            if out.shape != x.shape or out.dtype != x.dtype or out.get_device() != index or (unit != 1 and d > 1):
                raise ValueError("out must have x's shape, dtype and device, and unit stride along D")
            dst = out.data_ptr()
        if _folded(n, h, d, orow, ohead):
            raise ValueError("out's rows or heads overlap each other")
        if dst != src and n * h > 0 and _meet((dst - src) // x.element_size(), n, h, d, row, head, orow, ohead):
            raise ValueError("out overlaps x: pass x itself to rotate in place")
    raw, inside = _on(index, stream)
    if inside is not None:
        with inside:
            return mla_rope(x, positions, inv_freq, start=start, interleaved=interleaved, mscale=mscale, out=out)
    if out is None:
        out = torch.empty((n, h, d), dtype=x.dtype, device=x.device)
        dst, orow, ohead = out.data_ptr(), h * d, d
    rc = lib.dcp_mla_rope(src, row, head, positions.data_ptr(), wide, inv_freq.data_ptr(), n, h, d, start,
                          2 * inv_freq.shape[0], interleaved, mscale, dtype, dst, orow, ohead, raw)
    if rc:
        _b._check8(rc)
    return out


def mla_cache8_append(latent, k_rope, caches, scales, seq_lens, *, cu_new=None, block: int = 1, interleave: int = 1,
                      inv_freq=None, interleaved: bool = True, mscale: float = 1.0, tables=None,
                      stream=None) -> None:
    """Quantise new tokens into the caches, in place.

    latent: bf16 or fp16 [N, 512]; k_rope: [N, 64] of the same type, or None for
    512-wide caches (unit inner strides, row strides multiples of 8). Row b's new
    tokens are latent[cu_new[b]:cu_new[b + 1]] (int32 [B + 1]; None: N / B each),
    at positions seq_lens[b], ... (int32 [B]: the lengths before the call). With
    inv_freq (float64 [32]) k_rope is rotated on the way. A block's scale is the
    smallest power of two that holds its values; a block that already holds
    tokens is requantised where its scale grows. tables (int32 [B, M] per shard):
    the caches are pools of pages [P, page, Dk] (cache8_pages.py), B is theirs."""
    lib, torch = _ready()
    index, B, T, dk, kv, sc = _shards(caches, scales, block, interleave)
    if tables is not None:
        P, page = B, T
        B, M, tb = _tables(tables, caches, page, block, index)
    dtype = _DTYPES.get(latent.dtype)
    if dtype is None or dtype == _b.DCP_DTYPE_F32:
        raise TypeError("latent must be bf16 or fp16")
    if latent.dim() != 2 or latent.get_device() != index:
        raise ValueError("latent must be [N, 512] with unit inner stride, on the caches' device")
    n, width = latent.shape
    row, unit = latent.stride()
    if width != 512 or unit != 1:
        raise ValueError("latent must be [N, 512] with unit inner stride, on the caches' device")
    rope_ptr, rope_row = None, 0
    if dk == 576:
        if k_rope is None or k_rope.shape != (n, 64) or k_rope.dtype != latent.dtype or k_rope.stride(1) != 1 or \
                k_rope.get_device() != index:
            raise ValueError("k_rope must be [N, 64] of latent's dtype with unit inner stride, on the caches' device")
        rope_ptr, rope_row = k_rope.data_ptr(), k_rope.stride(0)
    elif k_rope is not None or inv_freq is not None:
        raise ValueError("512-wide caches have no rotary part: k_rope and inv_freq must be None")
    freq_ptr = None
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64 or inv_freq.shape != (32,) or not inv_freq.is_contiguous() or \
                inv_freq.get_device() != index:
            raise ValueError("inv_freq must be a contiguous float64 tensor [32] on the caches' device")
        freq_ptr = inv_freq.data_ptr()
    lens = _ints("seq_lens", seq_lens, B, index)
    if lens is None:
        raise ValueError("seq_lens is required")
    cu = _ints("cu_new", cu_new, B + 1, index)
    raw, inside = _on(index, stream)
    if inside is not None:
        with inside:
            return mla_cache8_append(latent, k_rope, caches, scales, seq_lens, cu_new=cu_new, block=block,
                                     interleave=interleave, inv_freq=inv_freq, interleaved=interleaved, mscale=mscale,
                                     tables=tables)
    if tables is None:
        rc = lib.dcp_mla_cache8_append(latent.data_ptr(), row, rope_ptr, rope_row, dtype, n, B, dk, cu, lens, kv, sc,
                                       len(caches), T, block, interleave, freq_ptr, interleaved, mscale, raw)
    else:
        rc = lib.dcp_mla_cache8_append_paged(latent.data_ptr(), row, rope_ptr, rope_row, dtype, n, B, dk, cu, lens,
                                             kv, sc, tb, len(caches), P, page, M, block, interleave, freq_ptr,
                                             interleaved, mscale, raw)
    if rc:
        _b._check8(rc)


def mla_cache8_read(caches, scales, total: int, *, starts=None, cu=None, block: int = 1, interleave: int = 1,
                    dtype=None, out=None, tables=None, stream=None):
    """Cached tokens as numbers: out[cu[b] + i] is position starts[b] + i of row b.

    total: packed tokens in all; cu: int32 [B + 1] (None: total / B each); starts:
    int32 [B] (None: 0). dtype: bf16 (default), fp16 or fp32. out: None allocates
    [total, Dk]; or a tensor of that shape, unit inner stride, rows and base on
    16-byte boundaries. Tokens that no held shard has are left as they were (in
    a tensor that the call allocates: undefined). tables: as for the append.
    Returns out."""
    lib, torch = _ready()
    index, B, T, dk, kv, sc = _shards(caches, scales, block, interleave)
    if tables is not None:
        P, page = B, T
        B, M, tb = _tables(tables, caches, page, block, index)
    if total < 0:
        raise ValueError("total must not be negative")
    dtype = (torch.bfloat16 if out is None else out.dtype) if dtype is None else dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError("dtype must be bf16, fp16 or fp32")
    start_ptr, cu_ptr = _ints("starts", starts, B, index), _ints("cu", cu, B + 1, index)
    raw, inside = _on(index, stream)
    if inside is not None:
        with inside:
            return mla_cache8_read(caches, scales, total, starts=starts, cu=cu, block=block, interleave=interleave,
                                   dtype=dtype, out=out, tables=tables)
    row = dk
    if out is None:
        out = torch.empty((total, dk), dtype=dtype, device=_cuda(index))
    elif out.shape != (total, dk) or out.dtype != dtype or out.get_device() != index or out.stride(1) != 1:
        raise ValueError("out must be [total, Dk] of dtype with unit inner stride, on the caches' device")
    else:
        row = out.stride(0)
        if row < dk and total > 1:
            raise ValueError("out's rows overlap each other")
    if tables is None:
        rc = lib.dcp_mla_cache8_read(kv, sc, len(caches), B, T, dk, block, interleave, start_ptr, cu_ptr, total,
                                     out.data_ptr(), row, code, raw)
    else:
        rc = lib.dcp_mla_cache8_read_paged(kv, sc, tb, len(caches), B, P, page, M, dk, block, interleave, start_ptr,
                                           cu_ptr, total, out.data_ptr(), row, code, raw)
    if rc:
        _b._check8(rc)
    return out


def mla_cache8_decode(q, caches, scales, seq_lens, scale: float, *, block: int = 1, interleave: int = 1,
                      window: int = 0, sinks: int = 0, lse_base_e: bool = True, out=None, lse=None, workspace=None,
                      status=None, flags: int = 0, tables=None, groups=None, shared=None, stream=None):
    """Single-token attention over the cached positions of each row.

    q: CUDA bf16 [B, H, Dk] (unit stride along Dk, even row and head strides);
    seq_lens: int32 [B] cached positions over all shards. window > 0 limits a row
    to its last ``window`` positions and its first ``sinks``. Returns (out, lse):
    bf16 [B, H, 512] and fp32 [B, H] (base e, or 2); heads [r H/cp, (r + 1) H/cp)
    of out are what destination r of mla_decode_dcp receives. With some shards
    None the result is the partial over the held ones, for ``merge``. workspace: a
    contiguous CUDA tensor of at least dcp_mla_cache8_decode_workspace_bytes bytes,
    256-byte aligned, allocated when not given and needed. status: None, or an
    int32 CUDA tensor (see the C header).

    tables: as for the append (workspace then: dcp_mla_cache8_decode_paged_workspace_bytes).
    With tables, groups (int32 [B, 2]: first row and rows of each row's group of
    consecutive rows) and shared (int32 [B]: positions that a group's rows have in
    common, in the same pages) let rows attend to a common prefix together;
    mla_cache8_groups makes both. A row that is shorter than that (length 0: it has
    ended) takes no part, the first one neither. The result is the same without: groups
    save time where the prefix is long beside the rows' own tokens, and cost some where
    it is short (see the C header)."""
    lib, torch = _ready()
    index, B, T, dk, kv, sc = _shards(caches, scales, block, interleave)
    if tables is not None:
        P, page = B, T
        B, M, tb = _tables(tables, caches, page, block, index)
        group_ptr = shared_ptr = None
        if groups is not None:
            if groups.dtype != torch.int32 or groups.shape != (B, 2) or groups.get_device() != index or \
                    not groups.is_contiguous():
                raise ValueError("groups must be a contiguous int32 tensor [B, 2] on the caches' device")
            if window > 0:
                raise ValueError("groups do not go together with a window")
            group_ptr, shared_ptr = groups.data_ptr(), _ints("shared", shared, B, index)
        if (groups is None) != (shared is None):
            raise ValueError("groups and shared come together")
    elif groups is not None or shared is not None:
        raise ValueError("groups need a paged cache: tables")
    if q.dim() != 3 or q.dtype != torch.bfloat16 or q.get_device() != index:
        raise ValueError("q must be bf16 [B, H, Dk] with unit inner stride, on the caches' device")
    qb, H, qd = q.shape
    row, head, unit = q.stride()
    if qb != B or qd != dk or unit != 1:
        raise ValueError("q must be bf16 [B, H, Dk] with unit inner stride, on the caches' device")
    lens = _ints("seq_lens", seq_lens, B, index)
    if lens is None:
        raise ValueError("seq_lens is required")
    cp = len(caches)
    if window < 0 or sinks < 0 or max(window, sinks) >= 1 << 63:
        raise ValueError("window and sinks must be in [0, 2^63)")
    raw, inside = _on(index, stream)
    if inside is not None:
        with inside:
            return mla_cache8_decode(q, caches, scales, seq_lens, scale, block=block, interleave=interleave,
                                     window=window, sinks=sinks, lse_base_e=lse_base_e, out=out, lse=lse,
                                     workspace=workspace, status=status, flags=flags, tables=tables, groups=groups,
                                     shared=shared)
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q.device)
    elif out.shape != (B, H, 512) or out.dtype != torch.bfloat16 or out.get_device() != index or \
            not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor [B, H, 512] on the caches' device")
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    elif lse.shape != (B, H) or lse.dtype != torch.float32 or lse.get_device() != index or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [B, H] on the caches' device")
    room = None
    if workspace is None:
        key = (cp, B, H, T, window, sinks, index) if tables is None else \
            (cp, B, H, T, window, sinks, index, M, groups is None)
        size = _ROOM.get(key)
        if size is None:
            if len(_ROOM) > 4096:
                _ROOM.clear()
            size = lib.dcp_mla_cache8_decode_workspace_bytes(cp, B, H, T, window, sinks, _sms(index)) \
                if tables is None else lib.dcp_mla_cache8_decode_paged_workspace_bytes(
                    cp, B, H, page, M, window, sinks, groups is not None, _sms(index))
            _ROOM[key] = size
        if size > 0:
            workspace = torch.empty((size,), dtype=torch.uint8, device=q.device)
            room = workspace.data_ptr()
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the caches' device")
    else:
        size, room = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    if status is not None:
        if status.dtype != torch.int32 or status.get_device() != index or status.numel() < 1:
            raise ValueError("status must be an int32 tensor on the caches' device")
        status = status.data_ptr()
    if tables is None:
        rc = lib.dcp_mla_cache8_decode(q.data_ptr(), row, head, kv, sc, lens, cp, B, H, dk, 512, T, block, interleave,
                                       window, sinks, scale, lse_base_e, room, size, out.data_ptr(), lse.data_ptr(),
                                       status, flags, raw)
    else:
        rc = lib.dcp_mla_cache8_decode_paged(q.data_ptr(), row, head, kv, sc, tb, lens, group_ptr, shared_ptr, cp, B,
                                             H, dk, 512, P, page, M, block, interleave, window, sinks, scale,
                                             lse_base_e, room, size, out.data_ptr(), lse.data_ptr(), status, flags,
                                             raw)
    if rc:
        _b._check8(rc)
    return out, lse
