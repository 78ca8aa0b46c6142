"""What the 8-bit cache's calls refuse, on the host: the C entry points with addresses that are never read, and the
torch wrappers with tensors that are not on a GPU. Nothing is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from decode_context_mla_dcp_gb300 import build as dcp_build

A = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    dcp_build.build()


def refused(code, fn, base, **change):
    kw = {**base, **change}
    with pytest.raises(dcp.DcpError) as e:
        fn(**kw)
    assert e.value.status == code
    assert dcp.dcp_mla_cache8_strerror(code) in str(e.value)


ROPE = dict(x=A, x_row=64, x_head=64, positions=A, pos64=True, inv_freq=A, N=4, H=1, D=64, start=0, rot=64,
            interleaved=True, mscale=1.0, dtype=0, out=2 * A, out_row=64, out_head=64, stream=0)
APPEND = dict(latent=A, latent_row=512, k_rope=A, rope_row=64, dtype=0, N=4, B=2, Dk=576, cu_new=A, seq_lens=A,
              kv_ptrs=[A], scale_ptrs=[A], cp=1, T=8, block=1, interleave=1, stream=0)
READ = dict(kv_ptrs=[A], scale_ptrs=[A], cp=1, B=2, T=8, Dk=576, block=1, interleave=1, starts=A, cu=A, N=4, out=A,
            out_row=576, dtype=0, stream=0)
DECODE = dict(q=A, q_row=576 * 16, q_head=576, kv_ptrs=[A], scale_ptrs=[A], seq_lens=A, cp=1, B=2, H=16, Dk=576,
              Dv=512, T=8, block=1, interleave=1, window=0, sinks=0, scale=1.0, lse_base_e=True, workspace=A,
              workspace_bytes=1 << 40, out=A, lse=A, stream=0)
NULL, SHAPE, BLOCK, CP, ALIGN, DTYPE, FLAGS, WS, WINDOW = range(-201, -210, -1)


@pytest.mark.parametrize("code,change", [
    (SHAPE, dict(N=-1)), (SHAPE, dict(H=0)), (SHAPE, dict(H=65536)), (SHAPE, dict(D=0)), (SHAPE, dict(rot=63)),
    (SHAPE, dict(rot=0)), (SHAPE, dict(rot=258, D=300)), (SHAPE, dict(start=1)), (SHAPE, dict(start=-1)),
    (SHAPE, dict(D=1 << 17)), (SHAPE, dict(N=1 << 31)), (DTYPE, dict(dtype=3)), (DTYPE, dict(dtype=-1)),
    (NULL, dict(x=None)), (NULL, dict(out=None)), (NULL, dict(positions=None)), (NULL, dict(inv_freq=None)),
    (ALIGN, dict(x=A + 1)), (ALIGN, dict(dtype=2, out=A + 2)), (ALIGN, dict(positions=A + 4)),
    (ALIGN, dict(inv_freq=A + 4)), (SHAPE, dict(out=A, out_row=128))])
def test_rope(code, change):
    refused(code, dcp.dcp_mla_rope, ROPE, **change)


def test_rope_of_no_tokens_is_nothing():
    dcp.dcp_mla_rope(**{**ROPE, "N": 0, "x": None})


SHARDS = [
    (BLOCK, dict(block=0)), (BLOCK, dict(block=3)), (BLOCK, dict(block=256)), (BLOCK, dict(block=-1)),
    (CP, dict(cp=0)), (CP, dict(cp=17, kv_ptrs=[A] * 17, scale_ptrs=[A] * 17)), (CP, dict(interleave=0)),
    (CP, dict(interleave=(1 << 24) + 1)), (NULL, dict(kv_ptrs=[None], scale_ptrs=[None])),
    (NULL, dict(scale_ptrs=[None])), (NULL, dict(cp=2, kv_ptrs=[A, None], scale_ptrs=[A, A])),
    (ALIGN, dict(kv_ptrs=[A + 8])), (ALIGN, dict(scale_ptrs=[A + 2])), (SHAPE, dict(B=-1)), (SHAPE, dict(B=65536)),
    (SHAPE, dict(T=-1)), (SHAPE, dict(T=1 << 31)), (SHAPE, dict(Dk=640))]


@pytest.mark.parametrize("code,change", SHARDS + [
    (SHAPE, dict(N=-1)), (SHAPE, dict(cu_new=None, N=3)), (SHAPE, dict(B=0)), (DTYPE, dict(dtype=2)),
    (NULL, dict(latent=None)), (NULL, dict(k_rope=None)), (NULL, dict(seq_lens=None)), (ALIGN, dict(latent=A + 2)),
    (ALIGN, dict(latent_row=516)), (ALIGN, dict(rope_row=68)), (ALIGN, dict(k_rope=A + 8)), (ALIGN, dict(cu_new=A + 1)),
    (ALIGN, dict(inv_freq=A + 4)), (CP, dict(cp=2, kv_ptrs=[A, A], scale_ptrs=[A, 2 * A])),
    (CP, dict(cp=3, kv_ptrs=[A, None, 2 * A], scale_ptrs=[A, None, A]))])
def test_append(code, change):
    refused(code, dcp.dcp_mla_cache8_append, APPEND, **change)


@pytest.mark.parametrize("code,change", SHARDS + [
    (SHAPE, dict(N=-1)), (SHAPE, dict(cu=None, N=3)), (SHAPE, dict(B=0)), (DTYPE, dict(dtype=5)), (NULL, dict(out=None)),
    (ALIGN, dict(out=A + 8)), (ALIGN, dict(out_row=580)), (ALIGN, dict(starts=A + 2))])
def test_read(code, change):
    refused(code, dcp.dcp_mla_cache8_read, READ, **change)


@pytest.mark.parametrize("code,change", SHARDS + [
    (SHAPE, dict(H=0)), (SHAPE, dict(H=1025)), (SHAPE, dict(Dv=256)), (SHAPE, dict(B=65535, T=(1 << 31) - 1)),
    (WINDOW, dict(window=-1)), (WINDOW, dict(sinks=-1, window=4)), (WINDOW, dict(sinks=4)), (FLAGS, dict(flags=2)),
    (NULL, dict(q=None)), (NULL, dict(out=None)), (NULL, dict(seq_lens=None)), (ALIGN, dict(q=A + 2)),
    (ALIGN, dict(q_row=577)), (ALIGN, dict(q_head=577)), (ALIGN, dict(out=A + 8)), (ALIGN, dict(lse=A + 2)),
    (ALIGN, dict(status=A + 2))])
def test_decode(code, change):
    refused(code, dcp.dcp_mla_cache8_decode, DECODE, **change)


def test_decode_of_no_rows_is_nothing():
    dcp.dcp_mla_cache8_decode(**{**DECODE, "B": 0, "workspace": None})
    dcp.dcp_mla_cache8_decode(**{**DECODE, "B": 0, "flags": dcp.DCP_FLAG_PDL | dcp.DCP_MLA_FLAG_TEST_STALL})


def test_decode_of_no_rows_takes_null_for_what_rows_have():
    """As empty tensors give it; what is wrong besides is refused all the same."""
    empty = {**DECODE, "B": 0, "q": None, "seq_lens": None, "out": None, "lse": None, "workspace": None}
    dcp.dcp_mla_cache8_decode(**empty)
    refused(WINDOW, dcp.dcp_mla_cache8_decode, empty, sinks=4)
    refused(NULL, dcp.dcp_mla_cache8_decode, empty, kv_ptrs=[None], scale_ptrs=[None])


def test_workspace_bytes():
    ws = dcp.dcp_mla_cache8_decode_workspace_bytes
    assert ws(1, 8, 128, 4096, 0, 0, 152) >= 2 * 152 * 64 * 513 * 4
    assert ws(1, 65535, 1024, 4096, 0, 0, 152) >= 2 * 144 * 64 * 513 * 4 + 65535 * 8  # 16 head blocks x 9 ranges
    # at most two tiles of 128 tokens a row: no row is split
    for cp, T, window, sinks, none in ((1, 256, 0, 0, True), (1, 257, 0, 0, False), (2, 128, 0, 0, True),
                                       (3, 100, 0, 0, False), (1, 10 ** 6, 128, 4, True), (1, 10 ** 6, 129, 4, False),
                                       (1, 10 ** 6, 256, 0, True), (2, 10 ** 6, 128, 0, True), (1, 0, 0, 0, True)):
        assert (ws(cp, 4, 16, T, window, sinks, 152) == 0) == none
    for bad in ((0, 1, 16, 9, 0, 0, 152), (17, 1, 16, 9, 0, 0, 152), (1, -1, 16, 9, 0, 0, 152),
                (1, 65536, 16, 9, 0, 0, 152), (1, 1, 0, 9, 0, 0, 152), (1, 1, 1025, 9, 0, 0, 152),
                (1, 1, 16, -1, 0, 0, 152), (1, 1, 16, 9, -1, 0, 152), (1, 1, 16, 9, 0, 0, 0)):
        assert ws(*bad) == -1


def test_null_pointer_arrays():
    lib = dcp.load()
    one = (ctypes.c_void_p * 1)(A)
    assert lib.dcp_mla_cache8_read(None, one, 1, 1, 8, 576, 1, 1, None, None, 1, A, 576, 0, None) == NULL
    assert lib.dcp_mla_cache8_decode(A, 576, 576, one, None, A, 1, 1, 1, 576, 512, 8, 1, 1, 0, 0, 1.0, 1, A, 1 << 40,
                                     A, A, None, 0, None) == NULL


def test_messages():
    seen = {dcp.dcp_mla_cache8_strerror(c) for c in range(-210, -200)}
    assert len(seen) == 10
    assert dcp.dcp_mla_cache8_strerror(0) == "success"
    assert dcp.dcp_mla_cache8_strerror(-4) == dcp.dcp_lse_reduce_strerror(-4)


# ---- the torch wrappers -------------------------------------------------------------


def cache(B=2, T=8, dk=576, block=1, dtype=torch.float8_e4m3fn):
    return torch.zeros((B, T, dk), dtype=torch.uint8).view(dtype), torch.ones((B, -(-T // block)))


def test_wrappers_need_cuda_tensors():
    kv, sc = cache()
    lens = torch.zeros((2,), dtype=torch.int32)
    freq, _ = dcp.mla_rope_inv_freq(64, device="cpu")
    x = torch.zeros((2, 3, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dcp.mla_rope(x, torch.zeros((2,), dtype=torch.int64), freq)
    with pytest.raises(ValueError, match="CUDA"):
        dcp.mla_cache8_append(torch.zeros((2, 512), dtype=torch.bfloat16), torch.zeros((2, 64), dtype=torch.bfloat16),
                              [kv], [sc], lens)
    with pytest.raises(ValueError, match="CUDA"):
        dcp.mla_cache8_read([kv], [sc], 2)
    with pytest.raises(ValueError, match="CUDA"):
        dcp.mla_cache8_decode(torch.zeros((2, 4, 576), dtype=torch.bfloat16), [kv], [sc], lens, 1.0)


def test_wrappers_check_shards():
    kv, sc = cache()
    read = lambda c, s, **k: dcp.mla_cache8_read(c, s, 2, **k)
    for c, s, k in [([], [], {}), ([kv], [sc, sc], {}), ([None], [None], {}), ([kv, None], [sc, sc], {}),
                    ([kv], [sc], dict(block=3)), ([kv], [sc], dict(block=2)), ([kv], [sc], dict(block=0)),
                    ([kv, cache(T=9)[0]], [sc, cache(T=9)[1]], {}), ([kv[:, ::2]], [sc[:, ::2]], {}),
                    ([kv[..., :500]], [sc], {}), ([kv] * 17, [sc] * 17, {})]:
        with pytest.raises(ValueError):
            read(c, s, **k)
    for c, s in [([kv.view(torch.uint8).float()], [sc]), ([kv], [sc.double()]),
                 ([kv.view(torch.uint8).view(torch.float8_e5m2)], [sc])]:
        with pytest.raises(TypeError):
            read(c, s)
    for il in (0, (1 << 24) + 1, (1 << 32) + 1):
        with pytest.raises(ValueError):
            read([kv], [sc], interleave=il)
    with pytest.raises(ValueError):
        dcp.mla_cache8_read([kv], [sc], -1)
    with pytest.raises(TypeError):
        read([kv], [sc], dtype=torch.float64)
    with pytest.raises(ValueError):
        read([kv], [sc], starts=torch.zeros((3,), dtype=torch.int32))
    with pytest.raises(ValueError):
        read([kv], [sc], cu=torch.zeros((3,), dtype=torch.int64))


def test_wrappers_check_the_rest():
    kv, sc = cache()
    lens = torch.zeros((2,), dtype=torch.int32)
    freq, _ = dcp.mla_rope_inv_freq(64, device="cpu")
    lat, pe = torch.zeros((2, 512), dtype=torch.bfloat16), torch.zeros((2, 64), dtype=torch.bfloat16)
    kv5, sc5 = cache(dk=512)
    for args, kw in [((lat[:, :500], pe), {}), ((lat, None), {}), ((lat, pe[:1]), {}), ((lat, pe.half()), {}),
                     ((lat, pe), dict(inv_freq=freq.float())), ((lat, pe), dict(inv_freq=freq[:16])),
                     ((lat, pe), dict(cu_new=lens)), ((lat.T.contiguous().T, pe), {})]:
        with pytest.raises(ValueError):
            dcp.mla_cache8_append(*args, [kv], [sc], lens, **kw)
    with pytest.raises(TypeError):
        dcp.mla_cache8_append(lat.float(), pe.float(), [kv], [sc], lens)
    with pytest.raises(ValueError):
        dcp.mla_cache8_append(lat, pe, [kv], [sc], None)
    with pytest.raises(ValueError):
        dcp.mla_cache8_append(lat, pe, [kv5], [sc5], lens)
    with pytest.raises(ValueError):
        dcp.mla_cache8_append(lat, None, [kv5], [sc5], lens, inv_freq=freq)
    q = torch.zeros((2, 4, 576), dtype=torch.bfloat16)
    for bad in (q.float(), q[:1], q[..., :512], q[0], q.transpose(1, 2)):
        with pytest.raises(ValueError):
            dcp.mla_cache8_decode(bad, [kv], [sc], lens, 1.0)
    with pytest.raises(ValueError):
        dcp.mla_cache8_decode(q, [kv], [sc], None, 1.0)
    for kw in (dict(window=-1), dict(window=1 << 64), dict(window=4, sinks=-1), dict(window=4, sinks=1 << 63)):
        with pytest.raises(ValueError, match="window"):
            dcp.mla_cache8_decode(q, [kv], [sc], lens, 1.0, **kw)
    x, pos = torch.zeros((2, 3, 64)), torch.zeros((2,), dtype=torch.int64)
    for start in (-1, 65, 1 << 32):
        with pytest.raises(ValueError, match="start"):
            dcp.mla_rope(x, pos, freq, start=start)
    for a in ((x[0], pos, freq), (x, pos[:1], freq), (x, pos.float(), freq), (x, pos, freq.float()),
              (x.transpose(1, 2), pos, freq)):
        with pytest.raises(ValueError):
            dcp.mla_rope(*a)
    with pytest.raises(TypeError):
        dcp.mla_rope(x.double(), pos, freq)


@pytest.mark.parametrize("kw", [dict(rot=63), dict(rot=0), dict(base=0.0), dict(factor=0.5), dict(scaling="ntk"),
                                dict(scaling="yarn", base=1.0), dict(original_len=0)])
def test_inv_freq_refusals(kw):
    with pytest.raises(ValueError):
        dcp.mla_rope_inv_freq(**{"device": "cpu", **kw})


def test_inv_freq_values():
    f, amp = dcp.mla_rope_inv_freq(64, device="cpu")
    assert f.dtype == torch.float64 and amp == 1.0 and f[0] == 1.0
    assert torch.allclose(f, 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32), rtol=1e-15, atol=0)
    y, amp = dcp.mla_rope_inv_freq(64, scaling="yarn", factor=40.0, mscale=1.0, mscale_all_dim=1.0, device="cpu")
    assert amp == 1.0 and (y <= f).all() and (y >= f / 40 * (1 - 1e-15)).all() and (y[:-1] > y[1:]).all()


@pytest.mark.parametrize("n,h,d,x,out", [
    # offset and strides of two views of one buffer
    (3, 2, 4, (0, 8, 4), (4, 8, 4)), (3, 2, 4, (0, 16, 8), (4, 16, 8)), (3, 2, 4, (0, 16, 8), (3, 16, 8)),
    (3, 2, 4, (0, 16, 8), (5, 16, 8)), (3, 2, 4, (20, 16, 8), (0, 16, 8)), (3, 2, 4, (0, 16, 8), (44, 16, 8)),
    (3, 2, 4, (0, 16, 8), (43, 16, 8)), (1, 2, 4, (0, 5, 12), (4, 3, 12)), (1, 2, 4, (0, 5, 12), (4, 3, 8)),
    (1, 1, 4, (0, 5, 12), (3, 3, 8)), (1, 1, 4, (0, 5, 12), (4, 3, 8)), (2, 3, 4, (0, 4, 8), (24, 4, 8)),
    (2, 3, 4, (0, 4, 8), (8, 4, 8)), (2, 3, 4, (50, 4, 8), (8, 4, 8)), (4, 1, 4, (0, 10, 0), (6, 10, 0)),
    (4, 1, 4, (0, 10, 0), (7, 10, 0)), (2, 2, 4, (0, 0, 8), (4, 8, 16))])
def test_overlaps_of_rotated_views(n, h, d, x, out):
    """Views that share an element are always found; views that do not are let through where they are different dims of
    the same heads, or lie apart."""
    from decode_context_mla_dcp_gb300 import cache8
    elems = lambda v: {v[0] + i * v[1] + j * v[2] + k for i in range(n) for j in range(h) for k in range(d)}
    said = cache8._meet(out[0] - x[0], n, h, d, *x[1:], *out[1:])
    a, b = elems(x), elems(out)
    if a & b:
        assert said
    elif x[1:] == out[1:] or max(a) < min(b) or max(b) < min(a):
        aside = n > 1 and h > 1 and x[1] < x[2]  # (heads outside rows: told apart only where the spans are)
        assert not said or aside


@pytest.mark.parametrize("n,h,d,row,head", [
    (4, 2, 64, 0, 64), (4, 2, 64, 128, 0), (1, 2, 64, 0, 64), (4, 1, 64, 64, 0), (1, 1, 64, 0, 0), (4, 2, 64, 64, 64),
    (4, 2, 64, 128, 64), (2, 4, 64, 64, 128), (4, 2, 64, 63, 256), (4, 2, 64, 64, 256), (4, 2, 64, 64, 255),
    (3, 2, 4, 8, 12), (2, 3, 4, 12, 8), (2, 2, 4, 12, 8), (2, 3, 4, 13, 8), (3, 3, 4, 20, 8), (3, 3, 4, 16, 8),
    (3, 3, 4, 19, 8), (2, 5, 3, 7, 10), (5, 2, 3, 7, 10), (5, 5, 3, 7, 10), (4, 4, 1, 3, 4), (3, 4, 1, 4, 3),
    (5, 4, 1, 4, 3), (0, 2, 4, 0, 4), (6, 7, 2, 11, 13), (12, 12, 2, 11, 13), (14, 12, 2, 11, 13)])
def test_rows_and_heads_that_share_elements(n, h, d, row, head):
    from decode_context_mla_dcp_gb300 import cache8
    places = [i * row + j * head + k for i in range(n) for j in range(h) for k in range(d)]
    assert cache8._folded(n, h, d, row, head) == (len(set(places)) < len(places))


def test_rope_in_place_refuses_what_repeats_rows_or_heads():
    """Every CTA would turn the same elements again: refused before anything looks at the device."""
    freq, _ = dcp.mla_rope_inv_freq(64, device="cpu")
    pos = torch.zeros((4,), dtype=torch.int64)
    base = torch.zeros((400,))
    for x in (torch.zeros((1, 2, 64)).expand(4, 2, 64), torch.zeros((4, 1, 64)).expand(4, 2, 64),
              base.as_strided((4, 2, 64), (32, 192, 1)), base.as_strided((4, 2, 64), (64, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            dcp.mla_rope(x, pos, freq, out=x)
    for x in (base.as_strided((1, 2, 64), (0, 64, 1)), base.as_strided((4, 1, 64), (64, 0, 1))):
        with pytest.raises(ValueError, match="CUDA"):  # (these share nothing: what is wrong is the device)
            dcp.mla_rope(x, pos[:x.shape[0]], freq, out=x)
