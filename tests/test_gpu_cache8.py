"""The 8-bit cache's operators against their plain 64-bit forms (oracle/cache8.py).

Tolerances, derived:
* rotary: fp32 arithmetic on two products, angles good to 2^-22 (the fp32 rounding of the half-turn and sincospi's
  two units): 2^-20 (|a| + |b|) |mscale|, plus half a step of the output's type.
* codes: the nearest e4m3 number. The latent part is exact arithmetic; a rotated key carries 2^-20 of its pair, which
  can move a value across a rounding boundary: within half a step of the code plus that.
* attention: a probability keeps 2^-8 of itself (two e4m3 parts: half a step of 2^-4 of half a step of 2^-4) and what
  lies below 2^-18 of its 32-token block's largest; the output half a step of bf16. Scores are fp32 sums of exact
  products: 2^-21 of the sum of their magnitudes. q's head is scaled so that its largest lies in (224, 448]; a bf16 is two
  e4m3 numbers exactly if its last bit is at least e4m3's smallest step, 2^-9: from 2^-2 up, which is 2^-2 / 224 < 2^-9 of
  the largest. Below that each of the two parts errs by at most half that step: 2 * 2^-10 / 224 < 2^-16 of the largest.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from oracle import cache8 as ref
from .conftest import record_error

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SCALE = 192 ** -0.5


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


# ---- rotary positions ------------------------------------------------------------


def check_rope(x, pos, inv_freq, start, interleaved, mscale, got):
    half = inv_freq.shape[0]
    x64 = x.double()
    want = ref.rotate(x64, pos, inv_freq, start, interleaved, mscale)
    if interleaved:
        pair = x64[..., start:start + 2 * half].abs().unflatten(-1, (half, 2)).sum(-1).repeat_interleave(2, -1)
    else:
        a = x64[..., start:start + 2 * half].abs()
        pair = (a[..., :half] + a[..., half:]).repeat(1, 1, 2)
    tol = HALF_STEP[x.dtype] * want.abs() * (1 + 2.0 ** -10)
    tol[..., start:start + 2 * half] += 2.0 ** -20 * pair * abs(mscale)
    tol[..., :start], tol[..., start + 2 * half:] = 0, 0  # dims that are not rotated are copied
    tiny = 2.0 ** -24 if x.dtype == torch.float16 else 0.0  # fp16 subnormals
    assert ((got.double() - want).abs() <= tol + tiny).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,h,d,start,rot", [
    (1, 1, 64, 0, 64), (1, 16, 64, 0, 64), (3, 128, 576, 512, 64), (17, 5, 192, 128, 64), (129, 7, 96, 16, 32),
    (5, 3, 71, 3, 30), (33, 2, 2, 0, 2), (2, 4, 256, 0, 256), (700, 1, 64, 0, 64), (2, 3, 300, 7, 250),
    (3, 65, 130, 64, 64)])
def test_rope(dtype, interleaved, n, h, d, start, rot):
    g = gen(n * 1000 + d)
    x = randn(g, n, h, d).to(dtype)
    inv_freq, _ = dcp.mla_rope_inv_freq(rot)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device=DEV)
    got = dcp.mla_rope(x, pos, inv_freq, start=start, interleaved=interleaved, mscale=0.9)
    check_rope(x, pos, inv_freq, start, interleaved, 0.9, got)
    # in place, 32-bit positions: the same bits
    y = x.clone()
    assert dcp.mla_rope(y, pos.int(), inv_freq, start=start, interleaved=interleaved, mscale=0.9, out=y) is y
    assert torch.equal(y, got)


@pytest.mark.parametrize("seed", range(24))
def test_rope_random(seed):
    """Random sizes, types, strides and places: into a new tensor, in place, or into a view of a wider one."""
    import random
    r = random.Random(seed)
    g = gen(seed)
    dtype = r.choice([torch.bfloat16, torch.bfloat16, torch.float16, torch.float32])
    rot = r.choice([2, 6, 32, 64, 128, 256])
    start, h = r.choice([0, 0, 8, 30, 128]), r.choice([1, 1, 2, 3, 7, 16, 40, 128])
    d = start + rot + r.choice([0, 0, 8, 5])
    n = min(r.choice([1, 2, 9, 100, 700, 5000]), max(1, 400000 // (h * d)))
    pad, lead = r.choice([0, 0, 8, 3]), r.choice([0, 0, 16, 1])
    buf = randn(g, n, h, lead + d + pad).to(dtype)
    if r.random() < 0.3:  # heads outside tokens
        buf = randn(g, h, n, lead + d + pad).to(dtype).transpose(0, 1)
    x = buf[..., lead:lead + d]
    pos = torch.randint(-1000, 200000, (n,), generator=g, device=DEV, dtype=r.choice([torch.int32, torch.int64]))
    inv_freq, _ = dcp.mla_rope_inv_freq(rot)
    kw = dict(start=start, interleaved=r.random() < 0.5, mscale=r.choice([1.0, 1.37]))
    x0, whole = x.clone(), buf.clone()
    how = r.choice(["new", "place", "view"])
    if how == "new":
        got = dcp.mla_rope(x, pos, inv_freq, **kw)
        assert torch.equal(buf, whole)
    elif how == "place":
        got = dcp.mla_rope(x, pos, inv_freq, out=x, **kw)
        assert torch.equal(buf[..., :lead], whole[..., :lead]) and torch.equal(buf[..., lead + d:], whole[..., lead + d:])
    else:
        other = torch.full((n, h, d + 24), 5.0, dtype=dtype, device=DEV)
        got = dcp.mla_rope(x, pos, inv_freq, out=other[..., 8:8 + d], **kw)
        assert (other[..., :8] == 5).all() and (other[..., 8 + d:] == 5).all()
    check_rope(x0, pos, inv_freq, start, kw["interleaved"], kw["mscale"], got)


def test_rope_far_and_negative_positions():
    x = randn(gen(0), 6, 4, 64)
    pos = torch.tensor([0, -1, (1 << 31) - 1, -(1 << 30), 10 ** 6 + 1, 163839], device=DEV)
    inv_freq, _ = dcp.mla_rope_inv_freq(64)
    for il in (True, False):
        check_rope(x, pos, inv_freq, 0, il, 1.0, dcp.mla_rope(x, pos, inv_freq, interleaved=il))


@pytest.mark.parametrize("scaling", ["linear", "yarn"])
def test_rope_scaled_frequencies(scaling):
    x = randn(gen(1), 9, 3, 64).bfloat16()
    pos = torch.arange(9, device=DEV) * 20011
    f, amp = dcp.mla_rope_inv_freq(64, scaling=scaling, factor=40.0)
    plain = dcp.mla_rope_inv_freq(64)[0]
    assert torch.allclose(f[-1] * 40, plain[-1], rtol=1e-14, atol=0)
    assert (f[0] == plain[0]) == (scaling == "yarn")
    assert amp == (pytest.approx(0.1 * math.log(40) + 1, abs=1e-15) if scaling == "yarn" else 1.0)
    check_rope(x, pos, f, 0, True, amp, dcp.mla_rope(x, pos, f, mscale=amp))


@pytest.mark.parametrize("n,h", [(1, 3), (7, 40), (2000, 1)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_of_frequencies_that_are_not_finite(n, h, interleaved):
    """Their pairs are NaN, in the appended cache too; the other pairs keep their bits."""
    g = gen(n)
    x, latent = randn(g, n, h, 64).bfloat16(), randn(g, n, 512).bfloat16()
    pos = torch.arange(n, device=DEV) + 5
    good, _ = dcp.mla_rope_inv_freq(64)
    bad = good.clone()
    bad[3], bad[10], bad[31] = math.nan, math.inf, -math.inf
    pairs = torch.arange(64, device=DEV)
    odd = torch.isin(pairs // 2 if interleaved else pairs % 32, torch.tensor([3, 10, 31], device=DEV))
    want = dcp.mla_rope(x, pos, good, interleaved=interleaved)
    got = dcp.mla_rope(x, pos, bad, interleaved=interleaved)
    assert got[..., odd].isnan().all() and torch.equal(got[..., ~odd], want[..., ~odd])
    for block in (1, 16):
        kv, sc = blank(1, 1, n + 5, 576, block)
        lens = torch.full((1,), 5, dtype=torch.int32, device=DEV)
        dcp.mla_cache8_append(latent, x[:, 0], kv, sc, lens, block=block, inv_freq=bad, interleaved=interleaved)
        codes = kv[0][0, 5:].float()
        assert codes[:, 512:][:, odd].isnan().all() and not codes[:, :512].isnan().any()
        assert not codes[:, 512:][:, ~odd].isnan().any()


def test_rope_into_a_view_leaves_the_rest():
    g = gen(2)
    buf = randn(g, 7, 12, 576).bfloat16()
    before = buf.clone()
    x = randn(g, 12, 7, 64).bfloat16().transpose(0, 1)  # heads first in memory
    pos = torch.randint(0, 5000, (7,), generator=g, device=DEV)
    inv_freq, _ = dcp.mla_rope_inv_freq(64)
    dcp.mla_rope(x, pos, inv_freq, out=buf[..., 512:])
    assert torch.equal(buf[..., :512], before[..., :512])
    check_rope(x, pos, inv_freq, 0, True, 1.0, buf[..., 512:])
    # an odd offset: the unaligned form
    buf2 = before.clone()
    dcp.mla_rope(x, pos, inv_freq, out=buf2[..., 3:67])
    assert torch.equal(buf2[..., 3:67], buf[..., 512:])
    assert torch.equal(buf2[..., :3], before[..., :3]) and torch.equal(buf2[..., 67:], before[..., 67:])


def test_rope_refuses_overlaps():
    x = torch.zeros((4, 2, 64), device=DEV)
    pos = torch.zeros((4,), dtype=torch.int32, device=DEV)
    inv_freq, _ = dcp.mla_rope_inv_freq(32)
    whole = torch.zeros((4, 2, 128), device=DEV)
    dcp.mla_rope(whole[..., :64], pos, inv_freq, out=whole[..., 64:])  # other dims of the same heads
    for out in (x.expand(4, 2, 64)[:1].expand(4, 2, 64), torch.zeros((4, 1, 64), device=DEV).expand(4, 2, 64),
                torch.zeros((400,), device=DEV).as_strided((4, 2, 64), (64, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            dcp.mla_rope(x, pos, inv_freq, out=out)
    with pytest.raises(ValueError, match="overlap"):
        dcp.mla_rope(whole[..., :64], pos, inv_freq, out=whole[..., 32:96])
    big = torch.zeros((5, 2, 64), device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        dcp.mla_rope(big[:4], pos, inv_freq, out=big[1:])
    heads_first = torch.zeros((2, 4, 64), device=DEV)
    assert dcp.mla_rope(x, pos, inv_freq, out=heads_first.transpose(0, 1)).data_ptr() == heads_first.data_ptr()


def test_rope_of_nothing():
    inv_freq, _ = dcp.mla_rope_inv_freq(64)
    x = torch.empty((0, 4, 64), device=DEV)
    assert dcp.mla_rope(x, torch.empty((0,), dtype=torch.int64, device=DEV), inv_freq).shape == (0, 4, 64)


# ---- the cache -----------------------------------------------------------------


def blank(cp, B, T, dk, block, seed=0, dtype=E4M3):
    """Caches filled with finite codes and power-of-two scales, as earlier contents."""
    g = gen(seed)
    kv = [(randn(g, B, T, dk) * 100).clamp(-448, 448).to(E4M3) for _ in range(cp)]
    sc = [torch.exp2(torch.randint(-8, 3, (B, -(-T // block)), generator=g, device=DEV).float()) for _ in range(cp)]
    return kv, sc


def bits(x):
    return x.view(torch.uint8)


APPENDS = [
    # B, counts, starts, cp, interleave, block, T, dk, dtype, interleaved, rotate
    (1, [1], [0], 1, 1, 1, 5, 576, torch.bfloat16, True, True),
    (1, [1], [6], 1, 1, 4, 7, 576, torch.bfloat16, True, True),
    (3, [4, 0, 9], [3, 5, 0], 1, 1, 1, 20, 576, torch.float16, False, True),
    (3, [4, 0, 9], [3, 5, 0], 1, 1, 8, 20, 576, torch.bfloat16, False, True),
    (4, [1, 1, 1, 1], [0, 15, 16, 17], 1, 1, 16, 33, 576, torch.bfloat16, True, False),
    (2, [131, 64], [1, 127], 1, 1, 128, 250, 576, torch.bfloat16, True, True),
    (2, [70, 200], [63, 1], 1, 1, 64, 210, 576, torch.float16, True, True),
    (2, [70, 33], [31, 1], 1, 1, 32, 110, 512, torch.bfloat16, True, False),
    (3, [40, 7, 1], [3, 0, 50], 2, 1, 1, 30, 576, torch.bfloat16, True, True),
    (3, [40, 7, 1], [3, 0, 50], 4, 1, 2, 30, 576, torch.bfloat16, True, True),
    (2, [90, 5], [13, 44], 3, 5, 16, 40, 576, torch.bfloat16, True, True),
    (2, [300, 17], [13, 100], 4, 16, 64, 90, 576, torch.bfloat16, False, True),
    (2, [20, 20], [13, 40], 2, 1, 8, 12, 576, torch.bfloat16, True, True),  # past the cache's end
    (5, [2, 3, 1, 4, 2], [9, 0, 31, 30, 2], 1, 1, 32, 40, 512, torch.float16, True, False),
]


def loud(g, n, width, dtype):
    """Tokens of very different sizes: some blocks grow, some do not."""
    return (randn(g, n, width) * torch.exp2(torch.randint(-9, 9, (n, 1), generator=g, device=DEV).float())).to(dtype)


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"B{c[0]}cp{c[3]}i{c[4]}b{c[5]}T{c[6]}d{c[7]}")
def test_append(case):
    B, counts, starts, cp, il, block, T, dk, dtype, inter, rot = case
    g = gen(len(str(case)))
    n = sum(counts)
    kv, sc = blank(cp, B, T, dk, block, seed=n)
    values, scales = [x.double() for x in kv], [x.double() for x in sc]
    latent = loud(g, n + 2, 512, dtype)
    rope = loud(g, n + 2, 64, dtype) if dk == 576 else None
    inv_freq = dcp.mla_rope_inv_freq(64)[0] if rot else None
    cu = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
    lens = torch.tensor(starts, device=DEV, dtype=torch.int32)
    pos = torch.cat([torch.arange(s, s + c, device=DEV) for s, c in zip(starts, counts)])
    x = latent[:n].double()
    slack = torch.zeros((n, dk), dtype=torch.float64, device=DEV)
    if dk == 576:
        k = rope[:n, None].double()
        if rot:
            slack[:, 512:] = 2.0 ** -20 * k[:, 0].abs().amax(1, keepdim=True) * 2
            k = ref.rotate(k, pos, inv_freq, 0, inter, 1.25)
        x = torch.cat((x, k[:, 0]), 1)
    ref.append(x, counts, starts, values, scales, cp, il, block)
    dcp.mla_cache8_append(latent, rope, kv, sc, lens, cu_new=cu, block=block, interleave=il, inv_freq=inv_freq,
                          interleaved=inter, mscale=1.25)
    # (two packed tokens behind cu[B] go nowhere)
    token = 0
    mine = [torch.zeros((B, T), dtype=torch.bool, device=DEV) for _ in range(cp)]
    for b in range(B):
        for i in range(counts[b]):
            j, t = ref.place(starts[b] + i, cp, il)
            if t < T:
                mine[j][b, t] = True
                s = float(sc[j][b, t // block])
                step = torch.exp2((torch.frexp(values[j][b, t].abs())[1] - 1).clamp(min=-6).double() - 3)
                err = (kv[j][b, t].double() - x[token] / s).abs()
                assert (err <= step / 2 + slack[token] / s).all()
            token += 1
    for j in range(cp):
        assert torch.equal(sc[j].double(), scales[j])
        same = kv[j].double() == values[j]
        same |= mine[j][..., None] & (torch.arange(dk, device=DEV) >= 512)  # checked above, to a rounding
        assert same.all()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("block", [1, 64])
def test_append_rotates_to_the_last_places(interleaved, block):
    """Codes of rotated keys lie within half a step and 2^-22 of the pair of the 64-bit value. In units of 2^-24 of the
    pair: the angle 0.41 (2^-27 of a half turn), sine and cosine 1, the factor 0.5, the products and their sum 1."""
    g = gen(block)
    n, mscale = 60000, 1.25
    latent, rope = randn(g, n, 512).bfloat16(), (3 * randn(g, n, 64)).bfloat16()
    inv_freq, _ = dcp.mla_rope_inv_freq(64)
    kv, sc = blank(1, 1, n + 5, 576, block)
    lens = torch.full((1,), 5, dtype=torch.int32, device=DEV)
    sc[0][0, 0] = 1.0
    dcp.mla_cache8_append(latent, rope, kv, sc, lens, block=block, inv_freq=inv_freq, interleaved=interleaved,
                          mscale=mscale)
    x = rope[:, None].double()
    want = ref.rotate(x, torch.arange(5, n + 5, device=DEV), inv_freq, 0, interleaved, mscale)[:, 0]
    a = x[:, 0].abs()
    pair = a.unflatten(-1, (32, 2)).sum(-1).repeat_interleave(2, -1) if interleaved else \
        (a[:, :32] + a[:, 32:]).repeat(1, 2)
    scale = sc[0][0, torch.arange(5, n + 5, device=DEV) // block].double()[:, None]
    codes = kv[0][0, 5:, 512:].double()
    step = torch.exp2((torch.frexp(want.abs() / scale)[1] - 1).clamp(min=-6).double() - 3)
    # (above a power of two the grid is coarser than below: the larger of the two steps where the code is one)
    step = torch.maximum(step, torch.exp2((torch.frexp(codes.abs())[1] - 1).clamp(min=-6).double() - 3))
    assert ((codes - want / scale).abs() <= step / 2 + 2.0 ** -22 * mscale * pair / scale).all()


def test_append_even_and_cu_agree_and_strides():
    g = gen(5)
    B, per, T = 6, 3, 64
    wide = randn(g, B * per, 1200).bfloat16()
    latent, rope = wide[:, 8:520], wide[:, 1024:1088]
    lens = torch.arange(B, device=DEV, dtype=torch.int32) * 7
    a, sa = blank(1, B, T, 576, 16)
    b, sb = [x.clone() for x in a], [x.clone() for x in sa]
    dcp.mla_cache8_append(latent, rope, a, sa, lens, block=16)
    cu = torch.arange(B + 1, device=DEV, dtype=torch.int32) * per
    dcp.mla_cache8_append(latent.contiguous(), rope.contiguous(), b, sb, lens, cu_new=cu, block=16)
    assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(sa[0], sb[0])


def test_append_token_by_token_equals_at_once_for_own_scales():
    g = gen(6)
    n, T = 23, 32
    latent, rope = randn(g, n, 512).bfloat16(), randn(g, n, 64).bfloat16()
    inv_freq, _ = dcp.mla_rope_inv_freq(64)
    a, sa = blank(2, 1, T, 576, 1)
    b, sb = [x.clone() for x in a], [x.clone() for x in sa]
    one = torch.zeros((1,), dtype=torch.int32, device=DEV)
    dcp.mla_cache8_append(latent, rope, a, sa, one, interleave=4, inv_freq=inv_freq)
    for i in range(n):
        dcp.mla_cache8_append(latent[i:i + 1], rope[i:i + 1], b, sb, one + i, interleave=4, inv_freq=inv_freq)
    for j in range(2):
        assert torch.equal(bits(a[j]), bits(b[j])) and torch.equal(sa[j], sb[j])


def test_append_a_block_that_grows_many_times():
    n, T, block = 40, 64, 32
    g = gen(7)
    latent = (randn(g, n, 512) * torch.exp2(torch.arange(n, device=DEV) * 0.7)[:, None]).bfloat16()
    kv, sc = blank(1, 1, T, 512, block)
    values, scales = [kv[0].double()], [sc[0].double()]
    lens = torch.zeros((1,), dtype=torch.int32, device=DEV)
    for i in range(n):
        dcp.mla_cache8_append(latent[i:i + 1], None, kv, sc, lens + i, block=block)
        ref.append(latent[i:i + 1].double(), [1], [i], values, scales, 1, 1, block)
    assert torch.equal(kv[0].double(), values[0]) and torch.equal(sc[0].double(), scales[0])


@pytest.mark.parametrize("block", [1, 8])
def test_append_nan_infinity_zero(block):
    latent = torch.zeros((8, 512), device=DEV, dtype=torch.bfloat16)
    rope = torch.zeros((8, 64), device=DEV, dtype=torch.bfloat16)
    latent[1, 3], latent[2, 4], rope[3, 5], latent[1, 9] = math.nan, math.inf, -math.inf, 2.0
    kv, sc = blank(1, 1, 8, 576, block)
    dcp.mla_cache8_append(latent, rope, kv, sc, torch.zeros((1,), dtype=torch.int32, device=DEV), block=block)
    v = kv[0].double()[0]
    assert v[1, 3].isnan() and v[2, 4].isnan() and v[3, 512 + 5].isnan() and int(v.isnan().sum()) == 3
    assert float(v[1, 9] * sc[0][0, 1 // block]) == 2.0
    assert float(sc[0][0, 7 // block]) == (2.0 ** -60 if block == 1 else 2.0 ** -7)
    assert int((v != 0).sum()) == 4


@pytest.mark.parametrize("block", [1, 16])
def test_append_skips_shards_that_are_not_held(block):
    g = gen(8)
    n, T, cp = 50, 40, 4
    latent, rope = randn(g, n, 512).bfloat16(), randn(g, n, 64).bfloat16()
    full, sf = blank(cp, 1, T, 576, block)
    part, sp = [x.clone() for x in full], [x.clone() for x in sf]
    lens = torch.full((1,), 5, dtype=torch.int32, device=DEV)
    dcp.mla_cache8_append(latent, rope, full, sf, lens, block=block, interleave=2)
    for j in range(cp):
        only = [part[k] if k == j else None for k in range(cp)]
        dcp.mla_cache8_append(latent, rope, only, [sp[k] if k == j else None for k in range(cp)], lens, block=block,
                              interleave=2)
    for j in range(cp):
        assert torch.equal(bits(part[j]), bits(full[j])) and torch.equal(sp[j], sf[j])


@pytest.mark.parametrize("B,cp,T", [(1500, 1, 8), (100, 2, 8), (100, 3, 8), (9, 1, 8)])
def test_append_many_rows_and_a_broken_cu(B, cp, T):
    """More rows than the shared copy of cu holds, and few; and offsets that a caller got wrong write nothing out of
    place."""
    g = gen(9)
    block = 4
    counts = [(i * 7) % 3 for i in range(B)]
    n = sum(counts)
    latent = randn(g, n, 512).bfloat16()
    kv, sc = blank(cp, B, T, 512, block)
    values, scales = [x.double() for x in kv], [x.double() for x in sc]
    starts = [i % 5 for i in range(B)]
    cu = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
    dcp.mla_cache8_append(latent, None, kv, sc, torch.tensor(starts, device=DEV, dtype=torch.int32), cu_new=cu,
                          block=block)
    ref.append(latent.double(), counts, starts, values, scales, cp, 1, block)
    for j in range(cp):
        assert torch.equal(kv[j].double(), values[j]) and torch.equal(sc[j].double(), scales[j])
    before = [bits(x).clone() for x in kv]
    for blk, scale in ((4, sc), (1, [torch.ones((B, T), device=DEV) for _ in range(cp)])):
        dcp.mla_cache8_append(latent, None, kv, scale, torch.full((B,), T * cp, device=DEV, dtype=torch.int32),
                              cu_new=cu, block=blk)
        dcp.mla_cache8_append(latent, None, kv, scale, torch.full((B,), -3 - T, device=DEV, dtype=torch.int32),
                              cu_new=torch.full((B + 1,), n + 5, device=DEV, dtype=torch.int32), block=blk)
        dcp.mla_cache8_append(latent, None, kv, scale, torch.full((B,), T * cp, device=DEV, dtype=torch.int32),
                              cu_new=torch.arange(B + 1, device=DEV, dtype=torch.int32).flip(0) - 3, block=blk)
    for j in range(cp):
        assert torch.equal(bits(kv[j]), before[j])


@pytest.mark.parametrize("B,cp,il,block", [(300, 2, 1, 32), (70, 4, 3, 64), (130, 2, 16, 128), (257, 1, 1, 2),
                                           (32, 8, 1, 16), (33, 8, 1, 16)])
def test_append_more_pairs_of_rows_and_shards(B, cp, il, block):
    """More than 256 pairs (256 themselves once), rows of no new token to several blocks, from inside a block on."""
    g = gen(B)
    T = 2 * block + 5
    counts = [(i * 13) % 5 if i % 11 else cp * block + i % 7 for i in range(B)]
    starts = [(i * 5) % (cp * T) for i in range(B)]
    n = sum(counts)
    latent = loud(g, n, 512, torch.bfloat16)
    kv, sc = blank(cp, B, T, 512, block)
    values, scales = [x.double() for x in kv], [x.double() for x in sc]
    cu = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
    dcp.mla_cache8_append(latent, None, kv, sc, torch.tensor(starts, device=DEV, dtype=torch.int32), cu_new=cu,
                          block=block, interleave=il)
    ref.append(latent.double(), counts, starts, values, scales, cp, il, block)
    for j in range(cp):
        assert torch.equal(kv[j].double(), values[j]) and torch.equal(sc[j].double(), scales[j])


@pytest.mark.parametrize("B,cp,il,block,n", [
    (5, 1, 1, 16, 1500), (300, 2, 3, 4, 1300), (512, 1, 1, 2, 1400), (513, 2, 1, 8, 1400), (40, 4, 16, 32, 900),
    (33, 16, 2, 64, 700), (3, 1, 1, 128, 500), (1, 5, 1, 16, 1218), (64, 3, 7, 16, 1217)])
def test_append_of_more_tokens_than_resident_ctas(B, cp, il, block, n):
    """Uneven rows, some of no tokens, that begin inside a block; a shard that is not held; rows that the cache has no
    room for; and offsets that a caller got wrong write nothing out of place."""
    g = gen(B + n)
    w = [(i * 29) % 7 if i % 6 else 40 for i in range(B)] if B > 1 else [1]
    counts = [n * x // sum(w) for x in w]
    counts[B // 2] += n - sum(counts)
    starts = [(i * 37) % 90 for i in range(B)]
    T = max(-(-(s + c) // cp) + 2 * il for s, c in zip(starts, counts)) - 9
    latent = loud(g, n, 512, torch.bfloat16)
    kv, sc = blank(cp, B, T, 512, block)
    values, scales = [x.double() for x in kv], [x.double() for x in sc]
    held = [j for j in range(cp) if cp == 1 or j != 1]
    only = lambda x: [x[j] if j in held else None for j in range(cp)]
    cu = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
    lens = torch.tensor(starts, device=DEV, dtype=torch.int32)
    dcp.mla_cache8_append(latent, None, only(kv), only(sc), lens, cu_new=cu, block=block, interleave=il)
    ref.append(latent.double(), counts, starts, values, scales, cp, il, block, held)
    for j in range(cp):
        assert torch.equal(kv[j].double(), values[j]) and torch.equal(sc[j].double(), scales[j])
    before = [bits(x).clone() for x in kv]
    full = torch.full((B,), T * cp + cp * il, device=DEV, dtype=torch.int32)
    for bad in (cu, torch.full((B + 1,), n + 5, device=DEV, dtype=torch.int32), cu.flip(0) - 3, -cu):
        dcp.mla_cache8_append(latent, None, kv, sc, full, cu_new=bad.contiguous(), block=block, interleave=il)
    for j in range(cp):
        assert torch.equal(bits(kv[j]), before[j])


@pytest.mark.parametrize("block", [1, 64])
def test_a_cache_whose_offsets_pass_32_bits(block):
    """Two rows of 4.3 GB: append, read back and attend behind 2^32 bytes and at the end of the last row."""
    g = gen(12)
    B, T, n, window = 2, 7_500_000, 300, 290
    kv = [torch.zeros((B, T, 576), dtype=torch.uint8, device=DEV).view(E4M3)]
    sc = [torch.ones((B, -(-T // block)), device=DEV)]
    starts = torch.tensor([T - n - 17, T - n], dtype=torch.int32, device=DEV)
    latent, rope = randn(g, B * n, 512).bfloat16(), randn(g, B * n, 64).bfloat16()
    dcp.mla_cache8_append(latent, rope, kv, sc, starts, block=block)
    got = dcp.mla_cache8_read(kv, sc, B * n, starts=starts, block=block, dtype=torch.float32)
    x = torch.cat((latent, rope), 1).double()
    for b in range(B):
        rows = slice(int(starts[b]), int(starts[b]) + n)
        scale = sc[0][b, torch.arange(rows.start, rows.stop, device=DEV) // block].double()[:, None]
        mine = x[b * n:(b + 1) * n]
        assert torch.equal(got[b * n:(b + 1) * n].double(), kv[0][b, rows].double() * scale)
        assert ((got[b * n:(b + 1) * n].double() - mine).abs() <=
                torch.maximum(2.0 ** -4 * mine.abs(), 2.0 ** -10 * scale)).all()
        assert (kv[0][b, rows.start - 5:rows.start].view(torch.uint8) == 0).all()
    q = randn(g, B, 16, 576).bfloat16()
    lens = starts + n
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=block, window=window)
    first = (T - 600) // 128 * 128  # the same rows in a short cache (whole blocks of it)
    short = [kv[0][:, first:].contiguous()]
    short_sc = [sc[0][:, first // block:].contiguous()]
    again = dcp.mla_cache8_decode(q, short, short_sc, lens - first, SCALE, block=block, window=window)
    check_decode(q, short, short_sc, lens - first, SCALE, 1, 1, block, window, 0, *again)
    check_decode(q, short, short_sc, lens - first, SCALE, 1, 1, block, window, 0, out, lse)


# ---- read-back --------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cp,il,block,T,dk,counts,starts", [
    (1, 1, 1, 9, 576, [1], [8]), (1, 1, 16, 50, 512, [50, 0, 13], [0, 3, 20]), (3, 4, 8, 40, 576, [100, 7, 1], [3, 60, 0]),
    (2, 1, 128, 300, 576, [500, 555], [77, 40]), (16, 1, 2, 10, 576, [150], [5])])
def test_read(dtype, cp, il, block, T, dk, counts, starts):
    B, n = len(counts), sum(counts)
    kv, sc = blank(cp, B, T, dk, block, seed=T)
    sc = [s * 1.3 for s in sc]  # any positive scale
    cu = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
    held = [j for j in range(cp) if cp == 1 or j != 1]
    out = torch.full((n + 1, dk + 8), 7.0, dtype=dtype, device=DEV)
    view = out[:, :dk]
    got = dcp.mla_cache8_read([kv[j] if j in held else None for j in range(cp)],
                              [sc[j] if j in held else None for j in range(cp)], n + 1,
                              starts=torch.tensor(starts, device=DEV, dtype=torch.int32), cu=cu, block=block,
                              interleave=il, out=view)
    assert got is view
    values, scales = [x.double() for x in kv], [x.double() for x in sc]
    at = 0
    for b in range(B):
        if counts[b]:
            want, ok = ref.gather(values, scales, b, range(starts[b], starts[b] + counts[b]), cp, il, block, held)
            want[~torch.tensor(ok, device=DEV)] = 7.0
            w = got[at:at + counts[b]].double()
            assert ((w - want).abs() <= (HALF_STEP[dtype] + 2.0 ** -24) * want.abs() +
                    (2.0 ** -25 if dtype == torch.float16 else 0)).all()
        at += counts[b]
    assert (out[n] == 7).all() and (out[:, dk:] == 7).all()


def test_read_of_what_was_appended():
    g = gen(11)
    n, T = 77, 64
    latent, rope = randn(g, n, 512).bfloat16(), randn(g, n, 64).bfloat16()
    kv, sc = blank(2, 1, T, 576, 1)
    dcp.mla_cache8_append(latent, rope, kv, sc, torch.zeros((1,), dtype=torch.int32, device=DEV))
    x = torch.cat((latent, rope), 1).double()
    got = dcp.mla_cache8_read(kv, sc, n, dtype=torch.float32).double()
    peak = x.abs().amax(1, keepdim=True)
    # half a step of e4m3, or of its subnormals (2^-10 of a scale that is at most 2 / 448 of the peak)
    assert ((got - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * peak * 2 / 448)).all()


# ---- attention ----------------------------------------------------------------------


def check_decode(q, kv, sc, lens, scale, cp, il, block, window, sinks, out, lse, base_e=True, held=None, rows=None):
    values, scales = [x.double() for x in kv], [x.double() for x in sc]
    T = kv[0].shape[1]
    st_v, st_s = torch.stack(values), torch.stack(scales)
    for b in (range(q.shape[0]) if rows is None else rows):
        pos = [p for p in ref.visible(min(max(int(lens[b]), 0), 16 * T * cp + 99), window, sinks)
               if ref.place(p, cp, il)[1] < T and (held is None or ref.place(p, cp, il)[0] in held)]
        qb = q[b].double()
        if not pos:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        j = torch.tensor([ref.place(p, cp, il) for p in pos], device=DEV)
        codes = st_v[j[:, 0], b, j[:, 1]]
        u = st_s[j[:, 0], b, j[:, 1] // block]
        k = codes * u[:, None]
        want, wl = ref.attend(qb, k, scale)
        s = scale * (qb @ k.T)
        p = torch.exp(s - wl[:, None])
        mass = p @ k[:, :512].abs()
        # what the split may lose: 2^-18 of the largest p u of 32 tokens, at most 32 of them for each maximum
        lost = 2.0 ** -18 * 32 * (p * u).sum(1, keepdim=True) * codes[:, :512].abs().amax()
        top = qb.abs().amax(1, keepdim=True)
        small = qb.abs() < 2.0 ** -9 * top
        ds = abs(scale) * (2.0 ** -21 * (qb.abs() @ k.abs().T) +
                           2.0 ** -16 * top * (small.double() @ k.abs().T)).amax(1, keepdim=True) + \
            2.0 ** -22 * (s.abs().amax(1, keepdim=True) + 1)
        err = (out[b].double() - want).abs()
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * ds + 2.0 ** -18) * mass + lost
        assert not out[b].isnan().any()
        assert (err <= tol).all(), f"row {b}: {float((err - tol).max())}"
        ln = lse[b].double() * (1.0 if base_e else math.log(2.0))
        assert ((ln - wl).abs() <= ds[:, 0] + 2.0 ** -20 * (wl.abs() + 1)).all(), f"row {b}"
        record_error("8-bit decode output |gpu - oracle| / sum p|v|", float((err / mass.clamp(min=1e-300)).max()))
        record_error("8-bit decode LSE |gpu - oracle|", float((ln - wl).abs().max()))


def make_cache(g, cp, B, T, dk, block):
    kv, sc = [], []
    for _ in range(cp):
        x = randn(g, B, T, dk) * torch.exp(0.4 * randn(g, B, T, 1))
        nb = -(-T // block)
        s = torch.exp2(torch.randint(-8, -6, (B, nb), generator=g, device=DEV).float())
        s = s * (1 + 0.5 * torch.rand((B, nb), generator=g, device=DEV))  # not only powers of two
        kv.append((x / s.repeat_interleave(block, 1)[:, :T, None]).clamp(-448, 448).to(E4M3))
        sc.append(s)
    return kv, sc


DECODES = [
    # H, dk, cp, interleave, block, T, lengths, window, sinks
    (16, 576, 1, 1, 1, 1, [1], 0, 0),
    (16, 576, 1, 1, 1, 200, [0, 1, 31, 32, 33, 127, 128, 129, 199, 200], 0, 0),
    (64, 576, 1, 1, 1, 300, [0, 1, 127, 128, 129, 256, 257, 300], 0, 0),
    (32, 576, 1, 1, 16, 300, [0, 5, 128, 299], 0, 0),
    (128, 576, 1, 1, 64, 1030, [1030, 0, 999, 64], 0, 0),
    (128, 512, 1, 1, 1, 700, [700, 3, 513], 0, 0),
    (16, 512, 1, 1, 128, 700, [700, 3, 513], 0, 0),
    (32, 512, 2, 1, 4, 300, [600, 3, 513], 0, 0),
    (1, 576, 1, 1, 1, 400, [400, 17], 0, 0),
    (8, 576, 2, 16, 16, 130, [259, 100, 16, 17], 0, 0),
    (24, 576, 4, 1, 1, 90, [360, 1, 2, 3, 0], 0, 0),
    (100, 576, 1, 1, 1, 300, [300, 129], 0, 0),
    (65, 576, 3, 7, 8, 260, [700, 41], 0, 0),
    (48, 576, 16, 1, 2, 40, [640, 7, 600], 0, 0),
    (64, 576, 1, 1, 1, 500, [500, 130, 129, 100, 0], 128, 0),
    (64, 576, 1, 1, 1, 900, [900, 600, 40], 300, 4),
    (16, 576, 1, 1, 16, 900, [900, 600, 404, 403], 400, 3),
    (128, 576, 2, 1, 1, 500, [1000, 700, 9], 333, 8),
    (32, 576, 4, 16, 64, 300, [1200, 900, 77, 0], 100, 130),
    (64, 512, 1, 1, 1, 700, [700, 640], 1, 0),
    (64, 576, 1, 1, 1, 700, [700, 640], 5, 1000),
    (16, 576, 1, 1, 1, 500, [10000, -5, 499], 0, 0),  # beyond the cache, negative
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"H{c[0]}d{c[1]}cp{c[2]}i{c[3]}b{c[4]}T{c[5]}w{c[7]}s{c[8]}")
def test_decode(case):
    H, dk, cp, il, block, T, lengths, window, sinks = case
    g = gen(H + T + window)
    B = len(lengths)
    kv, sc = make_cache(g, cp, B, T, dk, block)
    q = randn(g, B, H, dk).bfloat16()
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    # what no row sees may hold anything: NaN codes, NaN scales where a whole block is unseen
    for b, n in enumerate(lengths):
        seen = [set() for _ in range(cp)]
        for p in ref.visible(max(n, 0), window, sinks):
            seen[ref.place(p, cp, il)[0]].add(ref.place(p, cp, il)[1])
        for j in range(cp):
            for t in range(T):
                if t not in seen[j]:
                    bits(kv[j])[b, t] = 0x7F
            for k in range(sc[j].shape[1]):
                if not any(t in seen[j] for t in range(k * block, min(T, (k + 1) * block))):
                    sc[j][b, k] = math.nan
    base_e = H % 3 != 0
    status = torch.zeros((1,), dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=block, interleave=il, window=window, sinks=sinks,
                                     lse_base_e=base_e, status=status)
    for j in range(cp):  # (the plain form must not meet the NaNs of what it does not see)
        bits(kv[j])[kv[j].double().isnan()] = 0
        sc[j].nan_to_num_(1.0)
    check_decode(q, kv, sc, lens, SCALE, cp, il, block, window, sinks, out, lse, base_e)
    assert int(status) == 0
    again = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=block, interleave=il, window=window, sinks=sinks,
                                  lse_base_e=base_e)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("H,B,T,cp", [(16, 1, 40000, 1), (128, 1, 20001, 1), (64, 2, 9000, 2), (128, 37, 700, 1),
                                      (32, 5, 5000, 1)])
def test_decode_split_rows(H, B, T, cp):
    """Rows spread over many CTAs, unevenly."""
    g = gen(T)
    kv, sc = make_cache(g, cp, B, T, 576, 1)
    q = randn(g, B, H, 576).bfloat16()
    lens = (torch.rand((B,), generator=g, device=DEV) * cp * T).int()
    lens[0] = cp * T
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    check_decode(q, kv, sc, lens, SCALE, cp, 1, 1, 0, 0, out, lse, rows=range(0, B, 6))


def test_decode_more_rows_than_threads():
    g = gen(3)
    B, H, T = 1300, 16, 400
    kv, sc = make_cache(g, 1, B, T, 576, 1)
    q = randn(g, B, H, 576).bfloat16()
    lens = (torch.rand((B,), generator=g, device=DEV) * T).int()
    lens[::7] = 0
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    check_decode(q, kv, sc, lens, SCALE, 1, 1, 1, 0, 0, out, lse, rows=list(range(0, B, 61)) + [1, 512, 1299])
    assert (out[::7] == 0).all() and (lse[::7] == -math.inf).all()
    short = dcp.mla_cache8_decode(q, [kv[0][:, :256].contiguous()], [sc[0][:, :256].contiguous()], lens.clamp(max=256),
                                  SCALE)  # at most two tiles a row: no row is split
    check_decode(q, [kv[0][:, :256]], [sc[0][:, :256]], lens.clamp(max=256), SCALE, 1, 1, 1, 0, 0, *short,
                 rows=list(range(0, B, 61)) + [1, 512, 1299])


@pytest.mark.parametrize("gap", [8.0, 14.0, 25.0, 60.0, 300.0])
@pytest.mark.parametrize("first", [True, False])
def test_decode_one_token_far_above_the_rest(gap, first):
    """A first token that takes much of the mass, the rest spread over thousands: small probabilities must count."""
    g = gen(4)
    T, H = 6000, 16
    x = randn(g, 1, T, 576) * 0.3
    q = randn(g, 1, H, 576)
    at = 0 if first else T - 1
    direction = randn(g, 576)
    direction /= direction.norm()
    q = (q * 0.3 + 8 * direction).bfloat16()
    x[0, at] = direction * (gap / (8 * SCALE))
    s = torch.exp2(torch.floor(torch.log2(x.abs().amax(-1) / 448)) + 1)
    kv, sc = [(x / s[..., None]).to(E4M3)], [s]
    lens = torch.full((1,), T, dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    check_decode(q, kv, sc, lens, SCALE, 1, 1, 1, 0, 0, out, lse)


def test_decode_rising_scores():
    """Every tile's scores above the last one's by more than the reference may lag."""
    g = gen(12)
    T, H = 1000, 64
    direction = randn(g, 576)
    direction /= direction.norm()
    x = direction * torch.arange(T, device=DEV)[:, None] * 0.6 + randn(g, T, 576) * 0.1
    q = (direction * 8 + randn(g, 1, H, 576) * 0.1).bfloat16()
    for y in (x, x.flip(0)):
        s = torch.exp2(torch.floor(torch.log2(y.abs().amax(-1) / 448)) + 1)
        kv, sc = [(y / s[:, None]).to(E4M3)[None].contiguous()], [s[None].contiguous()]
        lens = torch.full((1,), T, dtype=torch.int32, device=DEV)
        out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
        check_decode(q, kv, sc, lens, SCALE, 1, 1, 1, 0, 0, out, lse)


@pytest.mark.parametrize("B,cp,window,sinks", [(33, 3, 0, 0), (40, 2, 150, 5), (513, 2, 130, 0), (600, 1, 200, 3)])
def test_decode_many_rows_with_shards_and_windows(B, cp, window, sinks):
    g = gen(B)
    H, T, block = 24, 330, 4
    kv, sc = make_cache(g, cp, B, T, 576, block)
    q = randn(g, B, H, 576).bfloat16()
    lens = (torch.rand((B,), generator=g, device=DEV) * cp * (T + 30)).int()  # (some past the end)
    lens[::5] = 0
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=block, interleave=2, window=window, sinks=sinks)
    check_decode(q, kv, sc, lens, SCALE, cp, 2, block, window, sinks, out, lse, rows=[0, 1, 2, 31, 32, B // 2, B - 1])


@pytest.mark.parametrize("H", [16, 128])
def test_decode_scales_over_their_whole_range(H):
    """Blocks of scales from 2^-60 to 2^32 in one row, small q."""
    g = gen(H)
    T, block = 500, 4
    q = (randn(g, 1, H, 576) * 2.0 ** -36).bfloat16()
    kv = [(randn(g, 1, T, 576) * 60).to(E4M3)]
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    for lo, hi in ((-60, 33), (-60, -59), (32, 33), (-10, 33)):
        sc = [torch.exp2(torch.randint(lo, hi, (1, T // block), generator=g, device=DEV).float())]
        out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=block)
        check_decode(q, kv, sc, lens, SCALE, 1, 1, block, 0, 0, out, lse)


def levelled(g, levels, u, T, B=1):
    """q [64 dims of 8 behind 512 zeros] and keys whose scores lie about levels[i] (base 2) in tile i of 128 tokens and
    whose scale there is u[i]; latents of about 100 codes."""
    lv = torch.tensor(levels, device=DEV, dtype=torch.float64).repeat_interleave(128)[:T]
    us = torch.tensor(u, device=DEV, dtype=torch.float64).repeat_interleave(128)[:T]
    codes = torch.cat((randn(g, B, T, 512) * 100, torch.zeros((B, T, 64), device=DEV)), 2).double()
    top = max(float((lv.abs() / us).amax()) / 300, 2.0 ** -60)  # what q has to be for the largest code to be about 300
    codes[..., 512:] = (lv / us / top)[:, None]
    q = torch.zeros((B, 576), device=DEV, dtype=torch.float64)
    q[:, 512:] = top / (64 * SCALE * math.log2(math.e))
    kv = codes.clamp(-448, 448).float().to(E4M3)
    return q, kv, us.float().expand(B, T).contiguous()


def check_levelled(q, kv, sc, lens, out, lse, rows=(0,)):
    """As check_decode for one shard in blocks of 1, where q splits exactly wherever a code is not zero: scores are fp32
    sums of exact products, and nothing else moves the sums. A scale of 0 counts as 2^-60 among the 32 tokens of a
    probability scale: its token has p u = p 2^-60 there (of codes of 0, or of 2^-60 times its codes), and the others
    may lose 2^-18 of that like of any other token's."""
    for b in rows:
        n = int(lens[b])
        codes, u = kv[b, :n].double(), sc[b, :n].double()
        k, qb = codes * u[:, None], q[b].double()
        want, wl = ref.attend(qb, k, SCALE)
        s = SCALE * (qb @ k.T)
        p = torch.exp(s - wl[:, None])
        ds = SCALE * 2.0 ** -21 * (qb.abs() @ k.abs().T).amax(1, keepdim=True) + \
            2.0 ** -22 * (s.abs().amax(1, keepdim=True) + 1)
        lost = 2.0 ** -18 * 32 * (p * u.clamp(min=2.0 ** -60)).sum(1, keepdim=True) * codes[:, :512].abs().amax()
        assert not out[b].isnan().any()
        assert ((lse[b].double() - wl).abs() <= ds[:, 0] + 2.0 ** -20 * (wl.abs() + 1)).all(), f"row {b}"
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * ds + 2.0 ** -18) * (p @ k[:, :512].abs()) + lost
        assert ((out[b].double() - want).abs() <= tol).all(), f"row {b}"


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("low", [-60.0, -91.0, -100.0, -128.0, -135.0, -150.0, -159.0, -161.0, -250.0])
@pytest.mark.parametrize("scale", [2.0 ** -60, 0.0])
def test_decode_a_zero_token_after_low_scores(H, low, scale):
    """A tile whose largest score and scale lie about 2^low below the reference's start, then, in another tile of the
    same segment, a token of zeros: score 0, and the scale that the append gives it. One row in one segment."""
    g = gen(int(-low) + H)
    q, kv, sc = levelled(g, [low + 7, low + 7], [2.0 ** -7] * 2, 256)
    bits(kv)[0, 200] = 0
    sc[0, 200] = scale
    q = (q[:, None] * (1 + 0.02 * torch.rand((1, H, 1), generator=g, device=DEV))).bfloat16()
    lens = torch.tensor([256], dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE)
    check_levelled(q, kv, sc, lens, out, lse)


@pytest.mark.parametrize("H,B", [(16, 16), (128, 16), (32, 40)])
def test_decode_zero_tokens_among_low_scores_in_split_rows(H, B):
    """The same in rows of many tiles that are split, a third of the tiles with a token of zeros; and over two shards,
    whose partial results go through merge."""
    g = gen(H)
    n = 3000
    tiles = -(-n // 128)
    q, kv, sc = levelled(g, [-128.0] * tiles, [2.0 ** -7] * tiles, n, B)
    zero = torch.arange(2 * 128 + 5, n, 3 * 128, device=DEV)
    bits(kv)[:, zero] = 0
    sc[:, zero] = 2.0 ** -60
    q = q[:, None].expand(B, H, 576).bfloat16()
    lens = torch.tensor([n - 7 * b for b in range(B)], dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE)
    rows = [0, 1, B // 2, B - 1]
    check_levelled(q, kv, sc, lens, out, lse, rows=rows)
    two, two_sc = [kv, kv.clone()], [sc, sc.clone()]
    parts = [dcp.mla_cache8_decode(q, [two[j] if j == k else None for j in range(2)],
                                   [two_sc[j] if j == k else None for j in range(2)], 2 * lens, SCALE)
             for k in range(2)]
    merged, ml = dcp.merge([p[0] for p in parts], [p[1] for p in parts], True)
    # the two halves are alike: the same output, rounded once more, and twice the sum
    assert ((torch.cat(merged, 1).double() - out.double()).abs() <= 2.0 ** -7 * out.double().abs()).all()
    assert ((torch.cat(ml, 1) - lse - math.log(2.0)).abs() <= 1e-4).all()


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("levels,exps", [
    ((0.0, 8.0), (-60, -7)), ((0.0, 20.0), (-60, -7)), ((0.0, 20.0), (-60, 0)), ((-9.0, 0.0), (-60, 32)),
    ((-9.0, 0.0), (-60, 31)), ((-40.0, 0.0), (-60, 32)), ((0.0, 133.0), (0, -60)), ((0.0, 160.0), (0, -60)),
    ((0.0, 127.0), (0, -60)), ((0.0, 0.0), (-60, 32)), ((0.0, 0.0), (32, -60)), ((0.0, 30.0), (32, -30)),
    ((0.0, 8.0), (-1000, -7)), ((0.0, 20.0), (-1000, 0)), ((-30.0, 0.0), (32, -1000))])
def test_decode_a_move_of_scores_and_scales(H, levels, exps):
    """Two tiles of one segment, each with its own score and its own scale: how far the reference moves goes by the one
    times the other, the sums by the scores alone."""
    g = gen(int(levels[1]) + exps[1] + H)
    q, kv, sc = levelled(g, levels, [2.0 ** e for e in exps], 256)
    q = q[:, None].expand(1, H, 576).bfloat16()
    lens = torch.tensor([256], dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE)
    check_levelled(q, kv, sc, lens, out, lse)


@pytest.mark.parametrize("H,B", [(16, 64), (64, 40), (32, 1)])
@pytest.mark.parametrize("order", ["up", "down", "steps"])
def test_decode_scales_in_order_along_the_row(H, B, order):
    """Scales over their whole range, one for each tile of 128 tokens: rising, falling, or the two ends in turn. All
    scores are 0, so every token counts alike."""
    g = gen(H + B)
    exps = {"up": list(range(-60, 33, 8)), "down": list(range(32, -61, -8)),
            "steps": [-60, 32, 31, -60, -59, 32] * 2}[order]
    T = 128 * len(exps)
    _, kv, sc = levelled(g, [0.0] * (len(exps) - 1) + [1.0], [2.0 ** e for e in exps], T, B)
    bits(kv)[..., 512:] = 0
    q = torch.zeros((B, H, 576), device=DEV)
    q[..., 512:] = randn(g, B, H, 64)
    q = q.bfloat16()
    lens = torch.tensor([T - b for b in range(B)], dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, [kv], [sc], lens, SCALE)
    check_levelled(q, kv, sc, lens, out, lse, rows=sorted({0, 1 % B, B // 2, B - 1}))


def test_decode_scores_out_of_range_are_nan():
    """Beyond 2^21 in units of ln 2: NaN, not a wrong number; the other heads and rows keep their bits."""
    g = gen(31)
    kv, sc = make_cache(g, 1, 2, 300, 576, 1)
    q = randn(g, 2, 32, 576).bfloat16()
    lens = torch.tensor([300, 200], dtype=torch.int32, device=DEV)
    clean = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    q[0, 5] *= 2.0 ** 24
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    same = torch.ones((2, 32), dtype=torch.bool, device=DEV)
    same[0, 5] = False
    assert out[0, 5].isnan().all() and lse[0, 5].isnan()
    assert torch.equal(out[same], clean[0][same]) and torch.equal(lse[same], clean[1][same])


def test_decode_q_word_by_word():
    """q whose heads are not on 16-byte boundaries, in each kernel form."""
    g = gen(32)
    for H in (5, 32, 64, 100):
        for dk in (512, 576):
            kv, sc = make_cache(g, 1, 2, 300, dk, 1)
            q = randn(g, 2, H, dk + 2).bfloat16()[..., 2:]
            lens = torch.tensor([300, 129], dtype=torch.int32, device=DEV)
            a = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
            b = dcp.mla_cache8_decode(q.contiguous(), kv, sc, lens, SCALE)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("level", [-3000.0, -200.0, -85.0, -40.0, 20.0, 60.0, 200.0, 3000.0])
@pytest.mark.parametrize("H", [16, 64])
def test_decode_scores_all_far_from_zero(level, H):
    """Scores about `level` (base 2) from the first tile on, and one row whose second tile jumps back to zero."""
    g = gen(int(level) + H)
    T = 300
    direction = randn(g, 576)
    direction /= direction.norm()
    a = torch.full((2, T, 1), level * math.log(2.0) / (8 * SCALE), device=DEV)
    a[1, 128:] = 0
    x = direction * a + randn(g, 2, T, 576) * 0.1
    q = (direction * 8 + randn(g, 2, H, 576) * 0.1).bfloat16()
    s = torch.exp2(torch.floor(torch.log2(x.abs().amax(-1) / 448)) + 1)
    kv, sc = [(x / s[..., None]).to(E4M3)], [s]
    lens = torch.tensor([T, T - 7], dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    check_decode(q, kv, sc, lens, SCALE, 1, 1, 1, 0, 0, out, lse)


def test_decode_q_of_very_different_heads_and_dims():
    g = gen(13)
    H, T = 64, 300
    kv, sc = make_cache(g, 1, 2, T, 576, 1)
    q = randn(g, 2, H, 576) * torch.exp2(torch.randint(-12, 3, (1, H, 1), generator=g, device=DEV).float())
    q = (q * torch.exp2(torch.randint(-14, 1, (1, 1, 576), generator=g, device=DEV).float())).bfloat16()
    q[0, 5] = 0
    lens = torch.tensor([300, 150], dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    check_decode(q, kv, sc, lens, SCALE, 1, 1, 1, 0, 0, out, lse)


def test_decode_zero_and_tiny_scales():
    """A block of zeros whose scale is the smallest one, or 0: scores 0, values 0."""
    g = gen(14)
    kv, sc = make_cache(g, 1, 1, 200, 576, 1)
    bits(kv[0])[0, 40:80] = 0
    sc[0][0, 40:60] = 2.0 ** -60
    sc[0][0, 60:80] = 0.0
    q = randn(g, 1, 32, 576).bfloat16()
    lens = torch.full((1,), 200, dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    check_decode(q, kv, sc, lens, SCALE, 1, 1, 1, 0, 0, out, lse)


def test_decode_nan_reaches_its_row_and_head_only():
    g = gen(15)
    kv, sc = make_cache(g, 1, 3, 700, 576, 1)
    q = randn(g, 3, 64, 576).bfloat16()
    lens = torch.tensor([700, 699, 650], dtype=torch.int32, device=DEV)
    clean = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    q[0, 7, 3], q[2, 9, 100] = math.nan, math.inf
    bits(kv[0])[1, 400, 17] = 0x7F
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    bad = torch.zeros((3, 64), dtype=torch.bool, device=DEV)
    bad[0, 7] = bad[2, 9] = True
    bad[1] = True  # every head's score of that token
    assert lse[bad].isnan().all() and out[bad][:, 17].isnan().all()
    assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


@pytest.mark.parametrize("H,T,block", [(16, 200, 1), (64, 700, 16), (128, 256, 64)])
def test_decode_a_visible_scale_that_is_nan(H, T, block):
    """It reaches every head of its row (a NaN scale of what is not visible: test_decode)."""
    g = gen(H)
    kv, sc = make_cache(g, 1, 3, T, 576, block)
    q = randn(g, 3, H, 576).bfloat16()
    lens = torch.tensor([T, T - 1, T - 70], dtype=torch.int32, device=DEV)
    clean = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=block)
    sc[0][1, 100 // block] = math.nan
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=block)
    assert out[1].isnan().all() and lse[1].isnan().all()
    for b in (0, 2):
        assert torch.equal(out[b], clean[0][b]) and torch.equal(lse[b], clean[1][b])


def test_decode_strided_q_given_outputs_and_flags():
    g = gen(16)
    B, H, T = 3, 40, 300
    kv, sc = make_cache(g, 1, B, T, 576, 1)
    wide = randn(g, H, B, 600).bfloat16()
    q = wide.transpose(0, 1)[..., 12:588]
    lens = torch.tensor([300, 1, 200], dtype=torch.int32, device=DEV)
    want = dcp.mla_cache8_decode(q.contiguous(), kv, sc, lens, SCALE)
    out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((B, H), dtype=torch.float32, device=DEV)
    n = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.full((dcp.dcp_mla_cache8_decode_workspace_bytes(1, B, H, T, 0, 0, n),), 0xFF, dtype=torch.uint8, device=DEV)
    codes = [x.view(torch.uint8) for x in kv]
    got = dcp.mla_cache8_decode(q, codes, sc, lens, SCALE, out=out, lse=lse, workspace=ws, flags=dcp.DCP_FLAG_PDL)
    assert got[0] is out and got[1] is lse
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_decode_partials_of_shards_merge_to_the_whole():
    g = gen(17)
    B, H, T, cp = 4, 64, 200, 4
    kv, sc = make_cache(g, cp, B, T, 576, 1)
    q = randn(g, B, H, 576).bfloat16()
    lens = torch.tensor([800, 3, 0, 555], dtype=torch.int32, device=DEV)
    kw = dict(interleave=2, window=600, sinks=4)
    outs, lses = [], []
    for j in range(cp):
        o, l = dcp.mla_cache8_decode(q, [kv[k] if k == j else None for k in range(cp)],
                                     [sc[k] if k == j else None for k in range(cp)], lens, SCALE, **kw)
        check_decode(q, kv, sc, lens, SCALE, cp, 2, 1, 600, 4, o, l, held=[j])
        outs.append(o)
        lses.append(l)
    merged, ml = dcp.merge(outs, lses, True)
    whole, wl = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, **kw)
    check_decode(q, kv, sc, lens, SCALE, cp, 2, 1, 600, 4, whole, wl)
    # each partial is rounded to bf16 once more: 2^-8 of the weighted partials, below 2^-8 of the largest output
    assert (torch.cat(merged, 1).double() - whole.double()).abs().max() <= 3 * 2.0 ** -8 * whole.double().abs().max()
    m, w = torch.cat(ml, 1), wl
    assert torch.equal(torch.isinf(m), torch.isinf(w))
    assert (m[~torch.isinf(m)] - w[~torch.isinf(w)]).abs().max() <= 1e-5 * w[~torch.isinf(w)].abs().max()


@pytest.mark.parametrize("B,H,T", [(3, 16, 200), (2, 64, 1000), (2, 128, 1000), (40, 32, 500), (700, 64, 256)])
def test_decode_after_waits_that_gave_up(B, H, T):
    """The first tile of every CTA never counts as landed: the status word reads 1 and the call ends; the next one is
    right, in the same workspace."""
    g = gen(B)
    kv, sc = make_cache(g, 1, B, T, 576, 1)
    q = randn(g, B, H, 576).bfloat16()
    lens = torch.full((B,), T, dtype=torch.int32, device=DEV)
    n = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.empty((max(dcp.dcp_mla_cache8_decode_workspace_bytes(1, B, H, T, 0, 0, n), 256),), dtype=torch.uint8,
                     device=DEV)
    status = torch.zeros((1,), dtype=torch.int32, device=DEV)
    dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, workspace=ws, status=status, flags=dcp.DCP_MLA_FLAG_TEST_STALL)
    torch.cuda.synchronize()
    assert int(status) == 1
    status.zero_()
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, workspace=ws, status=status)
    check_decode(q, kv, sc, lens, SCALE, 1, 1, 1, 0, 0, out, lse, rows=[0, B - 1])
    assert int(status) == 0


def test_decode_of_an_empty_cache_and_no_rows():
    q = torch.zeros((2, 16, 576), dtype=torch.bfloat16, device=DEV)
    empty = torch.empty((2, 0, 576), dtype=E4M3, device=DEV)
    sc = torch.empty((2, 0), dtype=torch.float32, device=DEV)
    # (an empty tensor has no address: one shard with room, no tokens in it)
    kv, s = blank(1, 2, 4, 576, 1)
    out, lse = dcp.mla_cache8_decode(q, kv, s, torch.zeros((2,), dtype=torch.int32, device=DEV), SCALE)
    assert (out == 0).all() and (lse == -math.inf).all()
    with pytest.raises(dcp.DcpError):
        dcp.mla_cache8_decode(q, [empty], [sc], torch.zeros((2,), dtype=torch.int32, device=DEV), SCALE)


@pytest.mark.parametrize("cp,held", [(1, [0]), (3, [0, 1, 2]), (3, [1])])
def test_a_batch_of_no_rows(cp, held):
    """Every call over a cache of no rows does nothing and gives empty results."""
    kv = [torch.empty((0, 64, 576), dtype=E4M3, device=DEV) if j in held else None for j in range(cp)]
    sc = [torch.empty((0, 4), device=DEV) if j in held else None for j in range(cp)]
    none = torch.empty((0,), dtype=torch.int32, device=DEV)
    zero = torch.zeros((1,), dtype=torch.int32, device=DEV)
    latent, rope = (torch.empty((0, w), dtype=torch.bfloat16, device=DEV) for w in (512, 64))
    inv_freq, _ = dcp.mla_rope_inv_freq(64)
    for cu in (None, zero):
        dcp.mla_cache8_append(latent, rope, kv, sc, none, cu_new=cu, block=16, inv_freq=inv_freq)
        assert dcp.mla_cache8_read(kv, sc, 0, starts=none, cu=cu, block=16).shape == (0, 576)
    for kw in ({}, dict(window=9, sinks=2)):
        out, lse = dcp.mla_cache8_decode(torch.empty((0, 16, 576), dtype=torch.bfloat16, device=DEV), kv, sc, none,
                                         SCALE, block=16, **kw)
        assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
    with pytest.raises(dcp.DcpError):  # packed tokens that belong to no row
        dcp.mla_cache8_append(latent.new_zeros((3, 512)), rope.new_zeros((3, 64)), kv, sc, none, block=16)
    with pytest.raises(dcp.DcpError):
        dcp.mla_cache8_read(kv, sc, 3, block=16)
    torch.cuda.synchronize()


@pytest.mark.parametrize("what", ["append", "read"])
def test_a_cache_of_no_tokens_is_refused(what):
    """An empty tensor has no address, so that a shard without tokens cannot be told from one that is not held."""
    kv, sc = [torch.empty((2, 0, 576), dtype=E4M3, device=DEV)], [torch.empty((2, 0), device=DEV)]
    lens = torch.zeros((2,), dtype=torch.int32, device=DEV)
    with pytest.raises(dcp.DcpError):
        if what == "append":
            dcp.mla_cache8_append(torch.zeros((2, 512), dtype=torch.bfloat16, device=DEV),
                                  torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV), kv, sc, lens)
        else:
            dcp.mla_cache8_read(kv, sc, 2)


@pytest.mark.parametrize("H,T,window", [(200, 300, 0), (1000, 300, 0), (1024, 900, 200), (1024, 128, 0)])
def test_decode_many_heads(H, T, window):
    g = gen(H + T)
    kv, sc = make_cache(g, 1, 3, T, 576, 4)
    q = randn(g, 3, H, 576).bfloat16()
    lens = torch.tensor([T, 77, 0], dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=4, window=window)
    check_decode(q, kv, sc, lens, SCALE, 1, 1, 4, window, 0, out, lse)


@pytest.mark.parametrize("scale", [0.0, -SCALE])
@pytest.mark.parametrize("H", [16, 64])
def test_decode_scale_of_zero_or_below(H, scale):
    g = gen(H)
    kv, sc = make_cache(g, 2, 2, 300, 576, 1)
    q = randn(g, 1, 1, 576).bfloat16().expand(2, H, 576)  # (rows and heads that q repeats)
    lens = torch.tensor([600, 131], dtype=torch.int32, device=DEV)
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, scale)
    check_decode(q, kv, sc, lens, scale, 2, 1, 1, 0, 0, out, lse)


def test_lengths_windows_and_places_at_their_limits():
    """Positions up to 2^31 - 1 over caches that end long before: nothing is written or read there, and the decode sees
    the first tokens alone."""
    g = gen(77)
    B, T, cp, big = 3, 300, 3, (1 << 31) - 1
    kv, sc = make_cache(g, cp, B, T, 576, 4)
    sc = [torch.exp2(torch.ceil(torch.log2(s))) for s in sc]
    before = [bits(x).clone() for x in kv], [x.clone() for x in sc]
    q = randn(g, B, 32, 576).bfloat16()
    lens = torch.tensor([big, big - 100, 40], dtype=torch.int32, device=DEV)
    for il in (1, 16, 1 << 24):
        for window, sinks in ((5, 9), (1, 1 << 40), (1 << 40, 0), (big, 3), (1 << 62, 1 << 62)):
            out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=4, interleave=il, window=window,
                                             sinks=sinks)
            for b in range(B):
                n = int(lens[b])
                rows, codes = [], []
                for j in range(cp):  # what shard j holds, by position
                    t = torch.arange(T, device=DEV)
                    pos = (t // il * cp + j) * il + t % il
                    see = (pos < n) & ((pos >= n - window) | (pos < sinks))
                    rows.append(kv[j][b, see].double() * sc[j][b, t[see] // 4].double()[:, None])
                k = torch.cat(rows)
                want, wl = ref.attend(q[b].double(), k, SCALE)
                if not len(k):
                    assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
                    continue
                # as in check_decode, with every rounding at its largest over these caches
                mass = torch.exp(SCALE * (q[b].double() @ k.T) - wl[:, None]) @ k[:, :512].abs()
                assert ((lse[b].double() - wl).abs() <= 1e-3).all()
                assert ((out[b].double() - want).abs() <= 2.0 ** -7 * mass + 2.0 ** -8 * want.abs() + 1e-2).all()
        latent, rope = randn(g, B * 50, 512).bfloat16(), randn(g, B * 50, 64).bfloat16()
        far = torch.full((B,), big - 20, dtype=torch.int32, device=DEV)
        for block in (1, 4):
            scales = sc if block == 4 else [torch.ones((B, T), device=DEV) for _ in range(cp)]
            dcp.mla_cache8_append(latent, rope, kv, scales, far, block=block, interleave=il)
        got = torch.full((B * 50, 576), 3.0, device=DEV)
        dcp.mla_cache8_read(kv, sc, B * 50, starts=far, block=4, interleave=il, dtype=torch.float32, out=got)
        assert (got == 3).all()
    for x, y in zip(kv + sc, before[0] + before[1]):
        assert torch.equal(bits(x) if x.dtype == E4M3 else x, y)


def test_decode_65535_rows():
    g = gen(65535)
    B, H, T = 65535, 16, 300
    one = (randn(g, 1, T, 576) * 30).clamp(-448, 448).to(E4M3)
    kv = [bits(one).expand(B, T, 576).contiguous().view(E4M3)]
    sc = [(2.0 ** -5 * (1 + torch.rand((B, T), generator=g, device=DEV)))]
    q = randn(g, 1, H, 576).bfloat16().expand(B, H, 576)
    lens = (torch.arange(B, device=DEV) * 7919 % (T + 1)).int()
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    check_decode(q, kv, sc, lens, SCALE, 1, 1, 1, 0, 0, out, lse, rows=[0, 1, 2, 511, 512, 40000, 65533, 65534])
    assert not out.isnan().any() and ((lse == -math.inf) == (lens == 0)[:, None]).all()


# ---- the chain, streams and graphs ------------------------------------------------------


def chain(step, st):
    """One serving step: rotate the queries, append the new tokens, attend, read the last tokens back."""
    inv_freq = st["inv_freq"]
    dcp.mla_rope(st["q_pe"][step], st["lens"], inv_freq, out=st["q"][..., 512:])
    dcp.mla_cache8_append(st["latent"][step], st["k_pe"][step], st["kv"], st["sc"], st["lens"], block=st["block"],
                          interleave=st["il"], inv_freq=inv_freq)
    st["lens"] += 1
    out, lse = dcp.mla_cache8_decode(st["q"], st["kv"], st["sc"], st["lens"], SCALE, block=st["block"],
                                     interleave=st["il"], window=st["window"], sinks=st["sinks"])
    last = dcp.mla_cache8_read(st["kv"], st["sc"], out.shape[0], starts=st["lens"] - 1, block=st["block"],
                               interleave=st["il"])
    return out, lse, last


def chain_state(block, il, cp, steps=5, B=3, H=32, T=160, window=0, sinks=0):
    g = gen(block + cp)
    kv, sc = blank(cp, B, T, 576, block)
    st = {"kv": kv, "sc": sc, "block": block, "il": il, "window": window, "sinks": sinks,
          "inv_freq": dcp.mla_rope_inv_freq(64)[0],
          "q": randn(g, B, H, 576).bfloat16(), "q_pe": randn(g, steps, B, H, 64).bfloat16(),
          "latent": randn(g, steps, B, 512).bfloat16(), "k_pe": randn(g, steps, B, 64).bfloat16()}
    counts = [100, 37, 1]
    st["lens"] = torch.zeros((B,), dtype=torch.int32, device=DEV)
    st["prompt"], st["prompt_pe"] = randn(g, sum(counts), 512).bfloat16(), randn(g, sum(counts), 64).bfloat16()
    st["cu"] = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
    dcp.mla_cache8_append(st["prompt"], st["prompt_pe"], kv, sc, st["lens"], cu_new=st["cu"], block=block,
                          interleave=il, inv_freq=st["inv_freq"])
    st["lens"] += torch.tensor(counts, device=DEV, dtype=torch.int32)
    st["counts"] = counts
    return st


@pytest.mark.parametrize("block,il,cp,window,sinks", [(1, 1, 1, 0, 0), (16, 4, 2, 0, 0), (64, 1, 4, 30, 2)])
def test_chain_against_unquantised_attention(block, il, cp, window, sinks):
    """Prompt, then five steps; each output against 64-bit attention over the tokens as they were given, rotated in 64
    bits. Quantising moves a key or value by at most 2^-4 of itself (and 2^-9 / 448 of its block's peak)."""
    st = chain_state(block, il, cp, window=window, sinks=sinks)
    B, H = st["q"].shape[:2]
    cu = st["cu"].tolist()
    keys = []
    for b in range(B):
        pos = torch.arange(st["counts"][b], device=DEV)
        k = ref.rotate(st["prompt_pe"][cu[b]:cu[b + 1], None].double(), pos, st["inv_freq"], 0, True)[:, 0]
        keys.append(torch.cat((st["prompt"][cu[b]:cu[b + 1]].double(), k), 1))
    for step in range(5):
        before = st["lens"].clone()
        out, lse, last = chain(step, st)
        qr = ref.rotate(st["q_pe"][step].double(), before, st["inv_freq"], 0, True)
        assert ((st["q"][..., 512:].double() - qr).abs() <= 2.0 ** -8 * qr.abs() + 1e-5).all()
        kr = ref.rotate(st["k_pe"][step][:, None].double(), before, st["inv_freq"], 0, True)[:, 0]
        for b in range(B):
            new = torch.cat((st["latent"][step, b].double(), kr[b]))
            keys[b] = torch.cat((keys[b], new[None]))
            peak = keys[b].abs().max()
            assert ((last[b].double() - new).abs() <= 2.0 ** -4 * new.abs() + 2.0 ** -9 * peak / 224 + 1e-5).all()
            k = keys[b][ref.visible(len(keys[b]), window, sinks)]
            want, wl = ref.attend(st["q"][b].double(), k, SCALE)
            # a score moves by at most e = scale * <|q|, 2^-4 |k|>, a probability by the factor exp(2 e): bounded
            # through the mean square instead, 576 independent roundings of at most 2^-4 each
            rms = SCALE * 2.0 ** -4 * (st["q"][b].double() ** 2 @ (k ** 2).T).sqrt().amax()
            assert (lse[b].double() - wl).abs().max() <= 6 * rms
            assert (out[b].double() - want).abs().max() <= (2.0 ** -4 + 12 * rms) * k.abs().max()


def test_chain_captured_and_replayed():
    eager = chain_state(16, 4, 2)
    captured = chain_state(16, 4, 2)
    want = [chain(s, eager) for s in range(3)]
    first = chain(0, captured)  # warm: the first step runs eagerly
    for a, b in zip(first, want[0]):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in (1, 2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(chain(s, captured))
        graphs.append(graph)
    torch.cuda.synchronize()
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for s in (1, 2):
        for a, b in zip(outs[s - 1], want[s]):
            assert torch.equal(a, b)
    for a, b in zip(captured["kv"] + captured["sc"], eager["kv"] + eager["sc"]):
        assert torch.equal(bits(a) if a.dtype == E4M3 else a, bits(b) if b.dtype == E4M3 else b)


def test_two_graphs_share_a_workspace():
    """Two captured decodes of different sizes in one workspace, replayed in turn on one stream."""
    n = torch.cuda.get_device_properties(0).multi_processor_count
    sizes = [(3, 64, 3000), (40, 16, 900)]
    ws = torch.full((max(dcp.dcp_mla_cache8_decode_workspace_bytes(1, B, H, T, 0, 0, n) for B, H, T in sizes),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    calls, want = [], []
    for k, (B, H, T) in enumerate(sizes):
        g = gen(50 + k)
        kv, sc = make_cache(g, 1, B, T, 576, 1)
        q = randn(g, B, H, 576).bfloat16()
        lens = (torch.rand((B,), generator=g, device=DEV) * T).int()
        want.append(dcp.mla_cache8_decode(q, kv, sc, lens, SCALE))
        calls.append((q, kv, sc, lens))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(dcp.mla_cache8_decode(*c, SCALE, workspace=ws))
        graphs.append(graph)
    for _ in range(3):
        for o, l in outs:
            o.fill_(9.0)
            l.fill_(9.0)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_two_host_threads():
    """The chain from two threads at once, each on a stream of its own, gives one thread's results."""
    import threading
    want = [chain(s, state) for state in [chain_state(16, 4, 2)] for s in range(3)]
    states = [chain_state(16, 4, 2) for _ in range(2)]
    torch.cuda.synchronize()
    got, wrong = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [chain(s, states[i]) for s in range(3)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # (seen by the main thread)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong
    for mine in got:
        for a, b in zip(mine, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_on_other_streams():
    """The same decode and append on three streams at once, each with buffers of its own, as a stream object and as a
    raw handle; and outputs that are allocated on the stream that writes them."""
    g = gen(21)
    B, H, T = 4, 64, 2000
    kv, sc = make_cache(g, 1, B, T, 576, 1)
    q = randn(g, B, H, 576).bfloat16()
    lens = torch.tensor([2000, 5, 1999, 700], dtype=torch.int32, device=DEV)
    latent = randn(g, B, 512).bfloat16()
    pe = randn(g, B, 64).bfloat16()
    want = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE)
    kv0, sc0 = [x.clone() for x in kv], [x.clone() for x in sc]
    dcp.mla_cache8_append(latent, pe, kv0, sc0, lens - 1)
    copies = [([x.clone() for x in kv], [x.clone() for x in sc]) for _ in range(3)]
    lens1 = lens - 1
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i, s in enumerate(streams):
        for _ in range(4):
            got.append(dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, stream=s if i else s.cuda_stream))
        dcp.mla_cache8_append(latent, pe, *copies[i], lens1, stream=s if i else s.cuda_stream)
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    for k, s in copies:
        assert torch.equal(bits(k[0]), bits(kv0[0])) and torch.equal(s[0], sc0[0])


@pytest.mark.parametrize("seed", range(12))
def test_random_chains(seed):
    """Seeded random sizes: an append onto a random cache, then a decode over all of it."""
    import random
    r = random.Random(seed)
    cp, il = r.choice([(1, 1), (2, 1), (3, 5), (4, 16), (8, 2)])
    block = r.choice([1, 2, 8, 16, 32, 64, 128])
    B, H, dk = r.randint(1, 6), r.choice([1, 5, 16, 17, 32, 40, 64, 96, 128]), r.choice([512, 576, 576])
    T = r.randint(1, 400)
    g = gen(seed)
    kv, sc = make_cache(g, cp, B, T, dk, block)
    # power-of-two scales, as the append writes them
    sc = [torch.exp2(torch.ceil(torch.log2(s))) for s in sc]
    room = (T // il) * il * cp if T >= il else 0
    starts = [r.randint(0, room) for _ in range(B)]
    counts = [r.randint(0, min(90, room - s)) for s in starts]
    n = sum(counts)
    latent, pe = randn(g, n, 512).bfloat16(), (randn(g, n, 64).bfloat16() if dk == 576 else None)
    cu = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
    lens = torch.tensor(starts, dtype=torch.int32, device=DEV)
    if n:
        dcp.mla_cache8_append(latent, pe, kv, sc, lens, cu_new=cu, block=block, interleave=il,
                              inv_freq=dcp.mla_rope_inv_freq(64)[0] if dk == 576 else None)
    lens = lens + torch.tensor(counts, dtype=torch.int32, device=DEV)
    window = r.choice([0, 0, r.randint(1, 500)])
    sinks = r.choice([0, 3, 200]) if window else 0
    q = randn(g, B, H, dk).bfloat16()
    out, lse = dcp.mla_cache8_decode(q, kv, sc, lens, SCALE, block=block, interleave=il, window=window, sinks=sinks)
    check_decode(q, kv, sc, lens, SCALE, cp, il, block, window, sinks, out, lse)
