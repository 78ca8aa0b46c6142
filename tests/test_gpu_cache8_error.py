"""How far the 8-bit decode is from 64 bits where scales are ordinary: within a factor of 2^3 of each other, so that the
size of what is summed, sum p |v|, says what an error means. (Tests with scales as far apart as the format goes allow for
what the split of the probabilities loses then, next to which that size can be nothing.)"""
import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from oracle import cache8 as ref
from .conftest import record_error
from .test_gpu_cache8 import make_cache, randn

pytestmark = pytest.mark.gpu

DEV, SCALE = "cuda", 192 ** -0.5


@pytest.mark.parametrize("H,dk,T,block,paged", [(16, 576, 300, 1, False), (32, 576, 2000, 16, False),
                                                (64, 512, 700, 1, False), (128, 576, 4096, 64, False),
                                                (16, 576, 3000, 1, True), (128, 576, 1024, 64, True)])
def test_error_with_ordinary_scales(H, dk, T, block, paged):
    g = torch.Generator(device=DEV)
    g.manual_seed(H + T)
    B = 3
    kv, sc = make_cache(g, 1, B, T, dk, block)
    q, n = randn(g, B, H, dk).bfloat16(), torch.tensor([T, T - 1, T // 2 + 1], dtype=torch.int32, device=DEV)
    if paged:  # the same tokens, each row's pages in order
        page = 64
        M = -(-T // page)
        pad = lambda x, m: torch.cat((x, torch.zeros((B, m - x.shape[1], *x.shape[2:]), dtype=x.dtype, device=DEV)), 1)
        pool = pad(kv[0].view(torch.uint8), M * page).view(B * M, page, dk)
        scales = pad(sc[0], M * page // block).view(B * M, page // block)
        tb = torch.arange(B * M, dtype=torch.int32, device=DEV).view(B, M)
        out, lse = dcp.mla_cache8_decode(q, [pool], [scales], n, SCALE, block=block, tables=[tb])
    else:
        out, lse = dcp.mla_cache8_decode(q, kv, sc, n, SCALE, block=block)
    for b in range(B):
        L = int(n[b])
        u = sc[0][b].double().repeat_interleave(block)[:L]
        codes = kv[0][b, :L].double()
        k, qb = codes * u[:, None], q[b].double()
        want, wl = ref.attend(qb, k, SCALE)
        p = torch.exp(SCALE * (qb @ k.T) - wl[:, None])
        size = p @ k[:, :512].abs()
        # the output's rounding and the probabilities', 2^-8 each of what they round, and scores in fp32: q's parts hold
        # it to 2^-21 of a product (2^-16 of its largest where it is below 2^-9 of that), twice, for P and for the sums
        top = qb.abs().amax(1, keepdim=True)
        small = (qb.abs() < 2.0 ** -9 * top).double()
        ds = SCALE * (2.0 ** -21 * (qb.abs() @ k.abs().T) + 2.0 ** -16 * top * (small @ k.abs().T)).amax(1) + \
            2.0 ** -22 * ((SCALE * (qb @ k.T)).abs().amax(1) + 1)
        # and what the split may lose, 2^-18 of the largest p u of 32 tokens in each of them
        lost = 2.0 ** -18 * 32 * (p * u).sum(1, keepdim=True) * codes[:, :512].abs().amax()
        ratio = (out[b].double() - want).abs() / size
        assert (ratio <= 2.0 ** -7 + 2.0 ** -18 + 2 * ds[:, None] + lost / size).all()
        record_error("8-bit decode output, ordinary scales: |gpu - oracle| / sum p|v|", float(ratio.max()))
        err = (out[b].double() - want).pow(2).sum().sqrt() / want.pow(2).sum().sqrt()
        record_error("8-bit decode output, ordinary scales: root mean square of gpu - oracle / of oracle", float(err))
