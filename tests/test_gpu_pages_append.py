"""Appends of blocks over tables that lack pages, in both ways in which a call finds its blocks."""
import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from .test_gpu_pages import DEV, ints, make_paged, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [2, 16, 32, 64, 128])
@pytest.mark.parametrize("B,count,missing", [
    (5, 700, 0.5), (5, 700, 1.0), (3, 1, 1.0), (600, 7, 0.5), (600, 40, 1.0),  # blocks found by their first tokens
    (7, 3000, 0.3), (500, 41, 0.5), (500, 41, 1.0),                            # counted, where there are many tokens
])
def test_blocks_without_a_page_are_left_alone(B, count, missing, block):
    """Half the pages, or all, are missing: the other blocks are those of a call that has them all, and no page of the
    pool changes that a call without them does not name."""
    page = 128
    g = torch.Generator(device=DEV)
    g.manual_seed(B * block + count)
    M = -(-(count + 70) // page)
    (kv,), (sc,), (tb,) = make_paged(g, 1, B, M, page, 576, block)
    lens = torch.randint(0, 70, (B,), generator=g, device=DEV, dtype=torch.int32)
    latent, rope = randn(g, B * count, 512).bfloat16(), randn(g, B * count, 64).bfloat16()
    gone = torch.rand((B, M), generator=g, device=DEV) < missing
    less = torch.where(gone, -1 - torch.arange(B * M, device=DEV, dtype=torch.int32).view(B, M), tb)
    whole, wscale = kv.view(torch.uint8).clone(), sc.clone()
    before, bscale = whole.clone(), sc.clone()
    kw = dict(block=block, inv_freq=dcp.mla_rope_inv_freq(64)[0])
    dcp.mla_cache8_append(latent, rope, [whole], [wscale], lens, tables=[tb], **kw)
    for _ in range(3):  # (twice more the same tokens on the state before)
        part, pscale = before.clone(), bscale.clone()
        dcp.mla_cache8_append(latent, rope, [part], [pscale], lens, tables=[less], **kw)
        named = torch.zeros((kv.shape[0],), dtype=torch.bool, device=DEV)
        named[tb[~gone].long()] = True
        assert torch.equal(part[named], whole[named]) and torch.equal(pscale[named], wscale[named])
        assert torch.equal(part[~named], before[~named]) and torch.equal(pscale[~named], bscale[~named])
