"""The serving step over pages as README.md writes it."""
import os

import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from .test_gpu_pages import DEV, check_paged, ints, randn

pytestmark = pytest.mark.gpu


def paged_example():
    """Its lines: the state, the step, the compaction."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code, = [part.split("```")[0] for part in text.split("```python\n")[1:] if "mla_cache8_pages_update" in part]
    head, rest = code.split("\n", 1)
    step, last = rest.strip().rsplit("\n", 1)
    assert head.startswith("tables, refs =") and "pages_compact" in last
    return head, step, last


def test_the_step_that_the_readme_shows():
    """Rows go on, fork, end and stay away; what ends gives its pages back and attends to nothing."""
    head, step, last = paged_example()
    g = torch.Generator(device=DEV)
    g.manual_seed(21)
    B, M, P, page, block = 64, 8, 300, 64, 64
    pools = [torch.zeros((P, page, 576), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((P, page // block), device=DEV) for _ in range(2)]
    inv_freq, _ = dcp.mla_rope_inv_freq(64)
    names = dict(torch=torch, dcp=dcp, B=B, M=M, P=P, caches_of_all_layers=pools, scales_of_all_layers=scales,
                 cache=pools[0], scale=scales[0], inv_freq=inv_freq)
    exec(head, names)
    # prompts in the first 40 rows
    first = [50 + 7 * b if b < 40 else 0 for b in range(B)]
    lens = ints([0] * B)
    dcp.mla_cache8_pages_update(names["tables"], names["refs"], ints(list(range(B))), lens, ints(first), page=page)
    cu = ints([0] + first).cumsum(0).int()
    for pool, scale in zip(pools, scales):
        dcp.mla_cache8_append(randn(g, sum(first), 512).bfloat16(), randn(g, sum(first), 64).bfloat16(), [pool], [scale],
                              lens, cu_new=cu, block=block, inv_freq=inv_freq, tables=[names["tables"]])
    # rows 0 to 9 end, 10 to 39 go on, 40 to 49 fork rows 10 to 19, the others stay away
    parents = [-1] * 10 + list(range(10, 40)) + list(range(10, 20)) + [-1] * 14
    have = [first[p] if p >= 0 else 0 for p in parents]
    for turn in range(3):
        lens = ints(have)
        names.update(parents=ints(parents), lens=lens, q=randn(g, B, 16, 576).bfloat16(),
                     latent=randn(g, B, 512).bfloat16(), k_pe=randn(g, B, 64).bfloat16())
        exec(step, names)
        tables, refs, want = names["tables"], names["refs"], [n + 1 if p >= 0 else 0 for n, p in zip(have, parents)]
        assert names["wants"].tolist() == want and names["wants"].dtype == torch.int32
        assert names["missing"].tolist() == [0]
        assert (tables >= 0).sum(1).tolist() == [-(-n // page) for n in want]
        assert refs.sum() == (tables >= 0).sum()
        check_paged(names["q"], [pools[0]], [scales[0]], [tables], ints(want), 1, 1, block, 0, 0, names["out"], names["lse"])
        ended = ints(want) == 0
        assert (names["out"][ended] == 0).all() and (names["lse"][ended] == -float("inf")).all()
        have, parents = want, [b if p >= 0 else -1 for b, p in enumerate(parents)]
    used = int((refs > 0).sum())
    exec(last, names)
    assert int(names["tables"].max()) == used - 1 and (names["refs"][used:] == 0).all()
