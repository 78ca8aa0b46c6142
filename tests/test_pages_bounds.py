"""Sizes and addresses at the limits of the calls on pages, on the host. Nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

import decode_context_mla_dcp_gb300 as dcp
from .test_pages_refusals import A, ALIAS, COMPACT, COPY, DECODE, SHAPE, UPDATE, built, refused  # noqa: F401


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
