"""Dense latent attention at the borders of what it may read and of what a token sees: page tables that end
inside a tile, sequences whose bounds are out of order, values that are not finite, and whether every tile
of a long context counts once.  (tests/test_mla.py holds the definition and its tolerances.)
"""
import math

import pytest
import torch

import dsa_sparse_attention_li_gb300 as dsa
from test_mla import (SCALE, check, definition, make_decode, make_prefill, run_decode, run_prefill, verify_decode,
                      verify_prefill)


@pytest.mark.parametrize("owned", [False, True], ids=["padding", "token"])
@pytest.mark.parametrize("length", [129, 150, 192])
def test_a_query_row_looks_up_only_pages_of_its_sequence(owned, length):
    """A tile is two pages.  Three pages of a sequence end inside its second tile, and the page table may end
    there: the number behind it (a guard of either kind) must not count for any row.  On the host, with the
    kernel's own rule; a row that belongs to no token counts as seeing 2^31 - 1 positions."""
    f = dsa.load_testhooks().dsa_test_mla_visible_columns
    got = []
    for guard in (0, -1, 10 ** 6):
        table = torch.tensor([0, 10 ** 6, 1, guard], dtype=torch.int32)
        seen = length if owned else 2 ** 31 - 1
        got.append([f(owned, seen, pos0, 1, table.data_ptr(), 2) for pos0 in (0, 64, 128, 192)])
    assert got[0] == got[1] == got[2]
    assert got[0] == ([64, 0, length - 128, length - 192] if owned else [64] * 4)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("bad", [0, 1, 2])
def test_decode_page_that_does_not_exist_in_a_table_that_ends_inside_a_tile(cuda_lib, fp8, bad):
    """The last sequence has three pages and the table no room for more; one of them does not exist."""
    c = make_decode([100, 170], [1, 1], 16, fp8, extra=1, tail=0)
    assert c["pt"].shape[1] == 4
    guarded = torch.full((7,), 10 ** 6, dtype=torch.int32, device="cuda")
    table = guarded[:6].view(2, 3)
    table.copy_(c["pt"][:, :3])
    table[1, bad] = (-1, 10 ** 6, 2 ** 31 - 1)[bad]
    c["pt"] = table
    out, lse, status = run_decode(c)
    assert status == dsa.DSA_ERR_DEVICE_CHECK
    keep = torch.ones(170, dtype=torch.bool)
    keep[64 * bad:64 * bad + 64] = False
    c["rows"][1] = c["rows"][1][keep.cuda()]
    c["lens"][1] = int(keep.sum())
    verify_decode(c, out, lse)
