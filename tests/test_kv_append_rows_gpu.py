"""pld_kv_append (HIP, gfx950) with so many rows that a workgroup takes four of
them: blocks that end inside four rows, every type and layout, rows in place,
pages that are bad under one row of four. Tolerances are
test_kv_append_gpu.py's."""

from __future__ import annotations

import numpy as np
import pytest

from prompt_lookup_gram_amd import binding as B
from test_kv_append_gpu import check, context, gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# 6 * 501 rows; blocks of 501, 1, 0, 4 n + 2, 4 n + 3 and 4 n rows
LENGTHS, DLEN, ROWS = [10, 1, 64, 7, 33, 100], [500, 0, -1, 41, 42, 43], 501


@pytest.mark.parametrize("dt,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"),
                                      ("f16", "e4m3")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_and_layouts(dt, cache, interleaved):
    check(LENGTHS, DLEN, ROWS, hq=3, hk=1, dt=dt, cache=cache, interleaved=interleaved,
          scales=cache == "e4m3", page=32, seed=50)


@pytest.mark.parametrize("dim,rot", [(64, 0), (128, 32), (96, 96), (128, 24), (192, 64),
                                     (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_the_head(dim, rot, interleaved):
    check([9, 1, 64, 7, 33, 100], [60, 0, -1, 41, 42, 43], 350, hq=2, hk=2, dim=dim, rot=rot,
          interleaved=interleaved, page=64, scaling="banded", magnitude=1.2, seed=51)


def test_in_place_without_q_and_strided():
    check(LENGTHS, DLEN, ROWS, hq=4, hk=1, in_place=True, seed=52)
    check(LENGTHS, DLEN, ROWS, with_q=False, seed=53)
    check(LENGTHS, DLEN, ROWS, hq=2, hk=1, pad=8, offset=8, seed=54)
    check(LENGTHS, DLEN, ROWS, hq=2, hk=1, pad=3, offset=1, seed=55)


@pytest.mark.parametrize("batch,rows", [(4, 512), (3, 683), (683, 3), (2050, 1), (5, 307),
                                        (96, 16), (29, 53)])
def test_both_sides_of_four_rows(batch, rows):
    # 2,048 rows and some more; 1,535, 1,536 and 1,537
    rng = np.random.default_rng([9102, rows])
    dlen = rng.integers(-1, min(rows, 20), batch)
    check(rng.integers(0, 40, batch).tolist(), dlen.tolist(), rows, hq=1, hk=1, seed=rows)


def test_a_bad_page_under_one_row_of_four():
    """The rows on the bad pages are not stored, the rows beside them are; q
    of all of them is rotated."""
    import torch
    rows, hq, hk, dim, page, n = 2100, 2, 1, 64, 16, 200
    gen = torch.Generator().manual_seed(56)
    x = torch.randn((rows, (hq + 2 * hk) * dim), generator=gen).bfloat16().cuda()
    table = torch.arange(20, dtype=torch.int32).flip(0).contiguous()
    bad = table.clone()
    # the block starts at position 6: page 1's rows 10.. and page 5's, each
    # starting and ending inside four rows
    bad[1], bad[5] = 20, -3
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    ctx = context(1, rows, 4096, hq, hk, dim, "bf16", "bf16", page)
    got = []
    try:
        for tab in (table, bad):
            kc = torch.ones((20, hk, page, dim), dtype=torch.bfloat16, device="cuda")
            vc = torch.ones((20, hk, dim, page), dtype=torch.bfloat16, device="cuda")
            oq = torch.ones((rows, hq * dim), dtype=torch.bfloat16, device="cuda")
            B.pld_kv_append(ctx, x, x.shape[1], x[:, hq * dim:], x[:, (hq + hk) * dim:],
                            x.shape[1], rows, one * 7, one * (n - 1), 1, tab.cuda(), 20, kc, vc,
                            20, None, None, oq)
            assert B.pld_sync(ctx) == (B.PLD_OK if tab is table else B.PLD_EINVAL)
            got.append((kc, vc, oq))
    finally:
        B.pld_destroy(ctx)
    (kc, vc, oq), (kb, vb, ob) = got
    assert torch.equal(oq, ob)
    for i in range(20):
        p = int(table[i])
        if i in (1, 5):
            assert bool((kb[p] == 1).all()) and bool((vb[p] == 1).all())
        else:
            assert torch.equal(kb[p], kc[p]) and torch.equal(vb[p], vc[p])
    assert not bool((kc[int(table[1])] == 1).all())
