"""pld_attend_tree (HIP, gfx950) over caches that hold a value that is not finite
in one dim: what the rows that see it and the rows that do not are given, on
every kernel that a tree can take, against the 64-bit reference.

Tolerances are those of tests/test_attend_gpu.py. In the dim that holds it a row
that sees it is that infinity, or NaN; every other dim is as if it were not there."""

from __future__ import annotations

import numpy as np
import pytest

import target_reference as R
import tree_reference as TR
from prompt_lookup_gram_amd import binding as B
from test_attend_gpu import gpu  # noqa: F401
from test_tree_attend_gpu import Case

pytestmark = pytest.mark.gpu

CACHES = [("bf16", "bf16", "inf"), ("bf16", "bf16", "nan"), ("f16", "f16", "-inf"),
          ("f16", "f16", "nan"), ("bf16", "e4m3", "nan"), ("f16", "e4m3", "nan")]


def put(c, i, p, head, d, value):
    """Position p of request i: `value` in one dim of V, which the reference
    leaves out."""
    import torch
    page = int(c.table[i, p // c.page])
    c.vc[page, head, d, p % c.page] = torch.tensor(value).to(c.vc.dtype)
    c.vc64[page, head, d, p % c.page] = 0.0


def lift_keys(c, i, lo, hi, by):
    """Keys of positions [lo, hi) of request i times a power of two."""
    import torch
    for p in range(lo, hi):
        page, at = int(c.table[i, p // c.page]), p % c.page
        c.kc64[page, :, at] *= by
        c.kc[page, :, at] = torch.from_numpy(c.kc64[page, :, at]).float().to(c.kc.dtype).cuda()


def sees(c, i, t, p, window):
    root = c.lengths[i] - 1
    up = TR.branch(c.parent[i], t)
    if p > root:
        s = p - root
        return s in up and (not window or up.index(s) < window)
    return not window or p > root + len(up) - 1 - window


def check_hits(c, out, lse, hits, value, window):
    """Every row: the value in the dims of the hits that it sees, the reference's
    elsewhere."""
    import torch
    assert bool(torch.isfinite(lse).all())
    want = torch.from_numpy(c.reference(window)[0]).to(out.dtype).cuda()
    v, group, seen = float(value), c.hq // c.hk, []
    for i, p, head, d in hits:
        for t in range(R.block_rows(c.lengths[i], c.dlen[i])):
            heads = slice(head * group, (head + 1) * group)
            if sees(c, i, t, p, window):
                seen.append((i, t, heads, d))
                got = out[i, t, heads, d]
                assert bool((got.isnan() if v != v else got == v).all()), (i, t, p, d)
    assert seen
    for at in seen:
        out[at] = want[at]
    c.compare(out, lse, window)


# 24, 48, 64, 96 and 160 query rows a kv head
@pytest.mark.parametrize("hq,hk,rows", [(4, 2, 12), (8, 2, 12), (8, 1, 8), (8, 1, 12), (8, 1, 20)])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("dt,cache,value", CACHES)
def test_other_dims_do_not_feel_a_value_that_is_not_finite(dt, cache, value, dim, hq, hk, rows):
    c = Case([101, 230, 700, 33], [rows - 1, rows - 3, rows - 2, 5], rows, hq=hq, hk=hk, dim=dim,
             dt=dt, cache=cache, page=32, seed=21)
    # 101: the tile of 64 positions that holds the root has far larger scores in
    # its second half, so that the first half's weights are taken down
    lift_keys(c, 0, 96, 100 + rows, 4.0)
    hits = [(0, 70, 0, 3), (0, 71, hk - 1, dim - 1), (0, 105, 0, 17), (0, 106, hk - 1, 3),
            (1, 229, 0, 40), (1, 232, 0, 41), (2, 690, hk - 1, 9), (3, 0, 0, 33), (3, 35, 0, 0)]
    for i, p, head, d in hits:
        put(c, i, p, head, d, float(value))
    ctx = c.context()
    try:
        for window in (0, 50):
            out, lse = c.outputs()
            c.call(ctx, out, lse, window)
            assert B.pld_sync(ctx) == B.PLD_OK
            live = [(i, t) for i in range(4) for t in range(rows) if t > c.dlen[i]]
            for i, t in live:
                assert bool((out[i, t] == 7.0).all()) and bool((lse[i, t] == 7.0).all())
            check_hits(c, out, lse, hits, value, window)
    finally:
        B.pld_destroy(ctx)


# narrow (8 and 24 query rows), wide and many-row kernels
@pytest.mark.parametrize("hq,rows,dim", [(2, 4, 64), (2, 12, 128), (8, 12, 96), (8, 12, 128)])
@pytest.mark.parametrize("back", [0, 1, 31, 32])
def test_a_root_alone_sees_its_own_last_positions(hq, rows, dim, back):
    """A request without drafts in a batch of trees has no branches to look at:
    what a workgroup before it left behind says nothing about what it sees."""
    quiet = Case([40] * 600, [0] * 600, rows, hq=hq, hk=1, dim=dim, seed=22)
    quiet.vc.zero_()
    c = Case([70, 64, 33, 41], [0, 0, 0, rows - 1], rows, hq=hq, hk=1, dim=dim, seed=23)
    hits = [(i, c.lengths[i] - 1 - back, 0, 7 + i) for i in range(4)]
    for i, p, head, d in hits:
        put(c, i, p, head, d, float("inf"))
    first, ctx = quiet.context(), c.context()
    try:
        out, lse = quiet.outputs()
        quiet.call(first, out, lse)
        assert B.pld_sync(first) == B.PLD_OK
        out, lse = c.outputs()
        c.call(ctx, out, lse)
        assert B.pld_sync(ctx) == B.PLD_OK
        check_hits(c, out, lse, hits, "inf", 0)
    finally:
        B.pld_destroy(first)
        B.pld_destroy(ctx)


@pytest.mark.parametrize("hq", [16, 40])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,first", [(16, 80), (16, 64), (64, 64), (128, 128)])
def test_a_page_that_the_window_left_behind_is_not_needed_by_many_rows(hq, dim, cache, page, first):
    # (64 and 160 query rows a kv head: the many-row kernel has its own fetch)
    c = Case([200], [3], 4, "star", hq=hq, hk=1, dim=dim, cache=cache, page=page, seed=24)
    ctx = c.context()
    try:
        table = c.table.copy()
        table[0, :first // page] = -1
        out, lse = c.outputs()
        c.call(ctx, out, lse, window=200 - first, table=table)  # the root sees from `first` on
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(out, lse, window=200 - first)
        c.call(ctx, out, lse, window=201 - first, table=table)
        assert B.pld_sync(ctx) == B.PLD_EINVAL
        assert bool(out[0, 0].isnan().all())
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("hq,hk,dim,dt,cache", [(4, 2, 128, "bf16", "bf16"),
                                                (8, 2, 128, "f16", "e4m3"),
                                                (16, 1, 128, "bf16", "bf16"),
                                                (16, 1, 64, "f16", "e4m3"),
                                                (8, 1, 96, "bf16", "bf16")])
def test_ragged_batches_repeat_themselves_bit_for_bit(hq, hk, dim, dt, cache):
    """Another call between them, and the spans' partial results of another
    batch in the workspace, change nothing."""
    import torch
    rng = np.random.default_rng(9703)
    lengths = [int(n) for n in rng.integers(1, 9000, 12)]
    dlen = [int(n) for n in rng.integers(0, 12, 12)]
    c = Case(lengths, dlen, 12, hq=hq, hk=hk, dim=dim, dt=dt, cache=cache, page=64, seed=25)
    ctx = c.context()
    try:
        want = c.outputs()
        c.call(ctx, *want)
        for _ in range(6):
            other = c.outputs()
            c.again(ctx, *other, window=700)
            out, lse = c.outputs()
            c.again(ctx, out, lse)
            assert B.pld_sync(ctx) == B.PLD_OK
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    finally:
        B.pld_destroy(ctx)
