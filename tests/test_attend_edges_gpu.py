"""pld_attend (HIP, gfx950) at the edges of its arguments: scales so small
that they vanish in 32 bits, results in q's place, the loosest bound on
lengths, and more requests than the workspace holds partial results for.
Tolerances are test_attend_gpu.py's."""

from __future__ import annotations

import pytest

from prompt_lookup_gram_amd import binding as B
from test_attend_gpu import Case, check, gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [1e-45, -1e-45, 1e-39, 1e-30])
@pytest.mark.parametrize("rows", [1, 4, 20])
def test_scales_that_vanish_weigh_every_position_the_same(cache, scale, rows):
    # (1e-45 times a cell scale below 1 is 0; masked scores stay out all the same)
    check([70, 33, 300], [rows - 1, 0, rows // 2], rows, scale=scale, cache=cache, window=40,
          seed=20)


@pytest.mark.parametrize("rows,lengths", [(1, [70, 9000]), (4, [300, 20]), (8, [9000, 5]),
                                          (40, [700, 3])])
def test_out_in_the_place_of_q(rows, lengths):
    import torch
    c = Case(lengths, [rows - 1, rows // 2], rows, hq=8, hk=2, dim=128, page=64, seed=21)
    ctx = c.context()
    try:
        out, lse = c.outputs()
        c.call(ctx, out, lse)
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(out, lse)
        q, again = c.q, torch.empty_like(lse).fill_(7.0)
        c.q = q.clone()
        c.call(ctx, c.q, again)
        assert B.pld_sync(ctx) == B.PLD_OK
        got = c.q.view(out.shape)
        for i in range(2):
            n = c.dlen[i] + 1
            assert torch.equal(got[i, :n], out[i, :n]) and torch.equal(again[i, :n], lse[i, :n])
            # rows past the block are left as they were
            assert torch.equal(got[i, n:], q.view(out.shape)[i, n:])
    finally:
        B.pld_destroy(ctx)


def test_out_over_strided_q_is_refused():
    import torch
    c = Case([50, 20], [2, 1], 3, pad=24, seed=22)
    ctx = c.context()
    try:
        kept = c.q.clone()
        with pytest.raises(B.PldError, match="q_stride") as e:
            c.call(ctx, c.q, None)
        assert e.value.status == B.PLD_EINVAL
        assert B.pld_sync(ctx) == B.PLD_OK and torch.equal(c.q, kept)
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("rows", [1, 5, 20])
@pytest.mark.parametrize("window", [0, 50])
def test_the_largest_bound_on_lengths(rows, window):
    c = Case([700, 9, 5000], [rows - 1, 0, rows // 2], rows, hq=8, hk=2, page=256, seed=23)
    ctx = c.context(max_len=2**30)
    try:
        for max_len in (0, 2**30 - 7, c.max_len):
            out, lse = c.outputs()
            c.call(ctx, out, lse, window, max_len=max_len)
            assert B.pld_sync(ctx) == B.PLD_OK
            c.compare(out, lse, window)
    finally:
        B.pld_destroy(ctx)


def test_more_requests_than_workgroups_to_split_among():
    lengths = [1 + 37 * i % 600 for i in range(1500)]
    check(lengths, [i % 3 - 1 for i in range(1500)], 2, hq=8, hk=4, seed=24)
