"""pld_verify (HIP, gfx950) at the sizes where it takes its other variants:
8,192 logits a piece and 2,048 a unit of the draw (full batches), both sides of
the sizes that choose them, vocabularies whose units are searched in more than
two steps, and two contexts at work at once. Tolerances are
test_verify_gpu.py's."""

from __future__ import annotations

import numpy as np
import pytest

from prompt_lookup_gram_amd import binding as B
from test_verify_gpu import Case, check, context, gpu, torch_type  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("head,src", [(0, False), (3, False), (3, True)])
@pytest.mark.parametrize("ragged", [False, True])
def test_full_batches(dt, head, src, ragged):
    dlen = [3, 2, 1, 0, -1, 3, 2, 1] * 8 if ragged else None
    acc = check(64, 4, 50257, dt=dt, head=head, src=src, temperature=0.8, dlen=dlen,
                seed=30 + head)
    assert acc.max() == 3 and acc.min() < 3


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_full_batches_of_mixed_temperatures(dt):
    check(64, 4, 50257, dt=dt, head=2, temperature=np.tile([0.0, 0.5, 1.0, 2.0], 16), seed=34)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_full_batches_greedy_with_ties(dt):
    check(64, 4, 33001, dt=dt, temperature=0.0, ties=True, spread=0.7, seed=35)


def test_full_batches_whose_excess_is_zero_draw_from_p():
    c = Case(64, 3, 40001, seed=36, head=2)
    e = np.exp(c.z[:, :2] - c.z[:, :2].max(-1, keepdims=True))
    c.probs = (2.0 * e / e.sum(-1, keepdims=True)).astype(np.float32)
    c.uniform[:, :2] = 0.9
    ctx = context(64, 3, 40001)
    try:
        out = c.outputs()
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert (c.compare(out) == 0).all()
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("vocab", [32767, 32768, 32769])
@pytest.mark.parametrize("head", [0, 1])
def test_both_sides_of_the_draws_unit(vocab, head):
    # 64 * 32768 = 2^21
    check(64, 2, vocab, dt="bf16", head=head, seed=vocab)


@pytest.mark.parametrize("batch,rows", [(73, 7), (64, 8), (57, 9)])
@pytest.mark.parametrize("vocab", [8192, 8191])
@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_many_pieces_of_many_requests(batch, rows, vocab, dt):
    # 511, 512 and 513 pieces of 8,192
    check(batch, rows, vocab, dt=dt, seed=batch)


@pytest.mark.parametrize("rows,vocab", [(31, 8192), (32, 8192), (33, 8192), (8, 24577),
                                        (7, 32768), (40, 2048), (40, 2049)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_few_pieces_of_one_request(rows, vocab, dt):
    # 31, 32 and 33 pieces of 8,192, 32 and 28 of several a row; rows of one
    # short piece and of one more logit
    check(1, rows, vocab, dt=dt, accept=0.95, seed=rows)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_vocabularies_of_more_than_4096_units(dt):
    """Above 64 * 64 units of 2,048 logits a lane's share of the units is
    itself searched in shares."""
    import torch
    vocab = 64 * 64 * 2048 + 12345
    gen = torch.Generator(device="cuda")
    gen.manual_seed(37)
    z = torch.randn((6, 1, vocab), generator=gen, device="cuda").to(torch_type(dt))
    z[5, 0, :8000000] = -float("inf")
    u = torch.tensor([0.0, 0.1, 0.31, 0.77, 1 - 2.0**-24, 0.5], device="cuda")[:, None]
    i32 = dict(dtype=torch.int32, device="cuda")
    tok, acc, cnt = torch.empty((6, 1), **i32), torch.empty(6, **i32), torch.empty(6, **i32)
    logp = torch.empty((6, 1), device="cuda")
    ctx = context(6, 1, vocab)
    try:
        for _ in range(2):
            B.pld_verify(ctx, z, vocab, 1, None, torch.zeros(6, **i32), None, None, 0, None, u, 6,
                         tok, acc, cnt, logp)
            assert B.pld_sync(ctx) == B.PLD_OK
            assert bool((acc == 0).all()) and bool((cnt == 1).all())
            for b in range(6):
                x = z[b, 0].double().cpu().numpy()
                c = np.cumsum(np.exp(x - x.max()))
                goal, got = float(u[b, 0]) * c[-1], int(tok[b, 0])
                # (sums in another order: 64-bit rounding over 8.4 million terms)
                slack = 2.0**-52 * vocab * c[-1]
                assert c[got] > goal - slack and (got == 0 or c[got - 1] <= goal + slack), b
                want = x[got] - x.max() - np.log(c[-1])
                assert abs(float(logp[b, 0]) - want) <= 2.0**-17 + 2.0**-23 * abs(want)
    finally:
        B.pld_destroy(ctx)


def test_many_requests_of_a_small_vocabulary():
    check(5000, 3, 97, dt="bf16", seed=38, temperature=np.tile([1.0, 0.0], 2500),
          dlen=[2, 1, 0, -1, 2] * 1000)


def test_two_contexts_on_two_streams_at_once():
    """Each context's workspace is its own: calls overlapping on two streams,
    then captured into two graphs that replay at the same time, give what
    they give one after the other."""
    import torch
    cases = [Case(24, 9, 30011, dt="bf16", seed=40, accept=0.9),
             Case(16, 6, 20001, head=4, src=True, temperature=0.8, seed=41)]
    ctxs = [context(c.batch, c.rows, c.vocab) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    try:
        args, want = [c.args() for c in cases], []
        for c, ctx, a in zip(cases, ctxs, args):
            want.append(c.outputs())
            B.pld_verify(ctx, *a, *want[-1])
            assert B.pld_sync(ctx) == B.PLD_OK
            c.compare(want[-1])
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(8):
            for i, (c, ctx, st) in enumerate(zip(cases, ctxs, streams)):
                with torch.cuda.stream(st):
                    got[i].append(c.outputs())
                    B.pld_verify(ctx, *args[i], *got[i][-1])
        graphs, outs = [], []
        for i, (c, ctx, st) in enumerate(zip(cases, ctxs, streams)):
            assert B.pld_sync(ctx, st) == B.PLD_OK
            for out in got[i]:
                assert all(torch.equal(x, y) for x, y in zip(out, want[i]))
            outs.append(c.outputs())
            graphs.append(torch.cuda.CUDAGraph())
            torch.cuda.synchronize()
            with torch.cuda.graph(graphs[i], stream=st):
                B.pld_verify(ctx, *args[i], *outs[i])
        for _ in range(5):
            for out in outs:
                for x in out:
                    x.fill_(-9)
            torch.cuda.synchronize()
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
            torch.cuda.synchronize()
            for out, ref in zip(outs, want):
                assert all(torch.equal(x, y) for x, y in zip(out, ref))
    finally:
        for ctx in ctxs:
            B.pld_destroy(ctx)
