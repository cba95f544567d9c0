"""pld_verify_tree's kernels themselves, run on the CPU a workgroup at a time
in several orders of its wavefronts (tests/host_device): results against the
64-bit reference, the counters and the workspace that the next call finds, and
barriers that all of a workgroup reach (no GPU needed)."""

from __future__ import annotations

import numpy as np
import pytest

import host_tree as T
import host_verify as H
import tree_reference as TR


@pytest.fixture(scope="module")
def libs(tmp_path_factory):
    folder = tmp_path_factory.mktemp("host_tree")
    return H.build(folder), T.build(folder, "tree_verify.cpp")


def trees(rng, batch, d, kind=None):
    return [TR.shapes(d)[kind] if kind else TR.random_tree(rng, d) for _ in range(batch)]


def inputs(rng, batch, d, vocab, dtype, parent, temperature, sure=0.8):
    """Logits whose children hold `sure` of their parent's mass."""
    z = rng.standard_normal((batch, d + 1, vocab)) * 2
    draft = rng.integers(0, vocab, (batch, max(1, d)))
    for b in range(batch):
        scale = temperature[b] if temperature[b] > 0 else 1.0
        for t in range(1, d + 1):
            p = parent[b][t - 1]
            kids = sum(1 for s in parent[b] if s == p)
            row = z[b, p] / scale
            m = np.delete(row, draft[b, t - 1])
            rest = m.max() + np.log(np.exp(m - m.max()).sum())
            share = sure * rng.uniform(0.5, 1.0) / kids
            z[b, p, draft[b, t - 1]] = scale * (rest + np.log(share / (1 - share)))
    raw, z64 = H.bits(z, dtype)
    return raw, z64, draft.astype(np.int32), rng.random((batch, d + 1)).astype(np.float32)


def compare(got, z64, draft, dlen, parent, u, temperature):
    tok, path, acc, cnt, logp, err, broken = got
    assert err == 0 and broken == 0
    for b in range(len(dlen)):
        if dlen[b] < 0:
            assert (tok[b] == -1).all() and (path[b] == -1).all() and acc[b] == 0 and cnt[b] == 0
            continue
        want, way, lp = TR.verify_one(z64[b], draft[b], parent[b], dlen[b],
                                      float(np.float32(temperature[b])), u[b], u[b, -1])
        n = len(want)
        assert tok[b, :n].tolist() == want and (tok[b, n:] == -1).all()
        assert path[b, :n].tolist() == way and (path[b, n:] == -1).all()
        assert acc[b] == n - 1 and cnt[b] == n
        # sums in 32 bits are good to 2^-17, the result is rounded to 32
        assert np.abs(logp[b, :n] - lp).max() <= 2.0**-17 + 2.0**-23 * np.abs(lp).max()
        assert (logp[b, n:] == 0).all()


@pytest.mark.parametrize("walk", [False, True])
@pytest.mark.parametrize("dtype", [H.F32, H.F16, H.BF16])
@pytest.mark.parametrize("batch,d,vocab", [(3, 0, 700), (2, 7, 1500), (3, 15, 2049), (2, 70, 301),
                                           (1, 255, 130), (2, 9, 9000)])
def test_both_ways_to_read(libs, dtype, batch, d, vocab, walk):
    rng = np.random.default_rng([9601, dtype, d])
    parent = trees(rng, batch, d)
    temp = rng.uniform(0.4, 1.3, batch)
    temp[-1] = 0.0 if batch > 1 else temp[-1]
    raw, z64, draft, u = inputs(rng, batch, d, vocab, dtype, parent, temp)
    dlen = [d] + [int(rng.integers(-1, d + 1)) for _ in range(batch - 1)]
    ctx = H.Context(libs[0], batch, d + 1, vocab)
    for order in H.ORDERS:
        got = T.verify(libs[1], ctx, raw, dtype, draft[:, :d], dlen, parent if d else None, u,
                       temp, order, walk)
        compare(got, z64, draft, dlen, parent, u, temp)
        assert ctx.clear()


@pytest.mark.parametrize("walk", [False, True])
@pytest.mark.parametrize("kind", ["chain", "star", "comb", "binary"])
@pytest.mark.parametrize("temperature", [0.0, 0.7])
def test_tree_shapes(libs, kind, temperature, walk):
    rng = np.random.default_rng([9603, len(kind)])
    batch, d, vocab = 4, 20, 90
    parent = trees(rng, batch, d, kind)
    temp = [temperature] * batch
    raw, z64, draft, u = inputs(rng, batch, d, vocab, H.F32, parent, temp, 0.9)
    dlen = [d, d, 5, 0]
    ctx = H.Context(libs[0], batch, d + 1, vocab)
    got = T.verify(libs[1], ctx, raw, H.F32, draft, dlen, parent, u, temp, walk=walk)
    compare(got, z64, draft, dlen, parent, u, temp)


def test_the_same_token_below_a_node_twice(libs):
    rng = np.random.default_rng(9604)
    batch, d, vocab = 6, 12, 8
    parent = [TR.random_tree(rng, d, kids=12, on=0.2) for _ in range(batch)]
    z = rng.standard_normal((batch, d + 1, vocab)).astype(np.float32)
    draft = rng.integers(0, vocab, (batch, d)).astype(np.int32)
    u = rng.random((batch, d + 1)).astype(np.float32)
    ctx = H.Context(libs[0], batch, d + 1, vocab)
    got = T.verify(libs[1], ctx, z, H.F32, draft, [d] * batch, parent, u, [1.0] * batch)
    compare(got, z.astype(np.float64), draft, [d] * batch, parent, u, [1.0] * batch)


def test_decisions_next_to_their_edge(libs):
    """Uniforms on both sides of the edge, where the 32-bit sum cannot tell:
    the first child refused, the second's edge hangs on what that left."""
    rng = np.random.default_rng(9605)
    vocab, d = 4000, 3
    z = rng.standard_normal((1, d + 1, vocab)).astype(np.float32)
    z[0, 0, :2] = [7.0, 7.5]
    p = np.exp(z[0, 0].astype(np.float64))
    p /= p.sum()
    draft, parent = np.array([[0, 1, 2]], np.int32), [[0, 0, 0]]
    edge = np.float32(p[1] / (1 - p[0]))
    ctx = H.Context(libs[0], 1, d + 1, vocab)
    for step in range(-3, 4):
        u = np.array([[0.999, edge + step * np.spacing(edge), 0.9, 0.5]], np.float32)
        got = T.verify(libs[1], ctx, z, H.F32, draft, [d], parent, u)
        compare(got, z.astype(np.float64), draft, [d], parent, u, [1.0])


@pytest.mark.parametrize("walk", [False, True])
def test_bad_requests_commit_nothing_and_are_flagged(libs, walk):
    rng = np.random.default_rng(9606)
    batch, d, vocab = 8, 6, 50
    parent = np.array([TR.random_tree(rng, d) for _ in range(batch)], np.int32)
    z = rng.standard_normal((batch, d + 1, vocab)).astype(np.float32)
    draft = rng.integers(0, vocab, (batch, d)).astype(np.int32)
    u = rng.random((batch, d + 1)).astype(np.float32)
    dlen, temp = np.full(batch, d), np.ones(batch, np.float32)
    parent[0, 3] = 4      # itself
    parent[1, 2] = -1
    draft[2, 5] = vocab
    u[3, 2] = 1.0
    dlen[4] = d + 1
    z[5, 0, 7] = np.nan
    temp[6] = -1.0
    ctx = H.Context(libs[0], batch, d + 1, vocab)
    tok, path, acc, cnt, logp, err, broken = T.verify(libs[1], ctx, z, H.F32, draft, dlen, parent,
                                                      u, temp, walk=walk)
    assert err == H.BAD_BLOCK and broken == 0 and ctx.clear()
    assert (tok[:7] == -1).all() and (path[:7] == -1).all()
    assert (acc[:7] == 0).all() and (cnt[:7] == 0).all() and (logp[:7] == 0).all()
    assert cnt[7] >= 1
    # entries past d are not read
    parent[7, 3:] = 99
    draft[7, 3:] = -5
    dlen[:] = [-1] * 7 + [3]
    got = T.verify(libs[1], ctx, z, H.F32, draft, dlen, parent, u, np.ones(batch), walk=walk)
    assert ctx.clear()
    compare(got, z.astype(np.float64), draft, dlen, parent, u, np.ones(batch))


def test_chains_are_the_chain_calls(libs):
    rng = np.random.default_rng(9607)
    batch, d, vocab = 5, 9, 600
    parent = trees(rng, batch, d, "chain")
    temp = [0.8, 1.0, 0.0, 0.5, 1.2]
    raw, z64, draft, u = inputs(rng, batch, d, vocab, H.BF16, parent, temp)
    dlen = [d, 4, d, 0, -1]
    ctx = H.Context(libs[0], batch, d + 1, vocab)
    want = ctx.verify(raw, H.BF16, draft, dlen, u, temperature=temp)
    for p in (parent, None):
        got = T.verify(libs[1], ctx, raw, H.BF16, draft, dlen, p, u, temp)
        for x, y in zip((got[0], got[2], got[3], got[4]), want):
            assert np.array_equal(x, y)


def test_grids_fit_the_hardware(libs):
    """Sizes that pass the argument checks are launched with fewer than 2^32
    threads, or refused."""
    for batch, rows, vocab in [(1, 1, 1), (64, 64, 151936), (1 << 16, 256, 1 << 24),
                               (1 << 22, 256, 1 << 24), (1 << 22, 1, 1)]:
        n = libs[1].host_verify_tree_grid(batch, rows, vocab, H.BF16)
        assert n < 2**32
    assert libs[1].host_verify_tree_grid(1 << 22, 256, 1 << 24, H.BF16) == 0
