"""pld_verify's kernels on the host, against the 64-bit reference, over orders
in which the wavefronts of a workgroup may run (no GPU needed): results, the
counters left for the next call, and barriers that all of a workgroup reach.
The tolerance of log probabilities is test_verify_gpu.py's."""

from __future__ import annotations

import os
import re

import numpy as np
import pytest

import host_verify as H
import target_reference as R


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return H.build(tmp_path_factory.mktemp("host"))


class Case:
    def __init__(self, batch, rows, vocab, dtype=H.F32, seed=0, temperature=1.0, head=0, accept=0.7,
                 dlen=None, zero_excess=False):
        rng = np.random.default_rng([9501, seed])
        d = rows - 1
        z = rng.standard_normal((batch, rows, vocab)) * 2.0
        self.draft = rng.integers(0, vocab, (batch, max(1, d))).astype(np.int32)[:, :d]
        self.temp = np.broadcast_to(np.asarray(temperature, np.float32), (batch,)).copy()
        for b in range(batch):
            for t in range(d):
                x, scale = self.draft[b, t], self.temp[b] or 1.0
                w = np.exp(z[b, t] / scale)
                if vocab > 1:
                    z[b, t, x] = scale * np.log((w.sum() - w[x]) * accept / (1 - accept))
        self.logits, self.z = H.bits(z, dtype)
        self.dtype, self.rows, self.batch, self.vocab = dtype, rows, batch, vocab
        self.dlen = np.full(batch, d) if dlen is None else np.asarray(dlen)
        self.uniform = rng.random((batch, rows)).astype(np.float32)
        self.probs = None
        if head:
            p = np.exp(self.z[:, :head] - self.z[:, :head].max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            # (twice p: nothing exceeds it, the draw falls back to p)
            q = 2.0 * p if zero_excess else p * np.exp(0.5 * rng.standard_normal(p.shape))
            if zero_excess:
                self.uniform[:, :d] = 0.9
            else:
                q /= q.sum(-1, keepdims=True)
            self.probs = q.astype(np.float32)

    def run(self, ctx, **kw):
        return ctx.verify(self.logits, self.dtype, self.draft, self.dlen, self.uniform,
                          probs=self.probs, temperature=self.temp, **kw)

    def compare(self, got):
        tok, acc, cnt, logp = got[:4]
        for b in range(self.batch):
            d = int(self.dlen[b])
            if d < 0:
                assert (tok[b] == -1).all() and cnt[b] == 0
                continue
            head = 0 if self.probs is None else self.probs.shape[1]
            want, lp = R.verify_one(self.z[b], self.draft[b], d, [t < head for t in range(d)],
                                    None if self.probs is None else
                                    self.probs[b].astype(np.float64), float(self.temp[b]),
                                    self.uniform[b], self.uniform[b, -1])
            n = len(want)
            assert cnt[b] == n and acc[b] == n - 1, (b, cnt[b], n)
            assert tok[b].tolist() == want + [-1] * (self.rows - n), b
            assert (np.abs(logp[b, :n] - lp) <= 2.0**-17 + 2.0**-23 * np.abs(lp)).all()
            assert (logp[b, n:] == 0).all()


def check(lib, case):
    ctx = H.Context(lib, case.batch, case.rows, case.vocab)
    for order in H.ORDERS:
        got = case.run(ctx, order=order)
        case.compare(got)
        assert got[4] == 0
        assert ctx.clear(), order


@pytest.mark.parametrize("dtype", [H.F32, H.F16, H.BF16])
@pytest.mark.parametrize("vocab", [1, 700, 2049, 9000])
def test_point_masses(lib, dtype, vocab):
    check(lib, Case(3, 5, vocab, dtype=dtype, seed=vocab))


@pytest.mark.parametrize("head", [1, 3])
def test_drafter_probabilities(lib, head):
    check(lib, Case(4, 4, 3001, head=head, temperature=0.7, seed=head))


def test_zero_excess_draws_from_p(lib):
    c = Case(3, 3, 2500, head=2, zero_excess=True, seed=5)
    check(lib, c)


def test_greedy_idle_and_ragged_requests(lib):
    check(lib, Case(6, 5, 1200, temperature=[0.0, 1.0, 0.0, 0.5, 1.0, 2.0],
                    dlen=[4, 4, 0, -1, 2, 0], seed=6))


def test_more_rows_than_a_wavefront(lib):
    check(lib, Case(2, 70, 130, accept=0.95, seed=7))


def test_a_refusal_seen_by_part_of_a_workgroup(lib):
    """A row is refused while the wavefronts of a workgroup behind it start:
    all of them go on or none does, and the results are the same."""
    c = Case(2, 6, 5000, seed=8, accept=0.9)
    c.uniform[:, 1] = 1.0 - 2.0**-24      # refused at position 1 at the latest
    ctx = H.Context(lib, c.batch, c.rows, c.vocab)
    for order in H.ORDERS:
        got = c.run(ctx, order=order, refuse_row=1)
        c.compare(got)
        assert ctx.clear()
        assert got[5] == 0, f"{got[5]} barriers that part of a workgroup never reached"


def test_workspace_is_what_the_header_says(lib):
    with open(os.path.join(H.ROOT, "include", "pld.h")) as f:
        text = " ".join(line.strip().removeprefix("* ") for line in f)
    m = re.search(r"max_batch \* vocab \* \(max_rows / (\d+) \+ 1 / (\d+)\) bytes, plus (\d+) "
                  r"bytes a row and (\d+) a request", text)
    assert m, "the header states no bound"
    per_row, once, row, request = (int(x) for x in m.groups())
    for batch in (1, 3, 64):
        for rows in (1, 2, 17, 500):
            for vocab in (1, 511, 2048, 32000, 151936, 1 << 24):
                says = batch * (vocab * (rows / per_row + 1 / once) + rows * row + request)
                size = lib.host_workspace(batch, rows, vocab)
                # (the last piece of a row, and of a request's sums, is 16 bytes)
                assert 0 <= says - size <= 16 * batch * (rows + 1), (batch, rows, vocab)


@pytest.mark.parametrize("dtype", [H.F32, H.F16, H.BF16])
@pytest.mark.parametrize("head", [0, 1])
def test_full_batches(lib, dtype, head):
    """8,192 logits a piece and units of 2,048 to draw from: both draw
    launches, pieces and units that end inside a row of odd length."""
    c = Case(64, 4, 33001, dtype=dtype, head=head, accept=0.5, seed=20 + head,
             dlen=[3, 2, 1, 0] * 16)
    ctx = H.Context(lib, c.batch, c.rows, c.vocab)
    for order in H.ORDERS[:2]:
        got = c.run(ctx, order=order)
        c.compare(got)
        assert got[4] == 0 and ctx.clear()


def test_more_units_than_two_steps_of_a_wavefront_find(lib):
    """Above 64 * 64 units of 2,048 logits a lane's share of the units is
    itself searched in shares."""
    vocab = 64 * 64 * 2048 + 12345
    rng = np.random.default_rng(9502)
    z = rng.standard_normal((2, 1, vocab), dtype=np.float32)
    logits, z64 = H.bits(z, H.F16)
    u = np.array([[0.31], [1 - 2.0**-24]], np.float32)
    ctx = H.Context(lib, 2, 1, vocab)
    tok, acc, cnt, logp, err, _ = ctx.verify(logits, H.F16, np.zeros((2, 0)), [0] * 2, u)
    assert err == 0 and ctx.clear() and (acc == 0).all() and (cnt == 1).all()
    for b in range(2):
        p = np.exp(z64[b, 0] - z64[b, 0].max())
        c = np.cumsum(p)
        want = int(np.searchsorted(c, float(u[b, 0]) * c[-1], side="right"))
        # (sums in another order: 64-bit rounding over 8.4 million terms)
        slack = 2.0**-52 * vocab * c[-1]
        near = c[want] - float(u[b, 0]) * c[-1] > slack and (
            want == 0 or float(u[b, 0]) * c[-1] - c[want - 1] > slack)
        assert not near or tok[b, 0] == want, b
        assert abs(int(tok[b, 0]) - want) <= 1
        assert abs(logp[b, 0] - (z64[b, 0, tok[b, 0]] - z64[b, 0].max() - np.log(c[-1]))) <= (
            2.0**-17 + 2.0**-23 * 20)


@pytest.mark.parametrize("dtype", [H.F32, H.F16, H.BF16])
def test_grids_fit_the_hardwares_count_of_threads(lib, dtype):
    """A grid is counted in threads, in 32 bits: sizes beyond are refused."""
    ran = 0
    for batch, rows, vocab, head in [
            (1, 1, 1, 0), (64, 17, 151936, 0), (2**24 - 1, 1, 100, 0), (2**24, 1, 100, 0),
            (2**20, 15, 100, 0), (2**20, 17, 100, 0), (2**30, 1, 1, 0), (2**20, 1, 151936, 0),
            (2**15, 4, 2**24, 1), (1, 2**24, 2048, 0), (2**12, 2**12, 9000, 3)]:
        threads = lib.host_verify_grid(batch, rows, vocab, dtype, head)
        assert threads < 2**32, (batch, rows, vocab)
        ran += threads > 0
    assert ran == 4
