"""pld_verify_tree (HIP, gfx950) against the 64-bit reference: tokens, paths and
counts equal, log probabilities within their bound.

Tolerances are those of tests/test_verify_gpu.py: 2^-17 + 2^-23 |ln p|, rows
being summed in the same pieces. Tokens and paths are compared exactly: the
inputs' random numbers lie off the edges by far more than 64-bit rounding."""

from __future__ import annotations

import numpy as np
import pytest

import tree_reference as TR
from prompt_lookup_gram_amd import binding as B
from test_verify_gpu import context, gpu, torch_type  # noqa: F401

pytestmark = pytest.mark.gpu


class Rows:
    """A request's logits: the reference looks at the rows on the path."""

    def __init__(self, rows):
        self.rows = rows

    def __getitem__(self, t):
        return self.rows[t].double().cpu().numpy()


class Case:
    def __init__(self, batch, rows, vocab, dt="f32", seed=0, temperature=1.0, accept=0.8, pad=0,
                 offset=0, dlen=None, kind=None, spread=2.0, ties=False):
        import torch
        rng = np.random.default_rng([9821, seed])
        self.batch, self.rows, self.vocab, self.dt = batch, rows, vocab, dt
        d, self.stride = rows - 1, vocab + pad
        self.parent = np.array([TR.shapes(d)[kind] if kind else TR.random_tree(rng, d)
                                for _ in range(batch)], np.int32).reshape(batch, d)
        self.draft = rng.integers(0, vocab, (batch, d)).astype(np.int32)
        self.temp = np.broadcast_to(np.asarray(temperature, np.float32), (batch,)).copy()
        raw = torch.zeros(batch * rows * self.stride + offset, dtype=torch_type(dt))
        view = raw[offset:].view(batch, rows, self.stride)
        for b in range(batch):
            z = rng.standard_normal((rows, vocab)) * spread
            scale = float(self.temp[b]) or 1.0
            kids = np.bincount(self.parent[b], minlength=rows)
            for t in range(1, rows):
                p, x = self.parent[b, t - 1], self.draft[b, t - 1]
                if vocab == 1:
                    continue
                w = z[p] / scale
                w[x] = -np.inf
                rest = w.max() + np.log(np.exp(w - w.max()).sum())
                share = accept * rng.uniform(0.5, 1.0) / kids[p]
                z[p, x] = scale * (rest + np.log(share / (1 - share)))
                if self.temp[b] == 0 and rng.random() < accept / kids[p]:
                    z[p, x] = z[p].max() + 1
            view[b, :, :vocab] = torch.from_numpy(np.round(z) if ties else z).to(raw.dtype)
        view[..., vocab:] = float("nan")
        self.raw = raw.cuda()
        self.logits = self.raw[offset:].view(batch, rows, self.stride)
        self.dlen = np.full(batch, d) if dlen is None else np.asarray(dlen)
        self.u = rng.random((batch, rows)).astype(np.float32)

    def device(self):
        import torch
        i32 = dict(dtype=torch.int32, device="cuda")
        self.d_draft = torch.from_numpy(self.draft).cuda() if self.rows > 1 else None
        self.d_dlen = torch.tensor(self.dlen, **i32)
        self.d_parent = torch.from_numpy(self.parent).cuda() if self.rows > 1 else None
        self.d_temp = torch.from_numpy(self.temp).cuda()
        self.d_u = torch.from_numpy(self.u).cuda()

    def outputs(self):
        import torch
        n = (self.batch, self.rows)
        i32 = dict(dtype=torch.int32, device="cuda")
        return (torch.full(n, -7, **i32), torch.full(n, -7, **i32), torch.full(n[:1], -7, **i32),
                torch.full(n[:1], -7, **i32), torch.full(n, 7.0, device="cuda"))

    def call(self, ctx, out, stream=None):
        B.pld_verify_tree(ctx, self.logits, self.stride, self.rows, self.d_draft, self.d_dlen,
                          self.d_parent, self.d_temp, self.d_u, self.batch, *out, stream)

    def compare(self, out, skip=()):
        tok, path, acc, cnt, logp = [x.cpu().numpy() for x in out]
        z = [Rows(x[:, :self.vocab]) for x in self.logits]
        for b in range(self.batch):
            if b in skip or self.dlen[b] < 0:
                assert (tok[b] == -1).all() and (path[b] == -1).all() and (logp[b] == 0).all()
                assert acc[b] == 0 and cnt[b] == 0
                continue
            want, way, lp = TR.verify_one(z[b], self.draft[b], self.parent[b], int(self.dlen[b]),
                                          float(self.temp[b]), self.u[b], self.u[b, -1])
            n = len(want)
            assert tok[b, :n].tolist() == want and (tok[b, n:] == -1).all(), b
            assert path[b, :n].tolist() == way and (path[b, n:] == -1).all(), b
            assert acc[b] == n - 1 and cnt[b] == n
            assert (np.abs(logp[b, :n] - lp) <= 2.0**-17 + 2.0**-23 * np.abs(lp)).all()
            assert (logp[b, n:] == 0).all()


class Large(Case):
    """More than 256 MiB of logits, made on the GPU: only rows on the path are
    read."""

    def __init__(self, batch, rows, vocab, dt="f32", seed=0, temperature=1.0, accept=0.8, dlen=None,
                 kind=None, pad=0, offset=0):
        import torch
        rng = np.random.default_rng([9823, seed])
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.batch, self.rows, self.vocab, self.dt = batch, rows, vocab, dt
        d, self.stride = rows - 1, vocab + pad
        self.parent = np.array([TR.shapes(d)[kind] if kind else TR.random_tree(rng, d)
                                for _ in range(batch)], np.int32)
        self.draft = rng.integers(0, vocab, (batch, d)).astype(np.int32)
        self.temp = np.broadcast_to(np.asarray(temperature, np.float32), (batch,)).copy()
        self.raw = torch.full((batch * rows * self.stride + offset,), float("nan"),
                              dtype=torch_type(dt), device="cuda")
        assert self.raw.nbytes > 256 << 20
        self.logits = self.raw[offset:].view(batch, rows, self.stride)
        for b in range(batch):
            z = torch.randn((rows, vocab), generator=gen, device="cuda") * 2
            scale = float(self.temp[b]) or 1.0
            parent = torch.from_numpy(self.parent[b]).long().cuda()
            x = torch.from_numpy(self.draft[b]).long().cuda()
            kids = torch.bincount(parent, minlength=rows)[parent]
            share = accept * torch.rand(d, generator=gen, device="cuda") / kids
            z[parent, x] = scale * (torch.logsumexp(z / scale, 1)[parent] + torch.logit(share))
            if self.temp[b] == 0:
                hit = torch.rand(d, generator=gen, device="cuda") < accept / kids
                z[parent[hit], x[hit]] = z.amax(1)[parent[hit]] + 1
            self.logits[b, :, :vocab] = z.to(self.raw.dtype)
        self.dlen = np.full(batch, d) if dlen is None else np.asarray(dlen)
        self.u = rng.random((batch, rows)).astype(np.float32)


@pytest.mark.parametrize("dt,batch,rows,vocab", [("f32", 9, 50, 151936), ("f32", 40, 256, 7001),
                                                 ("bf16", 16, 64, 151936), ("f16", 64, 50, 50257),
                                                 ("bf16", 300, 80, 6000), ("f32", 2, 40, 1 << 20)])
def test_rows_on_the_path_alone(dt, batch, rows, vocab):
    rng = np.random.default_rng(batch)
    temp = rng.uniform(0.3, 1.4, batch)
    temp[::3] = 0.0
    c = Large(batch, rows, vocab, dt, seed=rows, temperature=temp, accept=0.95,
              dlen=[rows - 1] + [int(x) for x in rng.integers(-1, rows, batch - 1)])
    ctx = context(batch, rows, vocab)
    try:
        c.device()
        for _ in range(2):
            out = c.outputs()
            c.call(ctx, out)
            assert B.pld_sync(ctx) == B.PLD_OK, B.pld_last_error()
            c.compare(out)
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("kind", ["chain", "star", "binary"])
@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_shapes_on_the_path_alone(kind, temperature):
    c = Large(4, 256, 70001, seed=3, kind=kind, temperature=temperature, accept=0.98, pad=3,
              offset=1)
    ctx = context(4, 256, 70001)
    try:
        c.device()
        out = c.outputs()
        c.call(ctx, out)
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(out)
    finally:
        B.pld_destroy(ctx)


def test_the_path_alone_twice_at_once_in_graphs_and_with_bad_requests():
    """Two contexts' walks on two streams, more workgroups than the chip holds:
    neither waits for the other. Then a graph of one, replayed."""
    import torch
    cases = [Large(24, 128, 50001, "bf16", seed=20 + i, accept=0.97) for i in range(2)]
    ctxs = [context(24, 128, 50001) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    try:
        want = []
        for c, ctx in zip(cases, ctxs):
            c.parent[1, 5], c.u[2, 3], c.dlen[3] = 90, 1.5, 128
            c.logits[4, 0, 77] = float("nan")
            c.device()
            want.append(c.outputs())
            c.call(ctx, want[-1])
            assert B.pld_sync(ctx) == B.PLD_EINVAL
            c.compare(want[-1], skip=(1, 2, 3, 4))
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(8):
            for i, (c, ctx, st) in enumerate(zip(cases, ctxs, streams)):
                with torch.cuda.stream(st):
                    got[i].append(c.outputs())
                    c.call(ctx, got[i][-1])
        for i in range(2):
            assert B.pld_sync(ctxs[i], streams[i]) == B.PLD_EINVAL
            for out in got[i]:
                for x, y in zip(out, want[i]):
                    assert torch.equal(x, y)
        c, ctx, out = cases[0], ctxs[0], cases[0].outputs()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            c.call(ctx, out)
        rng = np.random.default_rng(9824)
        for i in range(3):
            c.u[5:] = rng.random((19, 128)).astype(np.float32)
            c.d_u.copy_(torch.from_numpy(c.u))
            for x in out:
                x.fill_(-3)
            graph.replay()
            torch.cuda.synchronize()
            c.compare(out, skip=(1, 2, 3, 4))
    finally:
        for ctx in ctxs:
            B.pld_destroy(ctx)


def check(*args, **kw):
    c = Case(*args, **kw)
    ctx = context(c.batch, c.rows, c.vocab)
    try:
        c.device()
        for _ in range(2):  # (the second call finds what the first left)
            out = c.outputs()
            c.call(ctx, out)
            assert B.pld_sync(ctx) == B.PLD_OK, B.pld_last_error()
            c.compare(out)
    finally:
        B.pld_destroy(ctx)
    return c


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 63, 64, 65, 511, 512, 513, 2047, 2049, 8191, 8193,
                                   32000, 50257])
@pytest.mark.parametrize("temperature", [0.0, 0.7])
def test_vocabularies(dt, vocab, temperature):
    check(3, 12, vocab, dt, seed=vocab, temperature=temperature, dlen=[11, 5, 0])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("batch,rows,vocab", [(4, 64, 50257), (2, 48, 151936), (9, 33, 100003),
                                              (1, 256, 65001), (70, 8, 32003)])
def test_large_calls(dt, batch, rows, vocab):
    rng = np.random.default_rng(batch)
    temp = rng.uniform(0.3, 1.4, batch)
    temp[::3] = 0.0
    check(batch, rows, vocab, dt, seed=rows, temperature=temp, accept=0.9,
          dlen=[rows - 1] + [int(x) for x in rng.integers(-1, rows, batch - 1)])


@pytest.mark.parametrize("kind", ["chain", "star", "comb", "binary"])
@pytest.mark.parametrize("rows", [2, 64, 65, 256])
@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_tree_shapes(kind, rows, temperature):
    check(4, rows, 777, kind=kind, seed=rows, temperature=temperature, accept=0.95)


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 0), (5, 3)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1001, 140003])
def test_strides_and_alignments(pad, offset, dt, vocab):
    check(2, 60, vocab, dt, seed=pad, pad=pad, offset=offset, temperature=0.8)


@pytest.mark.parametrize("cls,batch,rows,vocab", [(Case, 3, 20, 9000), (Large, 40, 256, 7001)])
def test_no_temperature_and_no_log_probabilities(cls, batch, rows, vocab):
    # (no temperature is 1, and no buffer for the log probabilities is none written)
    import torch
    c = cls(batch, rows, vocab, seed=29)
    ctx = context(batch, rows, vocab)
    try:
        c.device()
        want, out = c.outputs(), c.outputs()
        c.call(ctx, want)
        c.d_temp = None
        c.call(ctx, (*out[:4], None))
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(want)
        assert all(torch.equal(x, y) for x, y in zip(out[:4], want))
        c.call(ctx, out)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert torch.equal(out[4], want[4])
    finally:
        B.pld_destroy(ctx)


def test_ties_and_peaked_and_flat_rows():
    check(6, 20, 3000, "bf16", seed=1, temperature=0.0, ties=True)
    check(6, 20, 3000, seed=2, temperature=0.05, spread=6.0)
    check(6, 20, 30000, seed=3, spread=0.01, accept=0.3)
    check(6, 20, 30000, seed=4, temperature=100.0)


@pytest.mark.parametrize("vocab,rows", [(500, 20), (140000, 60)])
def test_masked_logits(vocab, rows):
    """Tokens of probability 0: -inf, also as drafted tokens, and a row whose
    only token is drafted."""
    import torch
    c = Case(3, rows, vocab, seed=5)
    c.logits[:, :, ::2] = -float("inf")
    c.logits[1, 0] = -float("inf")
    c.logits[1, 0, c.draft[1, 0]] = 2.0
    c.parent[1, 0] = 0
    c.logits[2, 0, int(c.draft[2, 0])] = -float("inf")
    # rows after the first keep a finite logit
    c.logits[:, 1:, 1] = 0.5
    ctx = context(3, rows, vocab)
    try:
        c.device()
        out = c.outputs()
        c.call(ctx, out)
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(out)
        assert torch.isfinite(out[4]).all()
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("rows,vocab", [(12, 300), (64, 140000)])
def test_far_and_rising_logits(rows, vocab):
    """Logits in the millions, and ones that rise along a row, so that a sum's
    base moves often."""
    import torch
    for dt in ("f32", "bf16"):
        c = Case(2, rows, vocab, dt, seed=6)
        ramp = torch.linspace(0, 300, vocab, device="cuda")
        c.logits[0] = (c.logits[0].float() + 3e6).to(c.logits.dtype)
        c.logits[1] = (c.logits[1].float() + ramp).to(c.logits.dtype)
        ctx = context(2, rows, vocab)
        try:
            c.device()
            out = c.outputs()
            c.call(ctx, out)
            assert B.pld_sync(ctx) == B.PLD_OK
            c.compare(out)
        finally:
            B.pld_destroy(ctx)


@pytest.mark.parametrize("vocab", [4000, 152000])
def test_decisions_next_to_their_edge(vocab):
    """Uniforms a few steps from the edge of a second child, which hangs on
    what the first one left."""
    rows = 4 if vocab < 10000 else 48
    base = Case(1, rows, vocab, seed=7, kind="star", accept=0.0001)
    base.draft[0, :2] = [0, 1]
    base.logits[0, 0, 0], base.logits[0, 0, 1] = 7.0, 7.5
    z = base.logits.double().cpu().numpy()[0, 0]
    p = np.exp(z - z.max())
    p /= p.sum()
    edge = np.float32(p[1] / (1 - p[0]))
    ctx = context(1, rows, vocab)
    try:
        for step in range(-3, 4):
            base.u[0, 0], base.u[0, 1] = 0.99999, edge + step * np.spacing(edge)
            base.device()
            out = base.outputs()
            base.call(ctx, out)
            assert B.pld_sync(ctx) == B.PLD_OK
            base.compare(out)
    finally:
        B.pld_destroy(ctx)


def test_draws_at_every_place():
    """The draw's uniform over its range, refused tokens among the likeliest."""
    for i in range(24):
        c = Case(1, 6, 5000, seed=8, kind="star", accept=0.5)
        c.u[0, :-1], c.u[0, -1] = 0.99999, np.float32(min(i / 23, 1 - 2**-24))
        ctx = context(1, 6, 5000)
        try:
            c.device()
            out = c.outputs()
            c.call(ctx, out)
            assert B.pld_sync(ctx) == B.PLD_OK
            c.compare(out)
        finally:
            B.pld_destroy(ctx)


@pytest.mark.parametrize("rows,vocab", [(8, 100), (64, 100000)])
def test_bad_requests_commit_nothing_and_spare_the_others(rows, vocab):
    names = ["parent", "parent up", "token", "uniform", "draw", "dlen", "low dlen", "nan", "inf",
             "empty row", "negative T", "tiny T", "nan T"]
    batch = len(names) + 1
    if rows == 64:
        names, batch = names[::3], len(names[::3]) + 1
    c = Case(batch, rows, vocab, seed=9, dt="bf16" if rows == 64 else "f32")
    for b, what in enumerate(names):
        if what == "parent":
            c.parent[b, 3] = 4
        elif what == "parent up":
            c.parent[b, 2] = -2
        elif what == "token":
            c.draft[b, rows - 2] = vocab
        elif what == "uniform":
            c.u[b, 2] = 1.0
        elif what == "draw":
            c.u[b, -1] = np.nan
        elif what == "dlen":
            c.dlen[b] = rows
        elif what == "low dlen":
            c.dlen[b] = -2
        elif what == "nan":
            c.logits[b, 0, vocab - 1] = float("nan")
        elif what == "inf":
            c.logits[b, 0, 3] = float("inf")
        elif what == "empty row":
            c.logits[b, 0] = -float("inf")
        else:
            c.temp[b] = {"negative T": -1.0, "tiny T": 1e-39, "nan T": np.nan}[what]
    ctx = context(batch, rows, vocab)
    try:
        c.device()
        out = c.outputs()
        c.call(ctx, out)
        assert B.pld_sync(ctx) == B.PLD_EINVAL
        c.compare(out, skip=range(len(names)))
        # a row that the path does not come to may hold anything, and so may
        # entries past d
        good = Case(2, rows, vocab, seed=10, kind="star", dlen=[2, rows - 1])
        good.u[:, :-1] = 0.999999
        good.logits[:, 1:] = float("nan")
        good.draft[0, 2:], good.parent[0, 2:] = -9, 1000
        z = good.logits.clone()
        good.device()
        small = context(2, rows, vocab)
        try:
            out = good.outputs()
            good.call(small, out)
            assert B.pld_sync(small) == B.PLD_OK
            good.logits = z
            good.compare(out)
        finally:
            B.pld_destroy(small)
    finally:
        B.pld_destroy(ctx)


def test_chains_are_the_chain_calls_and_both_share_a_context():
    import torch
    c = Case(6, 17, 9000, "bf16", seed=11, kind="chain", temperature=[0.7, 1, 0, 0.4, 1.2, 1],
             dlen=[16, 8, 16, 0, -1, 3])
    ctx = context(6, 17, 9000)
    try:
        c.device()
        for _ in range(2):
            tok, _, acc, cnt, logp = want = c.outputs()
            B.pld_verify(ctx, c.logits, c.stride, c.rows, c.d_draft, c.d_dlen, None, None, 0,
                         c.d_temp, c.d_u, c.batch, tok, acc, cnt, logp)
            for parent in (c.d_parent, None):
                c.d_parent, keep = parent, c.d_parent
                out = c.outputs()
                c.call(ctx, out)
                c.d_parent = keep
                assert B.pld_sync(ctx) == B.PLD_OK
                for i in (0, 2, 3):
                    assert torch.equal(out[i], want[i])
                c.compare(out)
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("rows,vocab", [(16, 5000), (48, 140000)])
def test_graph_replays_and_two_contexts_at_once(rows, vocab):
    import torch
    cases = [Case(3, rows, vocab, "bf16", seed=12 + i, accept=0.9) for i in range(2)]
    ctxs = [context(3, rows, vocab) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    try:
        want = []
        for c, ctx in zip(cases, ctxs):
            c.device()
            want.append(c.outputs())
            c.call(ctx, want[-1])
            assert B.pld_sync(ctx) == B.PLD_OK
            c.compare(want[-1])
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(6):
            for i, (c, ctx, st) in enumerate(zip(cases, ctxs, streams)):
                with torch.cuda.stream(st):
                    got[i].append(c.outputs())
                    c.call(ctx, got[i][-1])
        for i in range(2):
            assert B.pld_sync(ctxs[i], streams[i]) == B.PLD_OK
            for out in got[i]:
                for x, y in zip(out, want[i]):
                    assert torch.equal(x, y)
        c, ctx, out = cases[0], ctxs[0], cases[0].outputs()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            c.call(ctx, out)
        rng = np.random.default_rng(9822)
        for i in range(4):
            c.u = rng.random(c.u.shape).astype(np.float32)
            c.dlen = rng.integers(0, rows, 3)
            c.d_u.copy_(torch.from_numpy(c.u))
            c.d_dlen.copy_(torch.from_numpy(c.dlen.astype(np.int32)))
            for x in out:
                x.fill_(-3)
            graph.replay()
            torch.cuda.synchronize()
            c.compare(out)
        assert B.pld_sync(ctx) == B.PLD_OK
    finally:
        for ctx in ctxs:
            B.pld_destroy(ctx)


def test_refusals_on_a_context():
    c = Case(2, 6, 100, seed=14)
    ctx = context(2, 300, 100)
    c.device()
    tok, path, acc, cnt, logp = c.outputs()
    good = dict(logits=c.logits, logits_stride=100, rows=6, draft=c.d_draft, draft_len=c.d_dlen,
                parent=c.d_parent, temperature=c.d_temp, uniform=c.d_u, batch=2, out_tokens=tok,
                out_path=path, out_accepted=acc, out_counts=cnt, out_logprobs=logp)
    try:
        B.pld_verify_tree(ctx, **{**good, "batch": 0})
        for field, value in [("rows", 0), ("rows", 257), ("rows", 301), ("batch", 3),
                             ("logits_stride", 99), ("draft", None), ("draft_len", None),
                             ("uniform", None), ("out_tokens", None), ("out_path", None),
                             ("out_accepted", None), ("out_counts", None),
                             ("parent", c.d_parent.data_ptr() + 2),
                             ("out_path", path.data_ptr() + 2)]:
            with pytest.raises(B.PldError) as e:
                B.pld_verify_tree(ctx, **{**good, field: value})
            assert e.value.status == B.PLD_EINVAL, field
        for field, value in [("parent", c.d_parent.long()), ("out_path", path.long()),
                             ("logits", c.logits.double())]:
            with pytest.raises(ValueError):
                B.pld_verify_tree(ctx, **{**good, field: value})
        assert bool((tok == -7).all()) and B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)
