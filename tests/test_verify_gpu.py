"""pld_verify (HIP, gfx950) against the 64-bit reference: tokens and counts
equal, log probabilities within their bound.

Tolerance of a log probability: ln p = (z - top) / T - ln(sum). The kernel's
sum of exponentials: an argument y is off by at most 1.5 * 2^-23 |y| (its
factor's two roundings and its own), which the softmax weighs to at most
1.5 ln V * 2^-23 < 19 * 2^-23 (the mean of |y| under the softmax is at most
ln V), the function by 2^-23, 40 additions by 20 * 2^-23: 40 * 2^-23 < 2^-17 in
all. The result is rounded to 32 bits once: 2^-17 + 2^-23 |ln p|. Tokens are compared exactly: the inputs' random
numbers lie off the edges by far more than 64-bit rounding."""

from __future__ import annotations

import numpy as np
import pytest

import target_reference as R
from prompt_lookup_gram_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.load()
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def context(batch, rows, vocab):
    p = B.pld_target_params_default()
    p.max_batch, p.max_rows, p.vocab = batch, rows, vocab
    return B.pld_create_target(p)


def torch_type(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


class Case:
    def __init__(self, batch, rows, vocab, dt="f32", seed=0, temperature=1.0, head=0, src=False,
                 accept=0.7, pad=0, offset=0, dlen=None, spread=2.0, ties=False):
        import torch
        rng = np.random.default_rng([9301, seed])
        self.batch, self.rows, self.vocab, self.head = batch, rows, vocab, head
        d = rows - 1
        self.stride = vocab + pad
        z = rng.standard_normal((batch, rows, vocab)) * spread
        self.draft = rng.integers(0, vocab, (batch, max(1, d))).astype(np.int32)[:, :d]
        self.temp = np.broadcast_to(np.asarray(temperature, np.float32), (batch,)).copy()
        for b in range(batch):
            for t in range(d):
                x = self.draft[b, t]
                if self.temp[b] == 0:
                    z[b, t, x] = z[b, t].max() + 1 if rng.random() < accept else -9.0
                elif self.temp[b] < 0.04:
                    # the same as below where exp(z / T) overflows
                    w = np.delete(z[b, t], x) / self.temp[b]
                    rest = w.max() + np.log(np.exp(w - w.max()).sum())
                    z[b, t, x] = self.temp[b] * (rest + np.log(accept / (1 - accept)))
                else:
                    # the draft token at probability `accept`
                    w = np.exp(z[b, t] / self.temp[b])
                    rest = w.sum() - w[x]
                    if vocab > 1:
                        z[b, t, x] = self.temp[b] * np.log(rest * accept / (1 - accept))
        if ties:
            z = np.round(z)
        raw = torch.zeros(batch * rows * self.stride + offset, dtype=torch_type(dt))
        view = raw[offset:].view(batch, rows, self.stride)
        view[..., :vocab] = torch.from_numpy(z).to(raw.dtype)
        view[..., vocab:] = float("nan")
        self.raw = raw.cuda()
        self.logits = self.raw[offset:].view(batch, rows, self.stride)
        self.z = self.logits.double().cpu().numpy()[..., :vocab]
        self.dlen = np.full(batch, d) if dlen is None else np.asarray(dlen)
        self.uniform = rng.random((batch, rows)).astype(np.float32)
        self.probs = None
        if head:
            q = np.exp(self.z[:, :head] / np.maximum(self.temp, 0.1)[:, None, None] +
                       0.5 * rng.standard_normal((batch, head, vocab)))
            self.probs = (q / q.sum(-1, keepdims=True)).astype(np.float32)
        self.src = rng.integers(0, 2**rows, batch).astype(np.int64) if src else None

    def device(self, x, dt=None):
        import torch
        return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def outputs(self):
        import torch
        n = (self.batch, self.rows)
        return (torch.full(n, -7, dtype=torch.int32, device="cuda"),
                torch.full(n[:1], -7, dtype=torch.int32, device="cuda"),
                torch.full(n[:1], -7, dtype=torch.int32, device="cuda"),
                torch.full(n, 7.0, dtype=torch.float32, device="cuda"))

    def args(self):
        return (self.logits, self.stride, self.rows,
                self.device(self.draft) if self.rows > 1 else None,
                self.device(self.dlen.astype(np.int32)), self.device(self.src),
                self.device(self.probs), self.head, self.device(self.temp),
                self.device(self.uniform), self.batch)

    def reference(self):
        tok = np.full((self.batch, self.rows), -1)
        logp = np.zeros((self.batch, self.rows))
        count = np.zeros(self.batch, int)
        for b in range(self.batch):
            d = int(self.dlen[b])
            if d < 0:
                continue
            claimed = [t < self.head and not (self.src is not None and (self.src[b] >> t) & 1)
                       for t in range(self.rows)]
            tk, lp = R.verify_one(self.z[b], self.draft[b], d, claimed,
                                  None if self.probs is None else
                                  self.probs[b].astype(np.float64), float(self.temp[b]),
                                  self.uniform[b], self.uniform[b, -1])
            tok[b, :len(tk)], logp[b, :len(tk)], count[b] = tk, lp, len(tk)
        return tok, np.maximum(count - 1, 0), count, logp

    def compare(self, out):
        tok, acc, cnt, logp = self.reference()
        g = [x.cpu().numpy() for x in out]
        assert np.array_equal(g[1], acc), (g[1], acc)
        assert np.array_equal(g[2], cnt)
        assert np.array_equal(g[0], tok), np.argwhere(g[0] != tok)[:5]
        assert (np.abs(g[3] - logp) <= 2.0**-17 + 2.0**-23 * np.abs(logp)).all()
        return acc


def check(*args, **kw):
    c = Case(*args, **kw)
    ctx = context(c.batch, c.rows, c.vocab)
    try:
        out = c.outputs()
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK, B.pld_last_error()
        return c.compare(out)
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 65, 255, 1000, 2047, 2048, 2049, 4097, 8191,
                                   8192, 8193, 32000, 50257])
def test_vocabularies_and_types(dt, vocab):
    check(5, 4, vocab, dt=dt, seed=vocab)


@pytest.mark.parametrize("rows", [1, 2, 8, 17, 65])
@pytest.mark.parametrize("batch", [1, 33])
def test_block_sizes(rows, batch):
    acc = check(batch, rows, 999, seed=rows, accept=0.9)
    if rows == 17 and batch > 1:
        assert acc.min() < 4 and acc.max() > 12


@pytest.mark.parametrize("temperature", [0.05, 0.7, 1.0, 3.0, 0.0])
@pytest.mark.parametrize("head", [0, 3, 6])
def test_temperatures_and_drafters(temperature, head):
    check(24, 7, 3001, temperature=temperature, head=head, seed=head + 1)


@pytest.mark.parametrize("temperature", [1e-4, 1e-8, 1e-20, 2e-38])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_tiny_temperatures_are_near_greedy_and_valid(temperature, dt):
    check(8, 4, 5001, dt=dt, temperature=temperature, seed=5, accept=0.4)


def test_far_logits():
    """Every logit near 1e6: only their differences count."""
    c = Case(6, 3, 3000, seed=6)
    c.logits[..., :3000] = torch_round(c.logits[..., :3000] * 4) / 4 + 2.0**20
    c.z = c.logits.double().cpu().numpy()[..., :3000]
    ctx = context(6, 3, 3000)
    try:
        out = c.outputs()
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(out)
    finally:
        B.pld_destroy(ctx)


def torch_round(x):
    import torch
    return torch.round(x)


def test_mixed_temperatures_and_sources():
    check(32, 9, 1501, temperature=np.tile([0.0, 0.5, 1.0, 2.0], 8), head=8, src=True, seed=3)
    check(32, 9, 1501, temperature=np.tile([0.0, 0.5, 1.0, 2.0], 8), head=5, seed=4)


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (13, 3)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_odd_strides_and_offsets(pad, offset, dt):
    check(4, 5, 4999, dt=dt, pad=pad, offset=offset, seed=pad)


def test_ragged_and_idle_requests():
    check(8, 6, 777, dlen=[-1, 0, 1, 2, 3, 4, 5, -1], seed=5)
    check(2, 6, 777, dlen=[-1, -1], seed=6)


def test_greedy_ties_go_to_the_lowest_index():
    acc = check(16, 5, 700, temperature=0.0, ties=True, dt="bf16", accept=0.8, seed=7)
    assert acc.max() > 0
    check(16, 1, 5000, temperature=0.0, ties=True, seed=8, spread=0.4)


def test_flat_and_peaked_rows():
    check(16, 3, 60000, spread=0.0, accept=1e-5, seed=9)
    check(16, 3, 60000, spread=12.0, seed=10)


def test_masked_tokens_are_never_committed():
    c = Case(8, 4, 300, seed=11)
    c.logits[..., 100:200] = -float("inf")
    c.logits[3, :, :] = -float("inf")
    c.logits[3, :, 250] = 1.0       # one token left
    c.z = c.logits.double().cpu().numpy()
    c.draft[:4, 0] = 150            # a masked draft token is refused ...
    c.uniform[0, 0] = 0.0           # ... at u = 0 too
    ctx = context(8, 4, 300)
    try:
        out = c.outputs()
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK
        acc = c.compare(out)
        assert (acc[:4] == 0).all() and int(out[0][3, 0]) == 250
    finally:
        B.pld_destroy(ctx)


def test_edges_of_the_random_numbers():
    c = Case(6, 2, 5000, seed=12, dlen=[0] * 6)
    top = np.float32(1.0 - 2.0**-24)
    c.uniform[:, -1] = [0.0, top, 0.0, top, 2.0**-24, 0.5]
    c.logits[2, 0, :4000] = -float("inf")
    c.logits[3, 0, 77:] = -float("inf")
    c.z = c.logits.double().cpu().numpy()
    ctx = context(6, 2, 5000)
    try:
        out = c.outputs()
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(out)
        got = out[0][:, 0].tolist()
        assert got[0] == 0 and got[2] == 4000 and got[3] == 76
    finally:
        B.pld_destroy(ctx)


def test_acceptance_next_to_its_edge():
    """u just below and just above p(x), in 32-bit steps of u: the decision
    is the 64-bit one on both sides."""
    c = Case(64, 2, 30000, seed=13, accept=0.5)
    p = []
    for b in range(64):
        z = c.z[b, 0]
        e = np.exp(z - z.max())
        p.append(e[c.draft[b, 0]] / e.sum())
    near = np.array(p).astype(np.float32)
    c.uniform[:, 0] = [np.nextafter(x, np.float32(b % 2)) if b % 4 < 2 else x
                       for b, x in enumerate(near)]
    ctx = context(64, 2, 30000)
    try:
        out = c.outputs()
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK
        acc = c.compare(out)
        assert 0 < acc.sum() < 64
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("dt,vocab", [("bf16", 151936), ("f32", 50257), ("f16", 700)])
@pytest.mark.parametrize("rel", [2.0**-24, 2.0**-21, 2.0**-18, 2.0**-15])
def test_acceptance_at_distances_that_take_different_sums(dt, vocab, rel):
    """u a given relative distance off p(x), above and below: the 32-bit sum,
    the one with 64-bit arguments and the 64-bit one agree on the side."""
    c = Case(4, 2, vocab, dt=dt, seed=18, accept=0.5)
    for b in range(4):
        e = np.exp(c.z[b, 0] - c.z[b, 0].max())
        c.uniform[b, 0] = e[c.draft[b, 0]] / e.sum() * (1 + rel * (-1) ** b)
    ctx = context(4, 2, vocab)
    try:
        out = c.outputs()
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK
        acc = c.compare(out)
        if rel > 2.0**-22:  # (past the rounding of u itself)
            assert acc.tolist() == [0, 1, 0, 1]
    finally:
        B.pld_destroy(ctx)


def test_drafter_equal_to_target_is_always_accepted_and_zero_excess_draws_from_p():
    import torch
    c = Case(8, 3, 256, seed=14, head=2)
    # q at least p everywhere: nothing exceeds it, so a refusal (forced by a
    # q of twice p and u near 1) draws from p itself
    e = np.exp(c.z[:, :2] - c.z[:, :2].max(-1, keepdims=True))
    c.probs = (2.0 * e / e.sum(-1, keepdims=True)).astype(np.float32)
    c.uniform[:, :2] = 0.9
    ctx = context(8, 3, 256)
    try:
        out = c.outputs()
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert (c.compare(out) == 0).all()
        c.probs = (0.5 * c.probs * (1 - 1e-6)).astype(np.float32)
        c.uniform[:, :2] = 1.0 - 2.0**-24
        out = c.outputs()
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert (out[1] == 2).all()
    finally:
        B.pld_destroy(ctx)


def test_defaults_without_temperature_and_logprobs():
    c = Case(5, 4, 1000, seed=15)
    ctx = context(5, 4, 1000)
    try:
        out = c.outputs()
        a = list(c.args())
        a[8] = None
        B.pld_verify(ctx, *a, *out[:3])
        assert B.pld_sync(ctx) == B.PLD_OK
        tok, acc, cnt, _ = c.reference()
        assert np.array_equal(out[0].cpu().numpy(), tok)
        assert bool((out[3] == 7).all())
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("what", ["dlen high", "dlen low", "token high", "token low", "temp nan",
                                  "temp negative", "temp inf", "temp subnormal", "u one", "u nan", "draw one",
                                  "nan", "inf", "all masked"])
def test_bad_inputs_commit_nothing_and_spare_the_others(what):
    c = Case(3, 4, 5000, seed=16, accept=0.999)
    c.uniform[:] = np.minimum(c.uniform, 0.9)
    good = Case(3, 4, 5000, seed=16, accept=0.999)
    good.uniform[:] = c.uniform
    if what == "dlen high":
        c.dlen = np.array([3, 4, 3])
    elif what == "dlen low":
        c.dlen = np.array([3, -2, 3])
    elif what.startswith("token"):
        c.draft[1, 2] = 5000 if what.endswith("high") else -1
    elif what.startswith("temp"):
        c.temp[1] = {"nan": np.nan, "negative": -1.0, "inf": np.inf,
                     "subnormal": 1e-39}[what.split()[1]]
    elif what == "draw one":
        c.uniform[1, -1] = 1.0
    elif what.startswith("u "):
        c.uniform[1, 1] = {"one": 1.0, "nan": np.nan}[what.split()[1]]
    elif what == "all masked":
        c.logits[1, 2, :5000] = -float("inf")
    else:
        c.logits[1, 2, 4321] = float(what)
    ctx = context(3, 4, 5000)
    try:
        out, ref = c.outputs(), good.outputs()
        B.pld_verify(ctx, *good.args(), *ref)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert int(ref[1][1]) == 3, "the bad row has to be needed"
        B.pld_verify(ctx, *c.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_EINVAL
        for i in (0, 2):
            for x, y in zip(out, ref):
                assert bool((x[i] == y[i]).all())
        assert bool((out[0][1] == -1).all()) and bool((out[3][1] == 0).all())
        assert int(out[1][1]) == 0 and int(out[2][1]) == 0
        # the context serves a clean call right after
        out = c.outputs()
        B.pld_verify(ctx, *good.args(), *out)
        assert B.pld_sync(ctx) == B.PLD_OK
        good.compare(out)
    finally:
        B.pld_destroy(ctx)


def test_rows_after_a_refusal_are_not_checked():
    c = Case(4, 5, 2000, seed=17)
    c.uniform[:, 1] = 1.0 - 2.0**-24      # refused at position 1 at the latest
    c.logits[:, 3:, 55] = float("nan")
    ctx = context(4, 5, 2000)
    try:
        for _ in range(10):
            out = c.outputs()
            B.pld_verify(ctx, *c.args(), *out)
            assert B.pld_sync(ctx) == B.PLD_OK
            assert (c.compare(out) <= 1).all()
    finally:
        B.pld_destroy(ctx)


def test_back_to_back_calls_of_different_sizes_and_graph_replays():
    import torch
    cases = [Case(7, 9, 40000, dt="bf16", seed=20, accept=0.9),
             Case(2, 3, 17, seed=21), Case(7, 1, 40000, seed=22),
             Case(5, 6, 9999, head=5, src=True, temperature=0.8, seed=23)]
    ctxs = {v: context(7, 9, v) for v in {c.vocab for c in cases}}
    try:
        outs = []
        for _ in range(3):
            for c in cases:
                outs.append((c, c.outputs()))
                a = c.args()
                B.pld_verify(ctxs[c.vocab], *a, *outs[-1][1])
                outs[-1] += (a,)
        for v in ctxs:
            assert B.pld_sync(ctxs[v]) == B.PLD_OK
        for c, out, _ in outs:
            c.compare(out)
        for c in (cases[0], cases[3]):
            a, out = c.args(), c.outputs()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                B.pld_verify(ctxs[c.vocab], *a, *out)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                B.pld_verify(ctxs[c.vocab], *a, *out)
            for i in range(4):
                c.uniform = np.roll(c.uniform, 1, 0)
                a[9].copy_(torch.from_numpy(c.uniform))
                for x in out:
                    x.fill_(-9)
                graph.replay()
                torch.cuda.synchronize()
                c.compare(out)
                # the program's own work between the replays
                eager = c.outputs()
                B.pld_verify(ctxs[c.vocab], *a, *eager)
                assert B.pld_sync(ctxs[c.vocab]) == B.PLD_OK
                assert all(torch.equal(x, y) for x, y in zip(out, eager))
    finally:
        for v in ctxs:
            B.pld_destroy(ctxs[v])


def test_refusals_on_a_context():
    import torch
    c = Case(2, 3, 50, seed=24)
    a = c.args()
    names = ("logits", "logits_stride", "rows", "draft", "draft_len", "src", "draft_probs",
             "head", "temperature", "uniform", "batch")
    out = c.outputs()
    good = dict(zip(names, a), out_tokens=out[0], out_accepted=out[1], out_counts=out[2],
                out_logprobs=out[3])
    ctx = context(2, 3, 50)
    try:
        B.pld_verify(ctx, **{**good, "batch": 0})
        for field, value in [("rows", 0), ("rows", 4), ("batch", 3), ("batch", -1),
                             ("logits_stride", 49), ("head", 1), ("head", -1), ("head", 3),
                             ("draft", None), ("draft_len", None), ("uniform", None),
                             ("out_tokens", None), ("out_accepted", None), ("out_counts", None),
                             ("uniform", a[9].data_ptr() + 2), ("src", a[4].data_ptr() + 4)]:
            with pytest.raises(B.PldError) as e:
                B.pld_verify(ctx, **{**good, field: value})
            assert e.value.status == B.PLD_EINVAL, field
        with pytest.raises(ValueError):
            B.pld_verify(ctx, **{**good, "logits": c.logits.double()})
        assert bool((out[0] == -7).all())
        assert B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)
