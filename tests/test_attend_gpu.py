"""pld_attend (HIP, gfx950) against the 64-bit reference: head layouts, types,
block sizes, lengths around tile and page edges, windows, cells that must not
be used, long caches, and bad inputs.

Tolerances. A score is a sum of head_dim products (exact in 32 bits for
16-bit factors) times the scale: off by at most (head_dim + 4) * 2^-24 of
S = the largest sum of |q k| * scale in the row. So each probability is off
by 2 ds relative, ds = that plus 2^-21 for exp and the statistics' rescaling
(at most one rounding for each of a few hundred tiles in a row, each 2^-24,
when they all move one way: 2^-15 covers 512). A probability is rounded to
dtype before it meets V, half a step; the output is rounded once. Hence
|out - ref| <= (h + 2 ds + 2^-15) * sum p|v| + h * (|ref| + that), h = eps / 2,
and |lse - ref| <= ds + 2^-15 + 2^-23 |ref|."""

from __future__ import annotations

import numpy as np
import pytest

import target_reference as R
from prompt_lookup_gram_amd import binding as B
from test_kv_append_gpu import context, dtype, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.load()
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


class Case:
    """Inputs of one call, on the GPU and in 64 bits."""

    def __init__(self, lengths, dlen, rows, hq=4, hk=2, dim=64, dt="bf16", cache=None, page=16,
                 seed=0, pad=0, peak=1.0, poison=True):
        import torch
        self.lengths, self.dlen, self.rows = lengths, dlen, rows
        self.hq, self.hk, self.dim, self.dt, self.page = hq, hk, dim, dt, page
        self.cache = cache or dt
        rng = np.random.default_rng([9201, seed])
        b = self.b = len(lengths)
        self.table, self.pages = table_for(rng, lengths, dlen, page)
        width = self.width = hq * dim + pad
        q = torch.from_numpy(rng.standard_normal((b * rows, width)) * peak).to(dtype(dt))
        self.q = q.cuda()
        kc = torch.from_numpy(rng.standard_normal((self.pages, hk, page, dim))).float()
        vc = torch.from_numpy(rng.standard_normal((self.pages, hk, dim, page))).float()
        kc, vc = kc.to(dtype(self.cache)), vc.to(dtype(self.cache))
        self.kc64, self.vc64 = kc.double().numpy(), vc.double().numpy()
        if poison:
            # every cell that no row sees: NaN (both types of cache have it)
            seen = np.zeros((self.pages, page), bool)
            for i in range(b):
                for p in range(lengths[i] - 1 + R.block_rows(lengths[i], dlen[i])):
                    seen[self.table[i, p // page], p % page] = True
            hide = torch.from_numpy(~seen)
            kc = kc.float().masked_fill(hide[:, None, :, None], float("nan")).to(kc.dtype)
            vc = vc.float().masked_fill(hide[:, None, None, :], float("nan")).to(vc.dtype)
        self.kc, self.vc = kc.cuda(), vc.cuda()
        self.ks = self.vs = None
        if self.cache == "e4m3":
            self.ks = torch.tensor(rng.uniform(0.2, 2.0, hk), dtype=torch.float32).cuda()
            self.vs = torch.tensor(rng.uniform(0.2, 2.0, hk), dtype=torch.float32).cuda()
        self.max_len = max([1] + [n + d for n, d in zip(lengths, dlen)])

    def context(self, max_len=None):
        return context(self.b, self.rows, max_len or self.max_len, self.hq, self.hk, self.dim,
                       self.dt, self.cache, self.page)

    def outputs(self):
        import torch
        return (torch.full((self.b, self.rows, self.hq, self.dim), 7.0, dtype=dtype(self.dt),
                           device="cuda"),
                torch.full((self.b, self.rows, self.hq), 7.0, device="cuda"))

    def call(self, ctx, out, lse, window=0, scale=0.0, max_len=0, table=None, stream=None):
        import torch
        self.ln = torch.tensor(self.lengths, dtype=torch.int32).cuda()
        self.dl = torch.tensor(self.dlen, dtype=torch.int32).cuda()
        self.tab = torch.from_numpy(self.table if table is None else table).cuda()
        B.pld_attend(ctx, self.q, self.width, self.rows, self.ln, self.dl, max_len, self.b,
                     self.tab, self.tab.shape[1], self.kc, self.vc, self.pages, self.ks, self.vs,
                     scale, window, out, lse, stream)

    def reference(self, window=0, scale=0.0):
        q = self.q.double().cpu().numpy()[:, :self.hq * self.dim]
        q = q.reshape(self.b, self.rows, self.hq, self.dim)
        ks = None if self.ks is None else self.ks.double().cpu().numpy()
        vs = None if self.vs is None else self.vs.double().cpu().numpy()
        return R.attend(q, self.kc64, self.vc64, self.table, self.lengths, self.dlen, self.page,
                        scale or self.dim ** -0.5, window, ks, vs)

    def compare(self, out, lse, window=0, scale=0.0):
        import torch
        want, wlse, mass, span = self.reference(window, scale)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        live = ~np.isnan(wlse)
        assert (out[~live] == 7.0).all() and (lse[~live] == 7.0).all(), "a padded row was written"
        h = float(torch.finfo(dtype(self.dt)).eps) / 2
        ds = (self.dim + 4) * 2.0**-24 * span + 2.0**-21
        lim = (h + 2 * ds[..., None] + 2.0**-15) * mass
        # (fp16 outputs below 2^-14 are rounded to steps of 2^-24)
        lim = lim + h * (np.abs(want) + lim) + 2.0**-25
        off = (np.abs(out - want) - lim)[live]
        assert not np.isnan(off).any(), "NaN"
        if off.size:
            assert off.max() <= 0, f"out off by {off.max()} more than allowed"
            offl = (np.abs(lse - wlse) - (ds + 2.0**-15 + 2.0**-23 * np.abs(wlse)))[live]
            assert offl.max() <= 0, f"lse off by {offl.max()} more than allowed"


def check(lengths, dlen, rows, window=0, scale=0.0, max_len=0, **kw):
    c = Case(lengths, dlen, rows, **kw)
    ctx = c.context()
    try:
        out, lse = c.outputs()
        c.call(ctx, out, lse, window, scale, max_len)
        assert B.pld_sync(ctx) == B.PLD_OK, B.pld_last_error()
        c.compare(out, lse, window, scale)
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("dt,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"),
                                      ("f16", "e4m3")])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("rows", [1, 5])
def test_types_and_head_dims(dt, cache, dim, rows):
    check([1, 77, 130], [0, rows - 1, min(2, rows - 1)], rows, dim=dim, dt=dt, cache=cache,
          seed=dim + rows)


@pytest.mark.parametrize("dt,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"),
                                      ("f16", "e4m3")])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("rows", [6, 10, 20, 40])
def test_types_and_head_dims_with_more_query_rows(dt, cache, dim, rows):
    # 24, 40, 80 and 160 query rows a kv head, spans joined (700 positions)
    check([1, 77, 700, 0], [rows - 1, 3, rows - 2, 5], rows, hq=8, hk=2, dim=dim, dt=dt,
          cache=cache, page=32, window=0 if dim != 128 else 90, seed=dim + rows)


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 2), (3, 1), (8, 2), (12, 2), (16, 1), (7, 1),
                                   (32, 2), (40, 1)])
@pytest.mark.parametrize("rows", [1, 2, 9])
def test_head_groups(hq, hk, rows):
    check([95, 33], [rows - 1, rows // 2], rows, hq=hq, hk=hk, seed=hq * 16 + rows)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129,
                               255, 256, 257, 511, 513])
@pytest.mark.parametrize("page", [16, 64])
def test_lengths_around_tiles_and_pages(n, page):
    check([n, 1, n], [0, 3, 3], 4, page=page, seed=n)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_page_sizes(page, cache):
    check([300, 257, 40, 5], [7, 0, 3, 1], 8, page=page, cache=cache, dim=128, seed=page)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 299, 300, 301, 5000])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_windows(window, cache):
    check([300, 1, 90], [7, 7, 0], 8, window=window, cache=cache, seed=window)


def test_idle_and_empty_requests_are_left():
    check([0, 50, 0, 20], [2, -1, -1, 1], 3)
    check([0, 50], [2, -1], 3)


@pytest.mark.parametrize("rows", [16, 17, 33, 64, 100])
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 1)])
def test_wide_blocks(rows, hq, hk):
    check([200, 1], [rows - 1, rows - 1], rows, hq=hq, hk=hk, seed=rows)


@pytest.mark.parametrize("batch", [1, 3])
@pytest.mark.parametrize("rows,dt,cache", [(1, "bf16", "bf16"), (16, "f16", "f16"),
                                           (8, "bf16", "e4m3")])
def test_long_contexts_are_split_and_joined(batch, rows, dt, cache):
    check([20001, 8192, 12345][:batch], [rows - 1] * batch, rows, hq=8, hk=1, dim=128, page=64,
          dt=dt, cache=cache, seed=batch, peak=3.0)


def test_peaked_scores_and_scale():
    # scores near +-60: one key carries the row, exp of the rest underflows
    check([500, 33], [3, 0], 4, dim=128, peak=8.0, seed=1)
    check([500, 33], [3, 0], 4, dim=128, scale=0.7, seed=2)
    check([500, 33], [3, 0], 4, dim=128, scale=-0.3, seed=3)


def test_strided_q_and_a_loose_bound():
    check([100, 40], [3, 1], 4, pad=24, seed=4)
    check([100, 40], [3, 1], 4, max_len=103, seed=5)


def test_infinite_and_nan_cells_in_sight():
    """Inside the rows' sight they count: a +inf score is NaN, NaN stays."""
    c = Case([40, 40, 40], [0, 0, 0], 1, hq=1, hk=1, seed=6, poison=False)
    c.q.abs_()
    for i, (buf, value) in enumerate(((c.kc, float("inf")), (c.kc, float("nan")),
                                      (c.vc, float("nan")))):
        page = int(c.table[i, 1])
        if buf is c.kc:
            buf[page, 0, 3, :] = value
        else:
            buf[page, 0, :, 3] = value
    ctx = c.context()
    try:
        out, lse = c.outputs()
        c.call(ctx, out, lse)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert bool(out.isnan().all())
        # ... and -inf scores weigh nothing
        c2 = Case([40], [0], 1, hq=1, hk=1, seed=7, poison=False)
        c2.q.abs_()
        page = int(c2.table[0, 1])
        c2.kc[page, 0, 3, :] = -float("inf")
        c2.vc[page, 0, :, 3] = 1000.0
        out, lse = c2.outputs()
        c2.call(ctx, out, lse)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert bool(out.isfinite().all()) and float(out.abs().max()) < 100
    finally:
        B.pld_destroy(ctx)


def test_a_context_whose_every_score_is_minus_infinity_is_nan():
    c = Case([600], [0], 1, hq=1, hk=1, seed=8, poison=False)
    c.q.abs_()
    c.kc.fill_(-float("inf"))
    ctx = c.context()
    try:
        out, lse = c.outputs()
        c.call(ctx, out, lse)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert bool(out.isnan().all())
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 1)])
def test_rows_do_not_see_what_is_not_finite_after_or_before_them(cache, value, hq, hk):
    """A draft position whose k and v overflowed touches the rows from it on
    only; a position that a window leaves behind touches none after that."""
    import torch
    rows = 12
    c = Case([90, 61, 300], [rows - 1, 7, rows - 1], rows, hq=hq, hk=hk, dim=64, cache=cache,
             seed=14)
    window = 40
    ctx = c.context()
    try:
        clean = c.outputs()
        c.call(ctx, *clean, window)
        assert B.pld_sync(ctx) == B.PLD_OK
        # request 0: position of row 5; 1: of row 0; 2: the window's first
        # position of row 3
        hit = [89 + 5, 60, 299 + 3 - window + 1]
        for i, p in enumerate(hit):
            page = int(c.table[i, p // c.page])
            x = torch.tensor(float(value)).to(c.vc.dtype)
            c.vc[page, :, :, p % c.page] = x
            c.kc[page, :, p % c.page, :] = x
        out, lse = c.outputs()
        c.call(ctx, out, lse, window)
        assert B.pld_sync(ctx) == B.PLD_OK
        for i in range(3):
            for t in range(R.block_rows(c.lengths[i], c.dlen[i])):
                p = c.lengths[i] - 1 + t
                if p - window < hit[i] <= p:
                    assert bool(out[i, t].isnan().all()), (i, t)
                else:
                    assert torch.equal(out[i, t], clean[0][i, t]), (i, t)
                    assert torch.equal(lse[i, t], clean[1][i, t]), (i, t)
        # an infinity in V alone, seen: it carries the row's dims
        if value == "inf" and cache == "bf16":
            c.kc.zero_()
            c.vc.zero_()
            page = int(c.table[0, 94 // c.page])
            c.vc[page, :, 3, 94 % c.page] = float("inf")
            c.call(ctx, out, lse, window)
            assert B.pld_sync(ctx) == B.PLD_OK
            assert bool((out[0, :5] == 0).all()) and bool((out[0, 5:, :, 3] == torch.inf).all())
            assert bool((out[0, 5:, :, 4:] == 0).all())
    finally:
        B.pld_destroy(ctx)


def test_cache_offsets_past_32_bits():
    import torch
    # 40,000 pages of 8 heads x 64 x 128: 2.6e9 elements a cache; the request
    # lives in pages whose element offsets pass 2^31
    pages, hk, page, dim = 40000, 8, 64, 128
    kc = torch.empty((pages, hk, page, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((pages, hk, dim, page), dtype=torch.bfloat16, device="cuda")
    c = Case([150], [2], 3, hq=16, hk=hk, dim=dim, page=page, seed=9)
    far = np.array([[39999, 33000, 32769]], np.int32)
    for i, p in enumerate(far[0]):
        kc[int(p)] = c.kc[int(c.table[0, i])]
        vc[int(p)] = c.vc[int(c.table[0, i])]
    ctx = c.context()
    try:
        out, lse = c.outputs()
        keep = c.kc, c.vc, c.pages
        c.kc, c.vc, c.pages = kc, vc, pages
        c.call(ctx, out, lse, table=far)
        assert B.pld_sync(ctx) == B.PLD_OK
        c.kc, c.vc, c.pages = keep
        c.compare(out, lse)
        # the writer reaches the same cells
        ln = torch.tensor([151], dtype=torch.int32).cuda()
        x = torch.full((1, 2 * hk * dim), 3.0, dtype=torch.bfloat16, device="cuda")
        B.pld_kv_append(ctx, None, 0, x, x, x.shape[1], 1, ln, ln * 0, 1,
                        torch.from_numpy(far).cuda(), 3, kc, vc, pages)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert bool((kc[32769, :, 150 % page] == 3).all())
        assert bool((vc[32769, :, :, 150 % page] == 3).all())
    finally:
        B.pld_destroy(ctx)


def test_bad_inputs_are_nan_and_reported_and_spare_the_others():
    import torch
    lengths, dlen, rows = [50, 50, 50], [2, 1, 2], 3
    for what, want in (("length", B.PLD_EINVAL), ("dlen", B.PLD_EINVAL), ("idle", B.PLD_EINVAL),
                       ("long", B.PLD_ECAPACITY), ("page", B.PLD_EINVAL),
                       ("negative page", B.PLD_EINVAL)):
        c = Case(lengths, dlen, rows, seed=10)
        ctx = c.context()
        try:
            good = c.outputs()
            c.call(ctx, *good)
            assert B.pld_sync(ctx) == B.PLD_OK
            table = c.table.copy()
            if what == "length":
                c.lengths = [50, -1, 50]
            elif what == "dlen":
                c.dlen = [2, 3, 2]
            elif what == "idle":
                c.dlen = [2, -2, 2]
            elif what == "long":
                c.lengths = [50, 52, 50]
            else:
                table[1, 1] = c.pages if what == "page" else -1
            out, lse = c.outputs()
            c.call(ctx, out, lse, table=table)
            assert B.pld_sync(ctx) == want, what
            for i in (0, 2):
                assert torch.equal(out[i], good[0][i]) and torch.equal(lse[i], good[1][i])
            n = 2 if "page" in what else rows
            assert bool(out[1, :n].isnan().all()) and bool(lse[1, :n].isnan().all()), what
            assert B.pld_sync(ctx) == B.PLD_OK
        finally:
            B.pld_destroy(ctx)


def test_a_table_that_is_too_short_is_a_bad_page():
    c = Case([50], [0], 1, seed=11)
    ctx = c.context()
    try:
        out, lse = c.outputs()
        c.call(ctx, out, lse, table=c.table[:, :3].copy())
        assert B.pld_sync(ctx) == B.PLD_EINVAL and "page" in B.pld_last_error()
        assert bool(out.isnan().all())
        # rows whose window leaves the missing page out do not see it
        table = c.table.copy()
        table[0, 0] = -1
        out, lse = c.outputs()
        c.call(ctx, out, lse, window=34, table=table)
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(out, lse, window=34)
    finally:
        B.pld_destroy(ctx)


def test_repeated_calls_are_bit_identical_and_graphs_replay():
    import torch
    c = Case([9000, 700, 4097], [7, 3, 0], 8, hq=8, hk=2, dim=128, page=64, seed=12)
    ctx = c.context()
    try:
        first = c.outputs()
        c.call(ctx, *first)
        assert B.pld_sync(ctx) == B.PLD_OK
        for _ in range(5):
            again = c.outputs()
            c.call(ctx, *again)
            assert B.pld_sync(ctx) == B.PLD_OK
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        out, lse = c.outputs()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            B.pld_attend(ctx, c.q, c.width, c.rows, c.ln, c.dl, 0, c.b, c.tab, c.tab.shape[1],
                         c.kc, c.vc, c.pages, None, None, 0.0, 0, out, lse)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            B.pld_attend(ctx, c.q, c.width, c.rows, c.ln, c.dl, 0, c.b, c.tab, c.tab.shape[1],
                         c.kc, c.vc, c.pages, None, None, 0.0, 0, out, lse)
        for i in range(4):
            out.fill_(7.0)
            lse.fill_(7.0)
            # the lengths a graph replays on are those on the device
            shorter = [n - 100 * i for n in c.lengths]
            c.ln.copy_(torch.tensor(shorter, dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            want = c.outputs()
            B.pld_attend(ctx, c.q, c.width, c.rows, c.ln, c.dl, 0, c.b, c.tab, c.tab.shape[1],
                         c.kc, c.vc, c.pages, None, None, 0.0, 0, *want)
            assert B.pld_sync(ctx) == B.PLD_OK
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    finally:
        B.pld_destroy(ctx)


def test_two_contexts_on_two_streams_at_once():
    """Each context's workspace is its own: calls overlapping on two streams
    give what they give one after the other; inputs are made on the stream
    that uses them."""
    import torch
    cases = [Case([6000, 300], [3, 3], 4, hq=8, hk=2, dim=128, page=64, seed=15),
             Case([9000, 5], [15, 0], 16, hq=8, hk=1, dim=64, page=16, seed=16)]
    ctxs = [c.context() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    try:
        want = []
        for c, ctx in zip(cases, ctxs):
            want.append(c.outputs())
            c.call(ctx, *want[-1])
            assert B.pld_sync(ctx) == B.PLD_OK
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(8):
            for i, (c, ctx, st) in enumerate(zip(cases, ctxs, streams)):
                with torch.cuda.stream(st):
                    got[i].append(c.outputs())
                    B.pld_attend(ctx, c.q, c.width, c.rows, c.ln, c.dl, 0, c.b, c.tab,
                                 c.tab.shape[1], c.kc, c.vc, c.pages, None, None, 0.0, 0,
                                 *got[i][-1])
        for i in range(2):
            assert B.pld_sync(ctxs[i], streams[i]) == B.PLD_OK
            for out in got[i]:
                assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])
    finally:
        for ctx in ctxs:
            B.pld_destroy(ctx)


def test_refusals_on_a_context():
    import torch
    c = Case([50, 20], [2, 1], 3, seed=13)
    ctx = c.context()
    out, lse = c.outputs()
    ln = torch.tensor(c.lengths, dtype=torch.int32).cuda()
    tab = torch.from_numpy(c.table).cuda()
    good = dict(q=c.q, q_stride=c.width, rows=3, lengths=ln, draft_len=ln, max_len=0, batch=2,
                page_table=tab, table_stride=tab.shape[1], k_cache=c.kc, v_cache=c.vc,
                n_pages=c.pages, out=out, out_lse=lse)
    try:
        B.pld_attend(ctx, **{**good, "batch": 0})
        for field, value in [("rows", 0), ("rows", 4), ("batch", 3), ("batch", -1),
                             ("q_stride", c.width - 8), ("q_stride", c.width + 4),
                             ("max_len", -1), ("max_len", c.max_len + 1), ("table_stride", 0),
                             ("n_pages", -1), ("q", None), ("out", None), ("lengths", None),
                             ("draft_len", None), ("page_table", None), ("k_cache", None),
                             ("v_cache", None), ("scale", float("nan")),
                             ("scale", float("inf")), ("window", -1),
                             ("q", c.q.data_ptr() + 2), ("out", out.data_ptr() + 8),
                             ("out_lse", lse.data_ptr() + 2)]:
            with pytest.raises(B.PldError) as e:
                B.pld_attend(ctx, **{**good, field: value})
            assert e.value.status == B.PLD_EINVAL, field
        with pytest.raises(ValueError):
            B.pld_attend(ctx, **{**good, "out": out.float()})
        assert bool((out == 7).all())
        assert B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)
