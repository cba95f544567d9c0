"""pld_attend_tree (HIP, gfx950) against the 64-bit reference: shapes of trees,
types, head layouts, lengths around tile and page edges, windows, cells that
must not be used, long caches, bad inputs, graphs and streams.

Tolerances are those of tests/test_attend_gpu.py: a tree changes which cells a
row sees, not how they are weighed and summed."""

from __future__ import annotations

import numpy as np
import pytest

import target_reference as R
import test_attend_gpu as A
import tree_reference as TR
from prompt_lookup_gram_amd import binding as B
from test_attend_gpu import gpu  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")]


class Case(A.Case):
    """A call's inputs, with trees; `kind` names their shape (random ones
    without)."""

    def __init__(self, lengths, dlen, rows, kind=None, **kw):
        super().__init__(lengths, dlen, rows, **kw)
        rng = np.random.default_rng([9701, kw.get("seed", 0)])
        self.parent = [TR.shapes(rows - 1)[kind] if kind else TR.random_tree(rng, rows - 1)
                       for _ in lengths]

    def call(self, ctx, out, lse, window=0, scale=0.0, max_len=0, table=None, stream=None,
             parent=None):
        import torch
        self.ln = torch.tensor(self.lengths, dtype=torch.int32).cuda()
        self.dl = torch.tensor(self.dlen, dtype=torch.int32).cuda()
        self.tab = torch.from_numpy(self.table if table is None else table).cuda()
        self.par = torch.tensor(self.parent if parent is None else parent,
                                dtype=torch.int32).cuda().view(self.b, self.rows - 1)
        self.again(ctx, out, lse, window, scale, max_len, stream)

    def again(self, ctx, out, lse, window=0, scale=0.0, max_len=0, stream=None):
        B.pld_attend_tree(ctx, self.q, self.width, self.rows, self.ln, self.dl, self.par, max_len,
                          self.b, self.tab, self.tab.shape[1], self.kc, self.vc, self.pages,
                          self.ks, self.vs, scale, window, out, lse, stream)

    def reference(self, window=0, scale=0.0):
        q = self.q.double().cpu().numpy()[:, :self.hq * self.dim]
        q = q.reshape(self.b, self.rows, self.hq, self.dim)
        ks = None if self.ks is None else self.ks.double().cpu().numpy()
        vs = None if self.vs is None else self.vs.double().cpu().numpy()
        return TR.attend(q, self.kc64, self.vc64, self.table, self.lengths, self.dlen,
                         self.parent, self.page, scale or self.dim ** -0.5, window, ks, vs)


def check(lengths, dlen, rows, kind=None, window=0, scale=0.0, max_len=0, **kw):
    c = Case(lengths, dlen, rows, kind, **kw)
    ctx = c.context(max(max_len, c.max_len))
    try:
        out, lse = c.outputs()
        c.call(ctx, out, lse, window, scale, max_len)
        assert B.pld_sync(ctx) == B.PLD_OK, B.pld_last_error()
        c.compare(out, lse, window, scale)
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("dt,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("rows", [5, 13])
def test_types_and_head_dims(dt, cache, dim, rows):
    # 10 and 26 query rows a kv head
    check([1, 77, 130], [rows - 1, rows - 1, min(2, rows - 1)], rows, dim=dim, dt=dt, cache=cache,
          seed=dim + rows)


@pytest.mark.parametrize("dt,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("rows", [10, 20, 40])
def test_types_and_head_dims_with_more_query_rows(dt, cache, dim, rows):
    # 40, 80 and 160 query rows a kv head, spans joined (700 positions)
    check([1, 77, 700, 0], [rows - 1, 3, rows - 2, 5], rows, hq=8, hk=2, dim=dim, dt=dt,
          cache=cache, page=32, window=0 if dim != 128 else 90, seed=dim + rows)


@pytest.mark.parametrize("kind", ["chain", "star", "comb", "binary"])
@pytest.mark.parametrize("rows,hq,hk", [(8, 2, 2), (33, 4, 2), (100, 2, 1), (256, 2, 2)])
@pytest.mark.parametrize("window", [0, 3, 20])
def test_tree_shapes(kind, rows, hq, hk, window):
    check([50, 1], [rows - 1, rows - 1], rows, kind, hq=hq, hk=hk, window=window, seed=rows)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (8, 2), (16, 1), (7, 1), (40, 1)])
@pytest.mark.parametrize("rows", [2, 9, 31])
def test_head_groups(hq, hk, rows):
    check([95, 33], [rows - 1, rows // 2], rows, hq=hq, hk=hk, seed=hq * 16 + rows)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255,
                               256, 257, 513])
@pytest.mark.parametrize("page,cache", [(16, "bf16"), (64, "bf16"), (16, "e4m3")])
def test_lengths_around_tiles_and_pages(n, page, cache):
    check([n, 1, n], [0, 6, 6], 7, page=page, cache=cache, seed=n)


@pytest.mark.parametrize("window", [1, 2, 5, 15, 16, 17, 64, 100, 299, 300, 301, 5000])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq", [2, 12])
def test_windows(window, cache, hq):
    check([300, 1, 90], [11, 11, 0], 12, window=window, cache=cache, hq=hq, hk=2, seed=window)


@pytest.mark.parametrize("rows,dt,cache", [(3, "bf16", "bf16"), (16, "f16", "f16"),
                                           (64, "bf16", "bf16"), (24, "bf16", "e4m3")])
def test_long_contexts_are_split_and_joined(rows, dt, cache):
    check([20001, 8192, 12345], [rows - 1] * 3, rows, hq=8, hk=1, dim=128, page=64, dt=dt,
          cache=cache, seed=rows, peak=3.0)


def test_idle_requests_strides_scales_and_a_loose_bound():
    check([0, 50, 0, 20], [2, -1, -1, 1], 3)
    check([100, 40], [3, 1], 4, pad=24, seed=4)
    check([100, 40], [3, 1], 4, max_len=103, seed=5)
    check([500, 33], [3, 0], 4, dim=128, peak=8.0, seed=1)
    check([500, 33], [3, 0], 4, dim=128, scale=-0.3, seed=3)
    # 128 query rows a kv head, and of them 64 or fewer
    for cache in ("bf16", "e4m3"):
        check([500, 333, 70], [15, 7, 0], 16, dim=128, hq=16, hk=2, cache=cache, peak=8.0, seed=6)
        check([500, 333, 70], [15, 7, 0], 16, dim=64, hq=16, hk=2, cache=cache, scale=-0.3, pad=8,
              seed=7)
        check([900, 333, 70], [15, 7, 0], 16, dim=128, hq=16, hk=2, cache=cache, max_len=70000,
              page=128, seed=8)


def test_chains_and_single_rows_are_the_chain_calls():
    import torch
    for rows, window in ((1, 0), (9, 0), (40, 25)):
        c = Case([300, 20], [rows - 1, 0], rows, "chain", hq=4, hk=2, seed=rows)
        ctx = c.context()
        try:
            want = c.outputs()
            A.Case.call(c, ctx, *want, window)
            for parent in ([None] if rows == 1 else [None, c.parent]):
                out, lse = c.outputs()
                c.par = None if parent is None else torch.tensor(parent, dtype=torch.int32).cuda()
                c.again(ctx, out, lse, window)
                assert B.pld_sync(ctx) == B.PLD_OK
                if parent is None:
                    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
                else:
                    c.compare(out, lse, window)
        finally:
            B.pld_destroy(ctx)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 1)])
def test_rows_do_not_see_what_is_not_finite_off_their_branch(cache, value, hq, hk):
    """A node whose k and v overflowed touches the rows below it only; a
    position that a window leaves behind touches no row after that."""
    import torch
    rows, window = 20, 40
    c = Case([90, 61, 300], [rows - 1, 9, rows - 1], rows, hq=hq, hk=hk, dim=64, cache=cache,
             seed=14)
    ctx = c.context()
    try:
        clean = c.outputs()
        c.call(ctx, *clean, window)
        assert B.pld_sync(ctx) == B.PLD_OK
        hit = [89 + 5, 61, 300 - window]
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
                up = TR.branch(c.parent[i], t)
                root = c.lengths[i] - 1
                if hit[i] > root:
                    sees = hit[i] - root in up
                else:
                    sees = hit[i] > root + len(up) - 1 - window
                if sees:
                    assert bool(out[i, t].isnan().all()), (i, t)
                else:
                    assert torch.equal(out[i, t], clean[0][i, t]), (i, t)
                    assert torch.equal(lse[i, t], clean[1][i, t]), (i, t)
    finally:
        B.pld_destroy(ctx)


def test_bad_inputs_are_nan_and_reported_and_spare_the_others():
    import torch
    lengths, dlen, rows = [50, 50, 50], [12, 11, 12], 13
    for hq in (2, 12):
        for what, want in (("length", B.PLD_EINVAL), ("dlen", B.PLD_EINVAL),
                           ("long", B.PLD_ECAPACITY), ("page", B.PLD_EINVAL),
                           ("parent itself", B.PLD_EINVAL), ("parent -1", B.PLD_EINVAL),
                           ("parent far", B.PLD_EINVAL)):
            c = Case(lengths, dlen, rows, hq=hq, hk=2, seed=10)
            ctx = c.context()
            try:
                good = c.outputs()
                c.call(ctx, *good)
                assert B.pld_sync(ctx) == B.PLD_OK
                table, parent = c.table.copy(), np.array(c.parent)
                if what == "length":
                    c.lengths = [50, -1, 50]
                elif what == "dlen":
                    c.dlen = [12, 13, 12]
                elif what == "long":
                    c.lengths = [50, 60, 50]
                elif what == "page":
                    table[1, 1] = c.pages
                else:
                    parent[1, 6] = {"itself": 7, "-1": -1, "far": 1 << 30}[what.split()[1]]
                parent[1, 11:] = 77  # past d: not read
                out, lse = c.outputs()
                c.call(ctx, out, lse, table=table, parent=parent)
                assert B.pld_sync(ctx) == want, what
                for i in (0, 2):
                    assert torch.equal(out[i], good[0][i]) and torch.equal(lse[i], good[1][i])
                n = 12 if "page" in what or "parent" in what else rows
                assert bool(out[1, 1:n].isnan().all()) and bool(lse[1, 1:n].isnan().all()), what
                assert B.pld_sync(ctx) == B.PLD_OK
            finally:
                B.pld_destroy(ctx)


def test_a_page_that_the_window_left_behind_is_not_needed():
    c = Case([50], [3], 4, "star", seed=11)
    ctx = c.context()
    try:
        table = c.table.copy()
        table[0, 0] = -1
        out, lse = c.outputs()
        c.call(ctx, out, lse, window=34, table=table)  # the root sees from 16 on
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(out, lse, window=34)
        c.call(ctx, out, lse, window=35, table=table)
        assert B.pld_sync(ctx) == B.PLD_EINVAL
    finally:
        B.pld_destroy(ctx)


def test_repeated_calls_are_bit_identical_and_graphs_replay():
    import torch
    c = Case([9000, 700, 4097], [31, 3, 0], 32, hq=8, hk=2, dim=128, page=64, seed=12)
    ctx = c.context()
    try:
        first = c.outputs()
        c.call(ctx, *first)
        assert B.pld_sync(ctx) == B.PLD_OK
        for _ in range(3):
            again = c.outputs()
            c.again(ctx, *again)
            assert B.pld_sync(ctx) == B.PLD_OK
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        out, lse = c.outputs()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.again(ctx, out, lse)
        rng = np.random.default_rng(9702)
        for i in range(4):
            out.fill_(7.0)
            lse.fill_(7.0)
            # the lengths and the trees that a graph replays on are those on the device
            c.ln.copy_(torch.tensor([n - 100 * i for n in c.lengths], dtype=torch.int32))
            c.par.copy_(torch.tensor([TR.random_tree(rng, 31) for _ in range(3)],
                                     dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            want = c.outputs()
            c.again(ctx, *want)
            assert B.pld_sync(ctx) == B.PLD_OK
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("rows", [3, 7, 12, 40])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("longest", [60, 3000])
def test_out_in_qs_place(rows, cache, longest):
    # 12, 28, 48 and 160 query rows a kv head, one span and several
    import torch
    c = Case([longest, 40, 0], [rows - 1, 2, 1], rows, hq=8, hk=2, dim=128, cache=cache, page=32,
             seed=rows)
    ctx = c.context()
    try:
        want, lse = c.outputs()
        c.call(ctx, want, lse)
        assert B.pld_sync(ctx) == B.PLD_OK
        c.compare(want, lse)
        q = c.q.clone()
        _, again = c.outputs()
        c.again(ctx, c.q, again)
        assert B.pld_sync(ctx) == B.PLD_OK
        assert torch.equal(lse, again)
        live = (lse[:, :, :1] != 7.0).unsqueeze(-1)
        # (padded rows keep q's values)
        assert torch.equal(c.q.view_as(want), torch.where(live, want, q.view_as(want)))
    finally:
        B.pld_destroy(ctx)


def test_two_contexts_on_two_streams_at_once():
    import torch
    cases = [Case([6000, 300], [15, 3], 16, hq=8, hk=2, dim=128, page=64, seed=15),
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
                    c.again(ctx, *got[i][-1])
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
    ctx = B.pld_create_target(_wide_params(c))
    out, lse = c.outputs()
    ln = torch.tensor(c.lengths, dtype=torch.int32).cuda()
    tab = torch.from_numpy(c.table).cuda()
    par = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    good = dict(q=c.q, q_stride=c.width, rows=3, lengths=ln, draft_len=ln, parent=par, max_len=0,
                batch=2, page_table=tab, table_stride=tab.shape[1], k_cache=c.kc, v_cache=c.vc,
                n_pages=c.pages, out=out, out_lse=lse)
    try:
        B.pld_attend_tree(ctx, **{**good, "batch": 0})
        for field, value in [("rows", 0), ("rows", 257), ("rows", 301), ("batch", 3),
                             ("q_stride", c.width - 8), ("parent", par.data_ptr() + 2),
                             ("max_len", -1), ("table_stride", 0), ("n_pages", -1), ("q", None),
                             ("out", None), ("scale", float("nan")), ("window", -1)]:
            with pytest.raises(B.PldError) as e:
                B.pld_attend_tree(ctx, **{**good, field: value})
            assert e.value.status == B.PLD_EINVAL, field
        with pytest.raises(ValueError):
            B.pld_attend_tree(ctx, **{**good, "parent": par.long()})
        assert bool((out == 7).all())
        assert B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)


def _wide_params(c):
    p = B.pld_target_params_default()
    p.max_batch, p.max_rows, p.max_len = 2, 300, 400
    p.q_heads, p.kv_heads, p.head_dim, p.page_tokens = c.hq, c.hk, c.dim, c.page
    return p
