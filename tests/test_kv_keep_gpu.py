"""pld_kv_keep (HIP, gfx950): every kept cell equal to the one it came from,
every other cell untouched, in each layer; paths that move onto their own
sources; bad paths and pages; graphs. Cells are bytes moved: all comparisons are
exact."""

from __future__ import annotations

import numpy as np
import pytest

import tree_reference as TR
from prompt_lookup_gram_amd import binding as B
from test_kv_append_gpu import context, dtype, gpu, table_for  # noqa: F401

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lengths, paths, rows, hk=2, dim=64, cache="bf16", page=16, layers=2, gap=0,
                 seed=0, dlen=None):
        import torch
        rng = np.random.default_rng([9811, seed])
        self.lengths, self.paths, self.rows, self.layers = lengths, paths, rows, layers
        self.accepted = [max(0, len(p) - 1) for p in paths]
        self.b, self.hk, self.dim, self.page, self.cache = len(lengths), hk, dim, page, cache
        self.dlen = dlen or [rows - 1] * self.b
        self.table, self.pages = table_for(rng, lengths, self.dlen, page)
        cells = self.pages * hk * page * dim
        self.stride = cells + gap
        kind = torch.uint8 if cache == "e4m3" else torch.int16
        lo, hi = (0, 255) if cache == "e4m3" else (-32768, 32767)
        self.raw = [torch.from_numpy(rng.integers(lo, hi, layers * self.stride)).to(kind).cuda()
                    for _ in range(2)]
        i32 = dict(dtype=torch.int32, device="cuda")
        path = np.full((self.b, rows), -1, np.int32)
        for i, p in enumerate(paths):
            path[i, :len(p)] = p
        self.ln, self.dl = torch.tensor(lengths, **i32), torch.tensor(self.dlen, **i32)
        self.path, self.acc = torch.from_numpy(path).cuda(), torch.tensor(self.accepted, **i32)
        self.tab = torch.from_numpy(self.table).cuda()

    def context(self):
        return context(self.b, self.rows, 1 << 20, self.hk, self.hk, self.dim,
                       "bf16" if self.cache == "e4m3" else self.cache, self.cache, self.page)

    def call(self, ctx, stream=None):
        k, v = [x.view(dtype(self.cache)) for x in self.raw]
        B.pld_kv_keep(ctx, self.ln, self.dl, self.path, self.acc, self.rows, self.b, self.tab,
                      self.tab.shape[1], k, v, self.pages, self.layers, self.stride, self.stride,
                      stream)

    def shaped(self, x, *shape):
        n = self.pages * self.hk * self.page * self.dim
        return x.cpu().numpy().reshape(self.layers, -1)[:, :n].reshape(
            self.layers, self.pages, self.hk, *shape)

    def check(self, before, moved=None):
        wk, wv = TR.keep(self.shaped(before[0], self.page, self.dim),
                         self.shaped(before[1], self.dim, self.page), self.table, self.lengths,
                         self.paths, self.accepted if moved is None else moved, self.page)
        assert np.array_equal(self.shaped(self.raw[0], self.page, self.dim), wk)
        assert np.array_equal(self.shaped(self.raw[1], self.dim, self.page), wv)
        n = self.pages * self.hk * self.page * self.dim
        for x, y in zip(self.raw, before):
            x, y = x.view(self.layers, -1)[:, n:], y.view(self.layers, -1)[:, n:]
            assert bool((x == y).all())


def check(lengths, paths, rows, **kw):
    c = Case(lengths, paths, rows, **kw)
    ctx = c.context()
    try:
        before = [x.clone() for x in c.raw]
        c.call(ctx)
        assert B.pld_sync(ctx) == B.PLD_OK, B.pld_last_error()
        c.check(before)
    finally:
        B.pld_destroy(ctx)


def some_path(rng, d, n):
    return [0] + sorted(rng.choice(np.arange(1, d + 1), n, replace=False).tolist())


@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_types_dims_and_pages(cache, dim, page):
    rng = np.random.default_rng([9812, dim, page])
    paths = [some_path(rng, 69, n) for n in (0, 1, 2, 5, 8, 9, 30, 69)]
    check([int(x) for x in rng.integers(1, 400, 8)], paths, 70, dim=dim, page=page, cache=cache,
          gap=64)


@pytest.mark.parametrize("hk,layers", [(1, 1), (3, 1), (8, 5), (1, 40), (5, 7)])
def test_heads_and_layers(hk, layers):
    rng = np.random.default_rng([9813, hk])
    check([100, 33, 8], [some_path(rng, 15, n) for n in (3, 7, 15)], 16, hk=hk, layers=layers)


@pytest.mark.parametrize("rows", [2, 17, 100, 256])
def test_moves_onto_each_others_sources(rows):
    d = rows - 1
    for path in (list(range(0, 1)) + list(range(2, rows)), list(range(rows)),
                 [0] + list(range(1, rows, 2)), [0] + list(range(rows // 2, rows))):
        check([17, 1], [path, [0, d]], rows)


def test_requests_without_rows_or_moves():
    c = Case([30, 0, 9, 20], [[-1], [0, 2], [0, 2], [0]], 8, dlen=[7, 7, -1, 7])
    ctx = c.context()
    try:
        before = [x.clone() for x in c.raw]
        c.acc[0] = 0
        c.call(ctx)
        assert B.pld_sync(ctx) == B.PLD_OK
        c.check(before, [0, 0, 0, 0])
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("path,accepted", [([0, 5, 5], 2), ([1, 2, 5], 2), ([0, 2, 8], 2),
                                           ([0, -3, 5], 2), ([0, 2, 5], 8), ([0, 2, 5], -1),
                                           ([0, 2], 2), ([0, 1 << 30, 5], 2)])
def test_bad_paths_move_nothing_and_spare_the_others(path, accepted):
    c = Case([20, 20], [path, [0, 2, 5]], 8)
    ctx = c.context()
    try:
        before = [x.clone() for x in c.raw]
        c.acc[0] = accepted
        c.call(ctx)
        assert B.pld_sync(ctx) == B.PLD_EINVAL
        c.check(before, [0, 2])
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("what,status", [("page", B.PLD_EINVAL), ("length", B.PLD_EINVAL),
                                         ("dlen", B.PLD_EINVAL)])
def test_bad_blocks_and_pages(what, status):
    c = Case([14, 20], [[0, 2, 5], [0, 2, 5]], 8)
    ctx = c.context()
    try:
        before = [x.clone() for x in c.raw]
        if what == "page":
            c.tab[0, 1] = c.pages
        elif what == "length":
            c.ln[0] = -3
        else:
            c.dl[0] = 8
        c.call(ctx)
        assert B.pld_sync(ctx) == status
        c.check(before, [0, 2])
    finally:
        B.pld_destroy(ctx)


def test_graph_replays():
    import torch
    c = Case([100, 33, 8], [[0, 2, 5, 6], [0, 1, 9], [0, 4]], 16, layers=3)
    ctx = c.context()
    try:
        before = [x.clone() for x in c.raw]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            c.call(ctx)
        for _ in range(3):
            for x, y in zip(c.raw, before):
                x.copy_(y)
            graph.replay()
            torch.cuda.synchronize()
            c.check(before)
        assert B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)


def test_offsets_past_32_bits():
    """Layers and pages whose element offsets pass 2^31."""
    import torch
    pages, hk, page, dim = 20000, 8, 64, 128
    k = torch.zeros((2, pages, hk, page, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((2, pages, hk, dim, page), dtype=torch.bfloat16, device="cuda")
    tab = torch.tensor([[19999, 18000]], dtype=torch.int32, device="cuda")
    k[1, 18000, :, 5] = 3.0
    v[1, 18000, :, :, 5] = 4.0
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx = context(1, 16, 1000, hk, hk, dim, "bf16", "bf16", page)
    try:
        # cell 69 (page 18000, slot 5) is node 7 of a root in cell 62; it goes to 63
        B.pld_kv_keep(ctx, torch.tensor([63], **i32), torch.tensor([15], **i32),
                      torch.tensor([[0, 7] + [-1] * 14], **i32), torch.tensor([1], **i32), 16, 1,
                      tab, 2, k, v, pages, 2, k.stride(0), v.stride(0))
        assert B.pld_sync(ctx) == B.PLD_OK
        assert bool((k[1, 19999, :, 63] == 3).all()) and bool((v[1, 19999, :, :, 63] == 4).all())
        assert int((k != 0).sum()) == int((v != 0).sum()) == 2 * hk * dim
    finally:
        B.pld_destroy(ctx)


def test_refusals_on_a_context():
    c = Case([100, 33], [[0, 2, 5, 6], [0, 1, 9]], 16)
    ctx = context(2, 300, 1000, 2, 2, 64, "bf16", "bf16", 16)
    before = [x.clone() for x in c.raw]
    k, v = [x.view(dtype("bf16")) for x in c.raw]
    good = dict(lengths=c.ln, draft_len=c.dl, path=c.path, accepted=c.acc, rows=16, batch=2,
                page_table=c.tab, table_stride=c.tab.shape[1], k_cache=k, v_cache=v,
                n_pages=c.pages, layers=2, k_layer_stride=c.stride, v_layer_stride=c.stride)
    try:
        B.pld_kv_keep(ctx, **{**good, "batch": 0})
        B.pld_kv_keep(ctx, **{**good, "layers": 0})
        for field, value in [("rows", 0), ("rows", 257), ("rows", 301), ("batch", 3),
                             ("layers", -1), ("k_layer_stride", c.stride - 8),
                             ("v_layer_stride", c.stride + 4), ("path", None), ("accepted", None),
                             ("lengths", None), ("n_pages", 0), ("path", c.path.data_ptr() + 2),
                             ("k_cache", k.data_ptr() + 2), ("table_stride", 0)]:
            with pytest.raises(B.PldError) as e:
                B.pld_kv_keep(ctx, **{**good, field: value})
            assert e.value.status == B.PLD_EINVAL, field
        with pytest.raises(ValueError):
            B.pld_kv_keep(ctx, **{**good, "k_cache": k.half()})
        assert B.pld_sync(ctx) == B.PLD_OK
        for x, y in zip(c.raw, before):
            assert bool((x == y).all())
    finally:
        B.pld_destroy(ctx)
