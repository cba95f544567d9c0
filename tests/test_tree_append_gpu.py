"""pld_kv_append_tree (HIP, gfx950) against the 64-bit reference: norms, rotary
layouts and scalings, trees, chains and prompts, strided inputs, 8-bit cells,
what must stay untouched, refusals, graphs and streams.

Tolerances are those of tests/test_kv_append_gpu.py, with the norm's: its sum of
squares is at most (head_dim + 6) additions and products of 2^-24 off, half of
which the root keeps, and the root, the quotient, the two products with it four
more roundings: below (head_dim / 2 + 8) * 2^-24 of a value."""

from __future__ import annotations

import numpy as np
import pytest

import target_reference as R
import tree_reference as TR
from prompt_lookup_gram_amd import binding as B
from test_kv_append_gpu import LARGEST, ROPE, context, dtype, gpu, stored, table_for  # noqa: F401

pytestmark = pytest.mark.gpu


def check(lengths, dlen, rows, tree=True, hq=4, hk=2, dim=64, dt="bf16", cache=None, page=16,
          rot=None, interleaved=False, scaling="plain", magnitude=1.0, seed=0, pad=0,
          scales=False, in_place=False, with_q=True, offset=0, norms="qk", eps=1e-6, kind=None,
          size=2.0):
    import torch
    cache, rot = cache or dt, dim if rot is None else rot
    rng = np.random.default_rng([9801, seed])
    b = len(lengths)
    parent = None
    if tree:
        parent = [TR.shapes(rows - 1)[kind] if kind else TR.random_tree(rng, rows - 1)
                  for _ in range(b)]
    table, pages = table_for(rng, lengths, dlen, page)
    wq, wk = hq * dim, hk * dim
    width = (0 if in_place else wq) + 2 * wk + pad
    raw = torch.from_numpy(rng.standard_normal(b * rows * width + offset) * size).to(dtype(dt))
    qkv = raw.cuda()[offset:].view(b * rows, width)
    if in_place:
        q = torch.from_numpy(rng.standard_normal((b * rows, wq)) * size).to(dtype(dt)).cuda()
        k, v = qkv[:, :wk], qkv[:, wk:2 * wk]
    else:
        q, k, v = qkv[:, :wq], qkv[:, wq:wq + wk], qkv[:, wq + wk:wq + 2 * wk]
    q0, k0, v0 = [x.double().cpu().numpy() for x in (q, k, v)]
    cells = torch.from_numpy(rng.standard_normal((2, pages * wk * page))).float()
    kc = cells[0].to(dtype(cache)).view(pages, hk, page, dim).cuda()
    vc = cells[1].to(dtype(cache)).view(pages, hk, dim, page).cuda()
    kc0, vc0 = kc.double().cpu().numpy(), vc.double().cpu().numpy()
    out_q = q if in_place else torch.full((b * rows, wq), 7.0, dtype=dtype(dt), device="cuda")
    oq0 = out_q.double().cpu().numpy()
    ks = torch.tensor(rng.uniform(0.01, 2.0, hk), dtype=torch.float32).cuda() if scales else None
    vs = torch.tensor(rng.uniform(0.01, 2.0, hk), dtype=torch.float32).cuda() if scales else None
    nq = rng.uniform(-1.5, 1.5, dim).astype(np.float32) if "q" in norms and with_q else None
    nk = rng.uniform(-1.5, 1.5, dim).astype(np.float32) if "k" in norms else None
    max_len = max(1, max(n + max(d, 0) for n, d in zip(lengths, dlen)))
    ctx = context(b, rows, max_len, hq, hk, dim, dt, cache, page, rot, interleaved, scaling,
                  magnitude)

    def gpu_(x, kind_=torch.float32):
        return None if x is None else torch.tensor(x, dtype=kind_).cuda()
    try:
        B.pld_kv_append_tree(ctx, q if with_q else None, wq if in_place else width, k, v, width,
                             rows, gpu_(lengths, torch.int32), gpu_(dlen, torch.int32),
                             gpu_(parent, torch.int32), b, torch.from_numpy(table).cuda(),
                             table.shape[1], kc, vc, pages, ks, vs, gpu_(nq), gpu_(nk), eps,
                             out_q if with_q else None)
        assert B.pld_sync(ctx) == B.PLD_OK, B.pld_last_error()
    finally:
        B.pld_destroy(ctx)
    gq, gk, gv = [x.double().cpu().numpy() for x in (out_q, kc, vc)]
    freq = R.rope_frequencies(rot, scaling, **ROPE)
    want_q, want_k, want_v = oq0.copy(), kc0.copy(), vc0.copy()
    tol_q, tol_k, tol_v = np.zeros_like(gq), np.zeros_like(gk), np.zeros_like(gv)
    off = 2.0**-20 + (dim / 2 + 8) * 2.0**-24
    for i in range(b):
        for t in range(R.block_rows(lengths[i], dlen[i])):
            r, cell = i * rows + t, lengths[i] - 1 + t
            deep = len(TR.branch(parent[i], t)) - 1 if tree else t
            at = lengths[i] - 1 + deep
            if with_q:
                x = TR.normed(q0[r].reshape(hq, dim), nq, eps)
                y, s = R.rotate(x, at, freq, rot, interleaved, magnitude)
                want_q[r] = y.reshape(-1)
                tol_q[r] = stored(dt, y, np.maximum(s, np.abs(x)), off).reshape(-1)
            x = TR.normed(k0[r].reshape(hk, dim), nk, eps)
            y, s = R.rotate(x, at, freq, rot, interleaved, magnitude)
            div = ks.double().cpu().numpy()[:, None] if scales else np.ones((hk, 1))
            y, s = y / div, (np.maximum(s, np.abs(x)) + np.abs(y) * 2.0**-4) / div
            top = LARGEST[cache]
            want_k[table[i, cell // page], :, cell % page] = np.clip(y, -top, top)
            tol_k[table[i, cell // page], :, cell % page] = stored(cache, y, s, off)
            div = vs.double().cpu().numpy()[:, None] if scales else np.ones((hk, 1))
            y = v0[r].reshape(hk, dim) / div
            want_v[table[i, cell // page], :, :, cell % page] = np.clip(y, -top, top)
            if cache != dt:
                tol_v[table[i, cell // page], :, :, cell % page] = stored(cache, y, np.abs(y),
                                                                          2.0**-24)
    for name, got, want, tol in (("q", gq, want_q, tol_q), ("k", gk, want_k, tol_k),
                                 ("v", gv, want_v, tol_v)):
        over = np.abs(got - want) - tol
        assert not np.isnan(over).any() and over.max() <= 0, (
            name, float(over.max()), np.unravel_index(np.argmax(over), over.shape))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_dims_and_layouts(dt, dim, interleaved):
    check([1, 40, 17], [5, 0, 3], 6, dim=dim, dt=dt, interleaved=interleaved, seed=dim)


@pytest.mark.parametrize("rot", [0, 2, 6, 16, 32, 62, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_the_head(rot, interleaved):
    check([30, 5], [9, 2], 10, dim=128, rot=rot, interleaved=interleaved, seed=rot)


@pytest.mark.parametrize("norms", ["", "q", "k", "qk"])
@pytest.mark.parametrize("rot", [64, 20])
def test_norms_on_either(norms, rot):
    check([30, 5], [9, 2], 10, rot=rot, norms=norms, seed=len(norms))


def test_small_large_and_zero_heads():
    # squares below fp32's smallest normal number, and above a float's range of
    # fp16 inputs; eps carries the zero heads
    check([30], [9], 10, dt="bf16", size=1e-3, eps=1e-5, seed=1)
    check([30], [9], 10, dt="f16", size=8000.0, eps=0.0, seed=2)
    check([30], [9], 10, dt="bf16", size=0.0, eps=1e-6, seed=3)


@pytest.mark.parametrize("scaling", ["linear", "banded"])
@pytest.mark.parametrize("start", [1, 262100, 2097000])
def test_far_positions(scaling, start):
    check([start], [30], 31, hq=2, hk=1, page=256, scaling=scaling, magnitude=1.25, seed=start)


@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 8), (12, 4), (16, 1), (5, 5), (64, 8)])
@pytest.mark.parametrize("page", [16, 256])
def test_heads_and_pages(hq, hk, page):
    check([250, 15, 16, 17, 63], [20, 1, 0, 15, 2], 21, hq=hq, hk=hk, page=page, seed=hq * page)


@pytest.mark.parametrize("kind", ["chain", "star", "comb", "binary"])
@pytest.mark.parametrize("rows", [64, 65, 256])
def test_deep_and_wide_trees(kind, rows):
    check([60, 1], [rows - 1, rows - 2], rows, kind=kind, hq=2, hk=1, seed=rows)


def test_chains_and_prompts():
    check([1, 100], [700, 33], 701, tree=False, hq=2, hk=1, page=64, seed=4)
    check([30, 5], [9, 2], 10, tree=False, rot=20, seed=5)
    check([30, 5], [0, 0], 1, tree=False, seed=6)


def test_empty_and_idle_requests_leave_everything():
    check([0, 5, 0, 9], [3, -1, -1, 2], 4)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("rot", [64, 20])
@pytest.mark.parametrize("scales", [False, True])
def test_eight_bit_cells(dt, rot, scales):
    check([30, 5, 16], [9, 2, 9], 10, dt=dt, cache="e4m3", rot=rot, scales=scales, seed=7)


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (8, 8), (5, 3)])
def test_strides_and_alignments(pad, offset):
    check([30, 5], [9, 2], 10, pad=pad, offset=offset, seed=8)


@pytest.mark.parametrize("rot", [64, 20])
def test_in_place_and_without_q(rot):
    check([30, 5], [9, 2], 10, rot=rot, in_place=True, seed=9)
    check([30, 5], [9, 2], 10, rot=rot, with_q=False, seed=10)


def _call(ctx, x, hq, hk, dim, rows, ln, dl, par, tab, kc, vc, pages, nq, nk, out, stream=None):
    w = x.shape[1]
    B.pld_kv_append_tree(ctx, x, w, x[:, hq * dim:], x[:, (hq + hk) * dim:], w, rows, ln, dl, par,
                         ln.numel(), tab, tab.shape[1], kc, vc, pages, None, None, nq, nk, 1e-6,
                         out, stream)


def _batch(rows=12, hq=4, hk=2, dim=64, page=16, b=3, seed=0):
    import torch
    rng = np.random.default_rng([9802, seed])
    lengths, dlen = [40, 7, 16], [rows - 1, 3, rows - 1]
    table, pages = table_for(rng, lengths, dlen, page)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(x=torch.randn(b * rows, (hq + 2 * hk) * dim).bfloat16().cuda(), hq=hq, hk=hk,
                dim=dim, rows=rows, ln=torch.tensor(lengths, **i32), dl=torch.tensor(dlen, **i32),
                par=torch.tensor([TR.random_tree(rng, rows - 1) for _ in range(b)], **i32),
                tab=torch.from_numpy(table).cuda(),
                kc=torch.zeros((pages, hk, page, dim), dtype=torch.bfloat16, device="cuda"),
                vc=torch.zeros((pages, hk, dim, page), dtype=torch.bfloat16, device="cuda"),
                pages=pages, nq=torch.rand(dim).cuda(), nk=torch.rand(dim).cuda(),
                out=torch.zeros((b * rows, hq * dim), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("rot", [64, 20])
@pytest.mark.parametrize("value", [-1, 5, 1 << 30])
def test_a_bad_parent_stores_nothing_and_spares_the_others(rot, value):
    import torch
    c = _batch()
    ctx = context(3, 12, 200, 4, 2, 64, "bf16", "bf16", 16, rot)
    try:
        _call(ctx, **c)
        assert B.pld_sync(ctx) == B.PLD_OK
        want = [x.clone() for x in (c["out"], c["kc"], c["vc"])]
        for x in (c["out"], c["kc"], c["vc"]):
            x.zero_()
        c["par"][0, 4] = value
        c["par"][1, 3:] = 99      # past its d
        _call(ctx, **c)
        assert B.pld_sync(ctx) == B.PLD_EINVAL
        assert bool((c["out"][:12] == 0).all())
        assert torch.equal(c["out"][12:], want[0][12:])
        mine = c["tab"][0, 2:4].long()   # positions 39 .. 50
        for got, w in ((c["kc"], want[1]), (c["vc"], want[2])):
            assert bool((got[mine] == 0).all())
            w[mine] = 0
            assert torch.equal(got, w)
    finally:
        B.pld_destroy(ctx)


@pytest.mark.parametrize("rot", [64, 20])
@pytest.mark.parametrize("field,value,status", [("dl", 12, B.PLD_EINVAL),
                                                ("dl", 2**31 - 1, B.PLD_EINVAL),
                                                ("dl", -2, B.PLD_EINVAL),
                                                ("ln", -1, B.PLD_EINVAL),
                                                ("ln", 195, B.PLD_ECAPACITY)])
def test_a_bad_block_stores_nothing(rot, field, value, status):
    c = _batch()
    ctx = context(3, 12, 200, 4, 2, 64, "bf16", "bf16", 16, rot)
    try:
        c[field][2] = value   # the last request: its tree ends the buffer
        _call(ctx, **c)
        assert B.pld_sync(ctx) == status
        assert bool((c["out"][24:] == 0).all()) and not bool((c["out"][:12] == 0).any())
        mine = c["tab"][2, :2].long()
        assert bool((c["kc"][mine] == 0).all()) and bool((c["vc"][mine] == 0).all())
    finally:
        B.pld_destroy(ctx)


def test_graph_replays_and_two_streams():
    import torch
    cases = [_batch(seed=1), _batch(seed=2)]
    ctxs = [context(3, 12, 200, 4, 2, 64, "bf16", "bf16", 16, 64) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    try:
        want = []
        for c, ctx in zip(cases, ctxs):
            _call(ctx, **c)
            assert B.pld_sync(ctx) == B.PLD_OK
            want.append([x.clone() for x in (c["out"], c["kc"], c["vc"])])
        for _ in range(4):
            for c in cases:
                for x in (c["out"], c["kc"], c["vc"]):
                    x.zero_()
            torch.cuda.synchronize()
            for c, ctx, st in zip(cases, ctxs, streams):
                with torch.cuda.stream(st):
                    _call(ctx, **c)
            for c, ctx, st, w in zip(cases, ctxs, streams, want):
                assert B.pld_sync(ctx, st) == B.PLD_OK
                for x, y in zip((c["out"], c["kc"], c["vc"]), w):
                    assert torch.equal(x, y)
        c, graph = cases[0], torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            _call(ctxs[0], **c)
        for i in range(3):
            for x in (c["out"], c["kc"], c["vc"]):
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip((c["out"], c["kc"], c["vc"]), want[0]):
                assert torch.equal(x, y)
    finally:
        for ctx in ctxs:
            B.pld_destroy(ctx)


def test_refusals_on_a_context():
    c = _batch()
    ctx = context(3, 300, 400, 4, 2, 64, "bf16", "bf16", 16, 64)
    x, w = c["x"], c["x"].shape[1]
    good = dict(q=x, q_stride=w, k=x[:, 256:], v=x[:, 384:], kv_stride=w, rows=12, lengths=c["ln"],
                draft_len=c["dl"], parent=c["par"], batch=3, page_table=c["tab"],
                table_stride=c["tab"].shape[1], k_cache=c["kc"], v_cache=c["vc"],
                n_pages=c["pages"], q_norm=c["nq"], k_norm=c["nk"], eps=1e-6, out_q=c["out"])
    try:
        B.pld_kv_append_tree(ctx, **{**good, "batch": 0})
        for change in ({"rows": 0}, {"rows": 257}, {"rows": 301}, {"batch": 4},
                       {"eps": -1e-6}, {"eps": float("nan")}, {"eps": float("inf")},
                       {"parent": c["par"].data_ptr() + 2}, {"q_norm": c["nq"].data_ptr() + 1},
                       {"k_norm": c["nk"].data_ptr() + 2}, {"q": None, "out_q": None},
                       {"q": None}, {"k": None}, {"v": None}, {"q_stride": 100},
                       {"kv_stride": 100}, {"n_pages": 0}, {"lengths": None}):
            with pytest.raises(B.PldError) as e:
                B.pld_kv_append_tree(ctx, **{**good, **change})
            assert e.value.status == B.PLD_EINVAL, change
        with pytest.raises(ValueError):
            B.pld_kv_append_tree(ctx, **{**good, "q_norm": c["nq"].half()})
        assert bool((c["kc"] == 0).all()) and B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)
