"""pld_kv_append_tree's and pld_kv_keep's kernels themselves, run on the CPU a
workgroup at a time in several orders of its wavefronts (tests/host_device),
against the 64-bit reference (no GPU needed).

Tolerances are those of tests/test_kv_append_gpu.py, with the norm's: its sum
of squares is at most (head_dim + 6) additions and products of 2^-24 off, half
of which the root keeps, and the root, the quotient, the two products with it
four more roundings: below (head_dim / 2 + 8) * 2^-24 of a value."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

import host_tree as T
import host_verify as H
import target_reference as R
import tree_reference as TR

F16, BF16 = H.F16, H.BF16


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return T.build(tmp_path_factory.mktemp("host_tree_kv"), "tree_kv.cpp")


def table_for(rng, lengths, dlen, page):
    need = [max(1, -(-(n + max(0, d)) // page)) for n, d in zip(lengths, dlen)]
    ids = rng.permutation(sum(need) + 2)
    table = np.zeros((len(need), max(need)), np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table, sum(need) + 2


def widen(raw, dtype):
    if dtype == F16:
        return np.ascontiguousarray(raw).view(np.float16).astype(np.float64)
    return (raw.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def append(lib, rng, lengths, dlen, rows, parent, hq=4, hk=2, dim=64, dtype=BF16, page=16, rot=64,
           interleaved=False, pad=0, norms=True, with_q=True, in_place=False, order=H.ORDERS[0],
           max_len=None, eps=1e-6):
    b = len(lengths)
    table, pages = table_for(rng, lengths, dlen, page)
    qw, kw = hq * dim + (0 if in_place else pad), hk * dim + pad
    q, q64 = H.bits(rng.standard_normal((b * rows, qw)), dtype)
    k, k64 = H.bits(rng.standard_normal((b * rows, kw)) * 3, dtype)
    v, v64 = H.bits(rng.standard_normal((b * rows, kw)), dtype)
    one = np.uint16(7)
    kc = np.full((pages, hk, page, dim), one, np.uint16)
    vc = np.full((pages, hk, dim, page), one, np.uint16)
    out = q if in_place else np.full((b * rows, hq * dim), one, np.uint16)
    wq = rng.uniform(0.5, 1.5, dim).astype(np.float32) if norms else None
    wk = rng.uniform(0.5, 1.5, dim).astype(np.float32) if norms else None
    freq = R.rope_frequencies(rot, base=1e4) if rot else np.zeros(0)
    turns = np.ascontiguousarray(freq / (2 * math.pi))
    q, k, v = (x.view(np.uint16) for x in (q, k, v))
    out = q if in_place else out
    ln, dl = np.asarray(lengths, np.int32), np.asarray(dlen, np.int32)
    par = None if parent is None else np.asarray(parent, np.int32)
    err = np.zeros(1, np.uint32)

    def ptr(x):
        return None if x is None else x.ctypes.data
    blk = H.BlockArgs(ptr(ln), ptr(dl), rows, b, max_len or 1 << 20, ptr(table), table.shape[1],
                      pages, int(math.log2(page)), hq, hk, dim, dtype, dtype, None, None, ptr(err))
    a = T.AppendArgs(H.KvArgs(blk, ptr(q) if with_q else None, qw, ptr(k), ptr(v), kw, ptr(kc),
                              ptr(vc), ptr(out) if with_q else None, ptr(turns), rot,
                              int(interleaved), 1.0), ptr(par), ptr(wq) if with_q else None,
                     ptr(wk), eps)
    o, report = np.asarray(order, np.int32), np.zeros(2, np.int64)
    assert lib.host_append_tree(ctypes.byref(a), o.ctypes.data, len(o), report.ctypes.data) == 0
    assert report[0] == 0 and report[1] == 0

    want_k, size_k = np.full(kc.shape, np.nan), np.zeros(kc.shape)
    want_v = np.full(vc.shape, np.nan)
    want_q = np.full((b * rows, hq, dim), np.nan)
    size_q = np.zeros(want_q.shape)
    for i in range(b):
        n = R.block_rows(lengths[i], dlen[i])
        for t in range(n):
            r, cell = i * rows + t, lengths[i] - 1 + t
            deep = t if parent is None else len(TR.branch(parent[i], t)) - 1
            at = lengths[i] - 1 + deep
            page_id, slot = table[i, cell // page], cell % page
            x = TR.normed(k64[r, :hk * dim].reshape(hk, dim), wk, eps)
            y, s = R.rotate(x, at, freq, rot, interleaved, 1.0)
            want_k[page_id, :, slot], size_k[page_id, :, slot] = y, np.maximum(s, np.abs(x))
            want_v[page_id, :, :, slot] = v64[r, :hk * dim].reshape(hk, dim)
            x = TR.normed(q64[r, :hq * dim].reshape(hq, dim), wq, eps)
            y, s = R.rotate(x, at, freq, rot, interleaved, 1.0)
            want_q[r], size_q[r] = y, np.maximum(s, np.abs(x))
    half = 2.0**-11 if dtype == F16 else 2.0**-8
    tiny = 2.0**-25 if dtype == F16 else 2.0**-134
    off = 2.0**-20 + (dim / 2 + 8) * 2.0**-24

    def check(got, want, size):
        live = ~np.isnan(want)
        assert (got[~live] == one).all(), "a cell of another position was written"
        lim = off * size + half * (np.abs(want) + off * size) + tiny
        assert (np.abs(widen(got, dtype) - want) <= lim)[live].all()
    check(kc, want_k, size_k)
    check(vc, want_v, np.zeros(vc.shape))
    if with_q and not in_place:
        check(out.reshape(b * rows, hq, dim), want_q, size_q)
    elif with_q:
        live = ~np.isnan(want_q)
        got = widen(out.reshape(b * rows, hq, dim), dtype)
        assert (np.abs(got - want_q) <= off * size_q + half * (np.abs(want_q) + off * size_q)
                + tiny)[live].all()
    return int(err[0])


@pytest.mark.parametrize("dim,rot", [(64, 64), (96, 96), (128, 128), (192, 128), (256, 64),
                                     (128, 0), (96, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_words(lib, dim, rot, interleaved):
    rng = np.random.default_rng([9611, dim, rot])
    parent = [TR.random_tree(rng, 9) for _ in range(3)]
    for order in H.ORDERS[:2]:
        assert append(lib, rng, [40, 1, 13], [9, 4, 0], 10, parent, dim=dim, rot=rot, hq=6,
                      interleaved=interleaved, order=order) == 0


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("pad,rot,dim", [(1, 64, 64), (3, 20, 96), (8, 12, 128)])
def test_elements(lib, dtype, pad, rot, dim):
    rng = np.random.default_rng([9612, dtype, pad])
    parent = [TR.random_tree(rng, 5) for _ in range(2)]
    for interleaved in (False, True):
        assert append(lib, rng, [20, 7], [5, 2], 6, parent, dim=dim, rot=rot, dtype=dtype,
                      pad=pad, interleaved=interleaved) == 0


def test_without_norms_without_q_in_place_and_as_a_chain(lib):
    rng = np.random.default_rng(9613)
    parent = [TR.random_tree(rng, 7) for _ in range(2)]
    assert append(lib, rng, [20, 7], [7, 6], 8, parent, norms=False) == 0
    assert append(lib, rng, [20, 7], [7, 6], 8, parent, with_q=False) == 0
    assert append(lib, rng, [20, 7], [7, 6], 8, parent, in_place=True) == 0
    assert append(lib, rng, [20, 7], [7, 6], 8, parent, in_place=True, rot=20) == 0
    assert append(lib, rng, [1, 30], [299, 17], 300, None, hk=1, hq=1) == 0


@pytest.mark.parametrize("kind", ["chain", "star", "comb", "binary"])
def test_deep_and_wide_trees(lib, kind):
    rng = np.random.default_rng(9614)
    assert append(lib, rng, [33], [255], 256, [TR.shapes(255)[kind]], hq=1, hk=1) == 0


def test_bad_parents_store_nothing(lib):
    rng = np.random.default_rng(9615)
    for bad in (-1, 3, 99):
        for words in (64, 20):
            parent = np.array([TR.random_tree(rng, 5) for _ in range(2)])
            parent[0, 2] = bad
            lengths, dlen = [20, 7], [5, 5]
            # (the reference leaves the request out: as if it had no rows)
            b, rows, hk, dim, page = 2, 6, 2, 64, 16
            table, pages = table_for(rng, lengths, dlen, page)
            q = np.zeros((b * rows, 4 * dim), np.uint16)
            kv = np.zeros((b * rows, hk * dim), np.uint16)
            kc, vc = (np.full((pages, hk, page * dim), 7, np.uint16) for _ in range(2))
            out = np.full_like(q, 7)
            turns = np.zeros(32)
            ln, dl = np.array(lengths, np.int32), np.array(dlen, np.int32)
            par, err = parent.astype(np.int32), np.zeros(1, np.uint32)
            blk = H.BlockArgs(ln.ctypes.data, dl.ctypes.data, rows, b, 1000, table.ctypes.data,
                              table.shape[1], pages, 4, 4, hk, dim, BF16, BF16, None, None,
                              err.ctypes.data)
            a = T.AppendArgs(H.KvArgs(blk, q.ctypes.data, 4 * dim, kv.ctypes.data, kv.ctypes.data,
                                      hk * dim, kc.ctypes.data, vc.ctypes.data, out.ctypes.data,
                                      turns.ctypes.data, words, 0, 1.0), par.ctypes.data, None,
                             None, 0.0)
            o, report = np.asarray(H.ORDERS[0], np.int32), np.zeros(2, np.int64)
            assert lib.host_append_tree(ctypes.byref(a), o.ctypes.data, 4, report.ctypes.data) == 0
            assert int(err[0]) == H.BAD_BLOCK
            assert (out[:6] == 7).all() and (out[6:] == 0).all()
            assert (kc == 0).sum() == (vc == 0).sum() == 6 * hk * dim


def kept(lib, rng, lengths, dlen, paths, accepted, rows, hk=2, dim=64, page=16, layers=2, byte=False,
         order=H.ORDERS[0], table=None, pages=None, gap=0):
    b = len(lengths)
    if table is None:
        table, pages = table_for(rng, lengths, dlen, page)
    kind = np.uint8 if byte else np.uint16
    cells = pages * hk * page * dim
    k = rng.integers(0, 200, layers * (cells + gap)).astype(kind)
    v = rng.integers(0, 200, layers * (cells + gap)).astype(kind)
    k0, v0 = k.copy(), v.copy()
    path = np.full((b, rows), -1, np.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = p
    ln, dl = np.asarray(lengths, np.int32), np.asarray(dlen, np.int32)
    acc, err = np.asarray(accepted, np.int32), np.zeros(1, np.uint32)
    blk = H.BlockArgs(ln.ctypes.data, dl.ctypes.data, rows, b, 1 << 20, table.ctypes.data,
                      table.shape[1], pages, int(math.log2(page)), hk, hk, dim, BF16,
                      3 if byte else BF16, None, None, err.ctypes.data)
    a = T.KeepArgs(blk, path.ctypes.data, acc.ctypes.data, k.ctypes.data, v.ctypes.data, layers,
                   cells + gap, cells + gap)
    o, report = np.asarray(order, np.int32), np.zeros(2, np.int64)
    assert lib.host_kv_keep(ctypes.byref(a), o.ctypes.data, len(o), report.ctypes.data) == 0
    assert report[0] == 0 and report[1] == 0

    def shaped(x, *shape):
        return x.reshape(layers, cells + gap)[:, :cells].reshape(layers, pages, hk, *shape)
    moves = [0 if err[0] and i in kept.bad else m for i, m in enumerate(accepted)]
    wk, wv = TR.keep(shaped(k0, page, dim), shaped(v0, dim, page), table, lengths, paths, moves,
                     page)
    assert np.array_equal(shaped(k, page, dim), wk)
    assert np.array_equal(shaped(v, dim, page), wv)
    assert np.array_equal(k.reshape(layers, -1)[:, cells:], k0.reshape(layers, -1)[:, cells:])
    return int(err[0])


kept.bad = ()


@pytest.mark.parametrize("byte", [False, True])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_kept_cells(lib, byte, dim, page):
    rng = np.random.default_rng([9621, dim, page])
    rows = 70
    for order in H.ORDERS[:2]:
        paths = [[0] + sorted(rng.choice(np.arange(1, 70), n, replace=False).tolist())
                 for n in (0, 1, 5, 9, 30, 69)]
        lengths = [int(x) for x in rng.integers(1, 100, 6)]
        assert kept(lib, rng, lengths, [69] * 6, paths, [len(p) - 1 for p in paths], rows,
                    dim=dim, page=page, byte=byte, order=order, gap=64) == 0


def test_moves_onto_each_others_sources(lib):
    rng = np.random.default_rng(9622)
    paths = [[0, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11], [0, 1, 2, 3], [0, 1, 3, 4, 7, 9, 10]]
    assert kept(lib, rng, [17, 30, 1], [11, 11, 11], paths, [10, 3, 6], 12, layers=3) == 0


def test_bad_paths_move_nothing(lib):
    rng = np.random.default_rng(9623)
    good = [0, 2, 5]
    for path, accepted in (([0, 5, 5], 2), ([1, 2, 5], 2), ([0, 2, 8], 2), ([0, -3, 5], 2),
                           ([0, 2, 5], 8), ([0, 2, 5], -1), ([0, 2], 2)):
        kept.bad = (0,)
        assert kept(lib, rng, [20, 20], [7, 7], [path, good], [accepted, 2], 8) == H.BAD_BLOCK
    kept.bad = ()
    # nothing accepted, and requests without rows: nothing to look at
    assert kept(lib, rng, [20, 0, 9], [7, 7, -1], [[-1], good, good], [0, 0, 0], 8) == 0


def test_bad_pages_move_nothing(lib):
    rng = np.random.default_rng(9624)
    table = np.array([[0, 9], [1, 2]], np.int32)
    kept.bad = (0,)
    try:
        assert kept(lib, rng, [16, 16], [3, 3], [[0, 2, 3], [0, 1, 3]], [2, 2], 4, table=table,
                    pages=4) == 512
    finally:
        kept.bad = ()
