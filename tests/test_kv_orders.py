"""pld_kv_append's kernels on the host, against the 64-bit reference, over orders
in which the wavefronts of a workgroup may run (no GPU needed). Tolerances are
test_kv_append_gpu.py's."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

import host_verify as H
import target_reference as R


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return H.build(tmp_path_factory.mktemp("host"), "kv.cpp")


def half(dtype, ref, extra):
    eps, tiny = (2.0**-11, 2.0**-25) if dtype == H.F16 else (2.0**-8, 2.0**-134)
    return extra + eps * (np.abs(ref) + extra) + tiny


def values(x, dtype):
    if dtype == H.F16:
        return x.astype(np.float64)
    return (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("dtype", [H.F16, H.BF16])
@pytest.mark.parametrize("interleaved", [0, 1])
@pytest.mark.parametrize("rot,pad,rows", [(64, 8, 6), (32, 8, 400), (64, 8, 400), (24, 8, 6),
                                          (64, 3, 6), (0, 8, 400)])
def test_orders(lib, dtype, interleaved, rot, pad, rows):
    # (rows 400: 1,600 rows, four a workgroup; rot 24 and pad 3: an element at a time)
    rng = np.random.default_rng([9601, rot, rows])
    batch, hq, hk, dim, page = 4, 2, 1, 64, 16
    lengths = np.array([30, 1, 7, 64], np.int32)
    dlen = np.array([min(rows - 1, 26), min(rows - 1, 3), 0, -1], np.int32)
    width = 8
    table = rng.permutation(batch * width).astype(np.int32).reshape(batch, width)
    stride = (hq + 2 * hk) * dim + pad
    x, x64 = H.bits(rng.standard_normal((batch * rows, stride)), dtype)
    freq = R.rope_frequencies(rot)
    turns = freq / (2 * math.pi)
    cells = batch * width * hk * page * dim
    wq = hq * dim
    for order in H.ORDERS:
        q = np.full((batch * rows, wq), 7, x.dtype)
        kc, vc = np.full(cells, 9, x.dtype), np.full(cells, 9, x.dtype)
        err, report = np.zeros(1, np.uint32), np.zeros(2, np.int64)
        size = x.dtype.itemsize
        blk = H.BlockArgs(lengths.ctypes.data, dlen.ctypes.data, rows, batch, 4096,
                          table.ctypes.data, width, batch * width, 4, hq, hk, dim, dtype, dtype,
                          None, None, err.ctypes.data)
        a = H.KvArgs(blk, x.ctypes.data, stride, x.ctypes.data + wq * size,
                     x.ctypes.data + (wq + hk * dim) * size, stride, kc.ctypes.data,
                     vc.ctypes.data, q.ctypes.data, turns.ctypes.data, rot, interleaved, 1.25)
        o = np.asarray(order, np.int32)
        assert lib.host_kv_append(ctypes.byref(a), o.ctypes.data, 4, report.ctypes.data) == 0
        assert err[0] == 0 and report.tolist() == [0, 0], report
        want_q, tol_q = values(np.full_like(q, 7), dtype), np.zeros(q.shape)
        want_k = values(np.full_like(kc, 9), dtype).reshape(-1, hk, page, dim)
        want_v = values(np.full_like(vc, 9), dtype).reshape(-1, hk, dim, page)
        tol_k = np.zeros_like(want_k)
        for b in range(batch):
            for t in range(R.block_rows(lengths[b], dlen[b])):
                r, p = b * rows + t, lengths[b] - 1 + t
                y, s = R.rotate(x64[r, :wq].reshape(hq, dim), p, freq, rot, bool(interleaved),
                                1.25)
                want_q[r], tol_q[r] = y.reshape(-1), half(dtype, y, 2.0**-20 * s).reshape(-1)
                y, s = R.rotate(x64[r, wq:wq + hk * dim].reshape(hk, dim), p, freq, rot,
                                bool(interleaved), 1.25)
                cell = table[b, p // page], slice(None), p % page
                want_k[cell], tol_k[cell] = y, half(dtype, y, 2.0**-20 * s)
                want_v[table[b, p // page], :, :, p % page] = (
                    x64[r, wq + hk * dim:wq + 2 * hk * dim].reshape(hk, dim))
        assert (np.abs(values(q, dtype) - want_q) <= tol_q).all(), order
        assert (np.abs(values(kc, dtype).reshape(want_k.shape) - want_k) <= tol_k).all(), order
        assert (values(vc, dtype).reshape(want_v.shape) == want_v).all(), order


@pytest.mark.parametrize("words", [0, 1])
def test_grids_fit_the_hardwares_count_of_threads(lib, words):
    """A grid is counted in threads, in 32 bits: sizes beyond are refused."""
    ran = 0
    for batch, rows, heads in [(1, 1, 1), (64, 16, 8), (2**20, 16, 1), (2**20, 17, 1),
                               (2**24 - 1, 1, 1), (2**24, 1, 1), (2**30, 1, 1), (1, 2**30, 1),
                               (2**20, 4, 16)]:
        threads = lib.host_kv_grid(batch, rows, heads, words)
        assert threads < 2**32, (batch, rows, heads)
        ran += threads > 0
    assert ran >= 3
