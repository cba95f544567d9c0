"""pld_verify_tree's, pld_kv_append_tree's and pld_kv_keep's kernels on the
host, one workgroup at a time, in a chosen order of its wavefronts
(tests/host_device). Arrays are numpy's."""

from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np

import host_verify as H

vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class VerifyArgs(ctypes.Structure):
    """TreeVerifyArgs of pld_target.h."""
    _fields_ = [("v", H.Args), ("parent", vp), ("out_path", vp)]


class AppendArgs(ctypes.Structure):
    """TreeAppendArgs of pld_target.h."""
    _fields_ = [("kv", H.KvArgs), ("parent", vp), ("q_norm", vp), ("k_norm", vp), ("eps", f32)]


class KeepArgs(ctypes.Structure):
    """KeepArgs of pld_target.h."""
    _fields_ = [("blk", H.BlockArgs), ("path", vp), ("accepted", vp), ("k_cache", vp),
                ("v_cache", vp), ("layers", i32), ("k_layer", i64), ("v_layer", i64)]


def build(folder, source):
    """The library of tests/host_device/<source>, compiled into `folder`."""
    lib = os.path.join(str(folder), "lib" + source + ".so")
    subprocess.run([H.CLANG, "-x", "c++", "-std=c++17", "-O2", "-mf16c", "-fPIC", "-shared",
                    "-Wno-keyword-macro", "-Wno-unused-value",
                    "-I", os.path.join(H.HERE, "host_device"),
                    "-I", os.path.join(H.ROOT, "include"),
                    "-I", os.path.join(H.ROOT, "prompt_lookup_gram_amd", "csrc"),
                    os.path.join(H.HERE, "host_device", source), "-o", lib], check=True)
    out = ctypes.CDLL(lib)
    if source == "tree_verify.cpp":
        out.host_verify_tree.argtypes = [ctypes.POINTER(VerifyArgs), vp, i32, i32, vp]
        out.host_verify_tree_grid.restype = ctypes.c_uint64
        out.host_verify_tree_grid.argtypes = [i32] * 4
    else:
        out.host_append_tree.argtypes = [ctypes.POINTER(AppendArgs), vp, i32, vp]
        out.host_kv_keep.argtypes = [ctypes.POINTER(KeepArgs), vp, i32, vp]
    return out


def verify(lib, ctx, logits, dtype, draft, dlen, parent, uniform, temperature=None,
           order=H.ORDERS[0], walk=False):
    """One call on a host_verify.Context: (tokens, path, accepted, counts,
    logprobs, error bits, broken barriers). walk: only the path's rows are
    read."""
    b, rows, v = logits.shape
    keep = [np.ascontiguousarray(x) if x is not None else None for x in (
        logits, np.asarray(draft, np.int32), np.asarray(dlen, np.int32),
        None if temperature is None else np.asarray(temperature, np.float32),
        np.asarray(uniform, np.float32),
        None if parent is None else np.asarray(parent, np.int32))]
    ptr = [None if x is None else x.ctypes.data for x in keep]
    tok, path = np.full((b, rows), -7, np.int32), np.full((b, rows), -7, np.int32)
    acc, cnt = np.full(b, -7, np.int32), np.full(b, -7, np.int32)
    logp, err = np.full((b, rows), 7.0, np.float32), np.zeros(1, np.uint32)
    a = VerifyArgs(H.Args(ptr[0], dtype, v, rows, b, v, ptr[1], ptr[2], None, None, 0, ptr[3],
                          ptr[4], tok.ctypes.data, acc.ctypes.data, cnt.ctypes.data,
                          logp.ctypes.data, err.ctypes.data, ctx.ptr, *ctx.size[:2]),
                   ptr[5], path.ctypes.data)
    o, report = np.asarray(order, np.int32), np.zeros(2, np.int64)
    assert lib.host_verify_tree(ctypes.byref(a), o.ctypes.data, len(o), int(walk),
                                report.ctypes.data) == 0
    assert report[1] == 0, "a workgroup waits for ever"
    assert (ctx.raw[:ctx.at] == 0xa5).all() and (
        ctx.raw[ctx.at + ctx.bytes:] == 0xa5).all(), "outside the workspace"
    return tok, path, acc, cnt, logp, int(err[0]), int(report[0])
