"""pld_verify's and pld_kv_append's kernels on the host, one workgroup at a
time, in a chosen order of its wavefronts (tests/host_device). Arrays are
numpy's."""

from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CLANG = os.environ.get("HOST_CLANG", "/opt/rocm/llvm/bin/clang++")
F32, F16, BF16 = 0, 1, 2
BAD_BLOCK = 256
ORDERS = [(0, 1, 2, 3), (3, 2, 1, 0), (2, 0, 3, 1), (1, 3, 0, 2)]

vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class Args(ctypes.Structure):
    """VerifyArgs of pld_target.h."""
    _fields_ = [("logits", vp), ("dtype", i32), ("stride", i64), ("rows", i32), ("batch", i32),
                ("vocab", i32), ("draft", vp), ("draft_len", vp), ("src", vp), ("probs", vp),
                ("head", i32), ("temperature", vp), ("uniform", vp), ("out_tokens", vp),
                ("out_accepted", vp), ("out_counts", vp), ("out_logprobs", vp), ("err", vp),
                ("stats", vp), ("max_batch", i32), ("max_rows", i32)]


class BlockArgs(ctypes.Structure):
    """BlockArgs of pld_target.h."""
    _fields_ = [("lengths", vp), ("draft_len", vp), ("rows", i32), ("batch", i32),
                ("max_len", i32), ("table", vp), ("table_stride", i64), ("n_pages", i64),
                ("page_shift", i32), ("q_heads", i32), ("kv_heads", i32), ("head_dim", i32),
                ("dtype", i32), ("cache_dtype", i32), ("k_scale", vp), ("v_scale", vp),
                ("err", vp)]


class KvArgs(ctypes.Structure):
    """KvAppendArgs of pld_target.h."""
    _fields_ = [("blk", BlockArgs), ("q", vp), ("q_stride", i64), ("k", vp), ("v", vp),
                ("kv_stride", i64), ("k_cache", vp), ("v_cache", vp), ("out_q", vp),
                ("turns", vp), ("rot_dim", i32), ("interleaved", i32), ("magnitude", f32)]


def build(folder, source="verify.cpp"):
    """The library of tests/host_device/<source>, compiled into `folder`."""
    lib = os.path.join(str(folder), "lib" + source + ".so")
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-O2", "-mf16c", "-fPIC", "-shared",
                    "-Wno-keyword-macro", "-Wno-unused-value",
                    "-I", os.path.join(HERE, "host_device"), "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "prompt_lookup_gram_amd", "csrc"),
                    os.path.join(HERE, "host_device", source), "-o", lib], check=True)
    out = ctypes.CDLL(lib)
    if source == "verify.cpp":
        out.host_workspace.restype = ctypes.c_size_t
        out.host_workspace.argtypes = [i32, i32, i32]
        out.host_clear.argtypes = out.host_counters_clear.argtypes = [vp, i32, i32, i32]
        out.host_verify.argtypes = [ctypes.POINTER(Args), vp, i32, i32, vp]
        out.host_verify_grid.restype = ctypes.c_uint64
        out.host_verify_grid.argtypes = [i32] * 5
    else:
        out.host_kv_append.argtypes = [ctypes.POINTER(KvArgs), vp, i32, vp]
        out.host_kv_grid.restype = ctypes.c_uint64
        out.host_kv_grid.argtypes = [i32] * 4
    return out


def bits(x, dtype):
    """Values rounded to a logits type: the array to pass, and as float64."""
    if dtype == F32:
        y = np.asarray(x, np.float32)
        return y, y.astype(np.float64)
    if dtype == F16:
        y = np.asarray(x, np.float16)
        return y, y.astype(np.float64)
    w = np.ascontiguousarray(np.asarray(x, np.float32)).view(np.uint32)
    y = ((w + 0x7fff + ((w >> 16) & 1)) >> 16).astype(np.uint16)
    return y, (y.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


class Context:
    """A workspace, guarded on both sides."""

    GUARD = 4096

    def __init__(self, lib, batch, rows, vocab):
        self.lib, self.size = lib, (batch, rows, vocab)
        self.bytes = lib.host_workspace(batch, rows, vocab)
        raw = np.full(self.bytes + 2 * self.GUARD + 64, 0xa5, np.uint8)
        skip = -(raw.ctypes.data + self.GUARD) % 64
        self.raw, self.at = raw, skip + self.GUARD
        assert lib.host_clear(raw.ctypes.data + self.at, *self.size) == 0

    @property
    def ptr(self):
        return self.raw.ctypes.data + self.at

    def verify(self, logits, dtype, draft, dlen, uniform, src=None, probs=None, temperature=None,
               order=ORDERS[0], refuse_row=0):
        """One call: (tokens, accepted, counts, logprobs, error bits, broken
        barriers)."""
        b, rows, v = logits.shape
        assert v == self.size[2]
        keep = [np.ascontiguousarray(x) if x is not None else None for x in (
            logits, np.asarray(draft, np.int32), np.asarray(dlen, np.int32),
            None if src is None else np.asarray(src, np.uint64),
            None if probs is None else np.asarray(probs, np.float32),
            None if temperature is None else np.asarray(temperature, np.float32),
            np.asarray(uniform, np.float32))]
        ptr = [None if x is None else x.ctypes.data for x in keep]
        tok = np.full((b, rows), -7, np.int32)
        acc, cnt = np.full(b, -7, np.int32), np.full(b, -7, np.int32)
        logp, err = np.full((b, rows), 7.0, np.float32), np.zeros(1, np.uint32)
        a = Args(ptr[0], dtype, v, rows, b, v, ptr[1], ptr[2], ptr[3], ptr[4],
                 0 if probs is None else probs.shape[1], ptr[5], ptr[6], tok.ctypes.data,
                 acc.ctypes.data, cnt.ctypes.data, logp.ctypes.data, err.ctypes.data, self.ptr,
                 *self.size[:2])
        o, report = np.asarray(order, np.int32), np.zeros(2, np.int64)
        assert self.lib.host_verify(ctypes.byref(a), o.ctypes.data, len(o), refuse_row,
                                    report.ctypes.data) == 0
        assert report[1] == 0, "a workgroup waits for ever"
        assert (self.raw[:self.at] == 0xa5).all() and (
            self.raw[self.at + self.bytes:] == 0xa5).all(), "outside the workspace"
        return tok, acc, cnt, logp, int(err[0]), int(report[0])

    def clear(self):
        """Whether the counters are as a call must leave them."""
        return bool(self.lib.host_counters_clear(self.ptr, *self.size))
