"""The tree's calls on the host: refusals before anything touches the GPU, the
checks of parents under sanitizers, and the 64-bit reference against values
derived by hand (no GPU needed)."""

from __future__ import annotations

import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import target_reference as R
import tree_reference as TR
from prompt_lookup_gram_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_null_context_refused():
    f32, lib = ctypes.c_float(0), B.load()
    assert lib.pld_kv_append_tree(None, None, 0, None, None, 0, 1, None, None, None, 0, None, 1,
                                  None, None, 0, None, None, None, None, f32, None,
                                  None) == B.PLD_EINVAL
    assert lib.pld_attend_tree(None, None, 0, 1, None, None, None, 0, 0, None, 1, None, None, 0,
                               None, None, f32, 0, None, None, None) == B.PLD_EINVAL
    assert lib.pld_verify_tree(None, None, 0, 1, 1, None, None, None, None, None, 0, None, None,
                               None, None, None, None) == B.PLD_EINVAL
    assert lib.pld_kv_keep(None, None, None, None, None, 1, 0, None, 1, None, None, 0, 1, 0, 0,
                           None) == B.PLD_EINVAL
    assert "ctx is null" in B.pld_last_error()


def test_binding_checks_tensors_before_the_call():
    import torch
    cpu, idx = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        B.pld_kv_append_tree(1, cpu.half(), 8, None, None, 0, 1, None, None, None, 0, None, 1,
                             None, None, 0)
    with pytest.raises(ValueError, match="on the GPU"):
        B.pld_attend_tree(1, None, 8, 1, None, None, idx, 0, 0, None, 1, None, None, 0)
    with pytest.raises(ValueError, match="on the GPU"):
        B.pld_verify_tree(1, cpu, 8, 1, None, None, None, None, None, 0, None, None, None, None)
    with pytest.raises(TypeError, match="logits"):
        B.pld_verify_tree(1, 1234, 8, 1, None, None, None, None, None, 0, None, None, None, None)
    with pytest.raises(ValueError, match="on the GPU"):
        B.pld_kv_keep(1, None, None, idx, None, 1, 0, None, 1, None, None, 0)


PARENTS = r"""
#include <climits>
#include <cstdio>
#include <memory>

#include "pld_tree.h"

int main()
{
    int fails = 0;
    const int32_t values[] = {INT_MIN, -1, 0, 1, 2, 3, 4, 5, 254, 255, 256, INT_MAX};
    for (int32_t rows : {1, 2, 6, 256})
        for (int32_t d : {INT_MIN, -1, 0, 1, 5, 255, 256, INT_MAX})
            for (int32_t value : values)
                for (int32_t t = -1; t < 260; ++t) {
                    // exactly as long as the call says
                    std::unique_ptr<int32_t[]> p(new int32_t[2 * (rows - 1) + 1]);
                    for (int i = 0; i < 2 * (rows - 1); ++i)
                        p[i] = value;
                    std::unique_ptr<int32_t[]> k(new int32_t[2]{0, d});
                    pld::BlockArgs a{};
                    a.rows = rows;
                    a.draft_len = k.get();
                    bool stray = false;
                    const int32_t got = pld::parent_of(rows > 1 ? p.get() : nullptr, a, 1, t, stray);
                    const bool node = t >= 1 && t <= d && t < rows;
                    const bool fine = value >= 0 && value < t;
                    if (got != (node && fine ? value : 0) || stray != (node && !fine))
                        printf("%d %d %d %d\n", rows, d, value, t), ++fails;
                    stray = false;
                    if (pld::parent_of(nullptr, a, 1, t, stray) != (node ? t - 1 : 0) || stray)
                        ++fails;
                }
    return fails != 0;
}
"""


def test_parents_under_sanitizers(tmp_path):
    src, exe = tmp_path / "parents.cpp", tmp_path / "parents"
    src.write_text(PARENTS)
    subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-Wall", "-Wextra", "-Werror",
                    "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "prompt_lookup_gram_amd", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120,
                       env={**os.environ,
                            "ASAN_OPTIONS": "detect_leaks=0:verify_asan_link_order=0"})
    assert r.returncode == 0, r.stdout + r.stderr


# ---------------------------------------------------------------------------
# the reference, against values derived by hand
# ---------------------------------------------------------------------------


def test_reference_branches_and_norms():
    parent = [0, 0, 1, 3]
    assert TR.branch(parent, 0) == [0] and TR.branch(parent, 4) == [4, 3, 1, 0]
    assert TR.branch(parent, 2) == [2, 0]
    x = np.array([[3.0, -4.0]])
    assert np.allclose(TR.normed(x, np.array([1.0, 2.0]), 0.0),
                       np.array([[3.0, -8.0]]) / math.sqrt(12.5))
    assert np.allclose(TR.normed(x, np.ones(2), 12.5), x / 5)
    for d in (1, 2, 7, 30):
        for kind, p in TR.shapes(d).items():
            assert len(p) == d and all(0 <= q < t for t, q in enumerate(p, 1)), kind


def test_reference_attention_of_a_chain_is_the_chains():
    rng = np.random.default_rng(9651)
    b, rows, hq, hk, dim, page = 2, 4, 4, 2, 8, 16
    q = rng.standard_normal((b, rows, hq, dim))
    kc, vc = rng.standard_normal((5, hk, page, dim)), rng.standard_normal((5, hk, dim, page))
    table = np.array([[0, 3], [4, 1]])
    for window in (0, 2, 9):
        want = R.attend(q, kc, vc, table, [20, 1], [3, 2], page, 0.4, window)
        got = TR.attend(q, kc, vc, table, [20, 1], [3, 2], [[0, 1, 2]] * 2, page, 0.4, window)
        for x, y in zip(got, want):
            assert np.allclose(x, y, equal_nan=True)


def test_reference_attention_of_siblings():
    # a root with two children: each sees the root and itself
    kc, vc = np.zeros((1, 1, 16, 2)), np.zeros((1, 1, 2, 16))
    vc[0, 0, 0, :3] = [1.0, 10.0, 100.0]
    q, table = np.zeros((1, 3, 1, 2)), np.zeros((1, 1), int)
    out, lse, _, _ = TR.attend(q, kc, vc, table, [1], [2], [[0, 0]], 16, 1.0, 0)
    assert np.allclose(out[0, :, 0, 0], [1.0, 5.5, 50.5])
    assert np.allclose(lse[0, :, 0], [0.0, math.log(2), math.log(2)])
    # a window of one: themselves
    out, _, _, _ = TR.attend(q, kc, vc, table, [1], [2], [[0, 0]], 16, 1.0, 1)
    assert np.allclose(out[0, :, 0, 0], [1.0, 10.0, 100.0])


def test_reference_verification():
    p0, p1, p2 = [0.5, 0.3, 0.2], [0.1, 0.6, 0.3], [0.25, 0.25, 0.5]
    z = np.log(np.array([p0, p1, p2]))
    tree = [0, 0]
    # the first child taken; then its row draws
    assert TR.verify_one(z, [0, 1], tree, 2, 1.0, [0.49, 0.0], 0.69)[:2] == ([0, 1], [0, 1])
    # refused: the second is tried with what is left, 0.3 of 0.5
    assert TR.verify_one(z, [0, 1], tree, 2, 1.0, [0.51, 0.59], 0.6)[:2] == ([1, 2], [0, 2])
    # both refused: only token 2 is left
    tok, path, logp = TR.verify_one(z, [0, 1], tree, 2, 1.0, [0.51, 0.61], 0.0)
    assert tok == [2] and path == [0] and np.allclose(logp, [math.log(0.2)])
    # the same token twice: nothing is left of it
    assert TR.verify_one(z, [0, 0], tree, 2, 1.0, [0.51, 0.0], 0.0)[:2] == ([1], [0])
    # greedy: the child that is the argmax, wherever it stands
    assert TR.verify_one(z, [1, 0], tree, 2, 0.0, [0.0, 0.9], 0.9)[:2] == ([0, 2], [0, 2])
    # a chain is target_reference's
    rng = np.random.default_rng(9652)
    for _ in range(50):
        z = rng.standard_normal((4, 5)) * 2
        x, u = rng.integers(0, 5, 3), rng.random(4)
        want = R.verify_one(z, x, 3, [False] * 3, None, 0.8, u, u[-1])
        got = TR.verify_one(z, x, [0, 1, 2], 3, 0.8, u, u[-1])
        assert got[0] == want[0] and np.allclose(got[2], want[1])


def test_reference_commits_the_targets_distribution():
    """Over a grid of random numbers the first committed token's frequencies
    are the target's probabilities, for a root with two children."""
    p = np.array([0.4, 0.3, 0.2, 0.1])
    z = np.log(np.stack([p, p, p]))
    grid = (np.arange(24) + 0.5) / 24
    hits = np.zeros(4)
    for u1 in grid:
        for u2 in grid:
            for ud in grid:
                hits[TR.verify_one(z, [2, 0], [0, 0], 2, 1.0, [u1, u2], ud)[0][0]] += 1
    # 24 steps: each of the three edges is off by at most half a step
    assert np.abs(hits / 24**3 - p).max() < 1.5 / 24


def test_reference_kept_cells():
    kc, vc = np.zeros((1, 2, 1, 16, 1)), np.zeros((1, 2, 1, 1, 16))
    kc[0, 0, 0, :, 0] = vc[0, 0, 0, 0] = np.arange(16)
    kc[0, 1, 0, :, 0] = vc[0, 1, 0, 0] = np.arange(100, 116)
    k, v = TR.keep(kc, vc, np.array([[0, 1]]), [15], [[0, 2, 4]], [2], 16)
    # cells 14 (the root), 15 <- 16, 16 <- 18
    for x in (k[0, :, 0, :, 0], v[0, :, 0, 0]):
        assert x[0, 14] == 14 and x[0, 15] == 100 and x[1, 0] == 102 and x[1, 1] == 101
