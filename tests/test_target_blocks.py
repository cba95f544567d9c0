"""The checks that stand between a verify step's device inputs and its
addresses (pld_block.h), compiled for the host under the address and
undefined-behaviour sanitizers: every combination of lengths, draft lengths,
table widths and page ids at the edges, with the arrays exactly as long as
the call says (no GPU needed)."""

from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <memory>

#include "pld_block.h"

static int fails = 0;
#define CHECK(x) do { if (!(x)) { printf("%d: %s\n", __LINE__, #x); ++fails; } } while (0)

int main()
{
    const int32_t lens[] = {INT_MIN, -1, 0, 1, 2, 15, 16, 17, 99, 100, 101, INT_MAX};
    const int32_t drafts[] = {INT_MIN, -2, -1, 0, 1, 6, 7, 8, 99, INT_MAX};
    for (int32_t max_len : {1, 16, 100, INT_MAX})
        for (int32_t rows : {1, 8})
            for (int32_t len : lens)
                for (int32_t d : drafts) {
                    std::unique_ptr<int32_t[]> l(new int32_t[1]{len}), k(new int32_t[1]{d});
                    pld::BlockArgs a{};
                    a.lengths = l.get();
                    a.draft_len = k.get();
                    a.rows = rows;
                    a.max_len = max_len;
                    int32_t got_len;
                    uint32_t err;
                    const int32_t n = pld::block_rows(a, 0, got_len, err);
                    const bool bad = len < 0 || d < -1 || d >= rows;
                    const bool none = len == 0 || d == -1;
                    const bool big = !bad && !none && (long long)len + d > max_len;
                    CHECK(got_len == len);
                    CHECK(n == (bad || big ? -1 : none ? 0 : d + 1));
                    CHECK((err != 0) == (n < 0));
                    CHECK(((err & pld::kErrLenCapacity) != 0) == big);
                    CHECK(((err & pld::kErrLenNegative) != 0) == (len < 0));
                    CHECK(((err & pld::kErrBlock) != 0) == (d < -1 || d >= rows));
                    // a row that exists stands inside [0, max_len)
                    CHECK(n <= 0 || (len >= 1 && (long long)len - 1 + n - 1 < max_len));
                }
    const int32_t ids[] = {0, 4, 5, -1, INT_MIN, INT_MAX, 3};
    for (int shift : {4, 5, 6, 7, 8})
        for (int64_t stride : {1, 2, 7})
            for (int64_t pages : {1, 5, INT_MAX}) {
                const int batch = 3;
                std::unique_ptr<int32_t[]> t(new int32_t[batch * stride]);
                for (int64_t i = 0; i < batch * stride; ++i)
                    t[i] = ids[i % 7];
                pld::BlockArgs a{};
                a.table = t.get();
                a.table_stride = stride;
                a.n_pages = pages;
                a.page_shift = shift;
                for (int b = 0; b < batch; ++b)
                    for (int64_t p : {(int64_t)0, (int64_t)15, (int64_t)16, (stride << shift) - 1,
                                      stride << shift, (int64_t)INT_MAX}) {
                        const int64_t i = p >> shift;
                        const int32_t got = pld::page_of(a, b, (int32_t)p);
                        const int32_t id = i < stride ? t[b * stride + i] : -1;
                        CHECK(got == (id >= 0 && id < pages ? id : -1));
                    }
            }
    return fails != 0;
}
"""


def test_blocks_and_pages_under_sanitizers(tmp_path):
    src, exe = tmp_path / "blocks.cpp", tmp_path / "blocks"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-Wall", "-Wextra", "-Werror",
                    "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "prompt_lookup_gram_amd", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    # leaks are not at issue, and the leak checker needs ptrace
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120,
                       env={**os.environ,
                            "ASAN_OPTIONS": "detect_leaks=0:verify_asan_link_order=0"})
    assert r.returncode == 0, r.stdout + r.stderr
