"""pld_kv_append (HIP, gfx950) against the 64-bit reference: rotary layouts
and scalings, part of a head, ragged and empty blocks, pages that end inside
a block, strided inputs, 8-bit cells, and what must stay untouched.

Tolerances. A rotated value is computed in 32 bits from sums of two products:
cos and sin carry an absolute error of at most 2^-21 (the reduced angle is
rounded to 24 bits of pi, 2^-23; the functions are good to 2 units, 2^-22),
the products and their sum three roundings of 2^-24, the factors (magnitude,
1 / scale) two more: below 2^-20 of (|x| + |y|) * magnitude in all. Storing
rounds once: half a step, finfo.eps / 2 of the value, or half the smallest
subnormal step. V is stored as it is (16 bits), or rounded once (8 bits; the
division by the scale adds 2^-24)."""

from __future__ import annotations

import numpy as np
import pytest

import target_reference as R
from prompt_lookup_gram_amd import binding as B

pytestmark = pytest.mark.gpu

SCALINGS = {"plain": 0, "linear": 1, "banded": 2}
ROPE = dict(base=10000.0, factor=8.0, original_len=4096, beta_fast=32.0, beta_slow=1.0)
# half the smallest subnormal step
TINY = {"bf16": 2.0**-134, "f16": 2.0**-25, "e4m3": 2.0**-10}
LARGEST = {"bf16": np.inf, "f16": np.inf, "e4m3": 448.0}


def dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[name]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.load()
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def table_for(rng, lengths, dlen, page, spare=3):
    """A table of distinct random pages: (table, pages)."""
    need = [max(1, -(-max(1, n + max(0, d)) // page)) for n, d in zip(lengths, dlen)]
    ids = rng.permutation(sum(need) + spare)
    table = np.zeros((len(need), max(need)), np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table, sum(need) + spare


def context(batch, rows, max_len, hq, hk, dim, dt, cache, page, rot=0, interleaved=False,
            scaling="plain", magnitude=1.0, rope=None):
    p = B.pld_target_params_default()
    p.max_batch, p.max_rows, p.max_len = batch, rows, max_len
    p.q_heads, p.kv_heads, p.head_dim, p.page_tokens = hq, hk, dim, page
    p.dtype, p.cache_dtype = B.PLD_TYPES[dtype(dt)], B.PLD_TYPES[dtype(cache)]
    p.rope.rot_dim, p.rope.interleaved = rot, int(interleaved)
    p.rope.scaling, p.rope.magnitude = SCALINGS[scaling], magnitude
    for k, v in (rope or ROPE).items():
        setattr(p.rope, k, v)
    return B.pld_create_target(p)


def stored(name, ref, size, extra):
    """Bounds on a stored value: |got - ref| <= this."""
    import torch
    half = float(torch.finfo(dtype(name)).eps) / 2
    return extra * size + half * (np.abs(ref) + extra * size) + TINY[name]


def check(lengths, dlen, rows, hq=4, hk=2, dim=64, dt="bf16", cache=None, page=16, rot=None,
          interleaved=False, scaling="plain", magnitude=1.0, seed=0, pad=0, scales=False,
          in_place=False, with_q=True, offset=0):
    import torch
    cache = cache or dt
    rot = dim if rot is None else rot
    rng = np.random.default_rng([9101, seed])
    b = len(lengths)
    table, pages = table_for(rng, lengths, dlen, page)
    wq, wk = hq * dim, hk * dim
    width = (0 if in_place else wq) + 2 * wk + pad
    raw = torch.from_numpy(rng.standard_normal(b * rows * width + offset) * 2).to(dtype(dt))
    raw = raw.cuda()
    qkv = raw[offset:].view(b * rows, width)
    if in_place:
        q = torch.from_numpy(rng.standard_normal((b * rows, wq)) * 2).to(dtype(dt)).cuda()
        k, v = qkv[:, :wk], qkv[:, wk:2 * wk]
    else:
        q, k, v = qkv[:, :wq], qkv[:, wq:wq + wk], qkv[:, wq + wk:wq + 2 * wk]
    q0, k0, v0 = [x.double().cpu().numpy() for x in (q, k, v)]
    ctab = torch.from_numpy(rng.standard_normal((2, pages * wk * page))).float()
    kc = ctab[0].to(dtype(cache)).view(pages, hk, page, dim).cuda()
    vc = ctab[1].to(dtype(cache)).view(pages, hk, dim, page).cuda()
    kc0, vc0 = kc.double().cpu().numpy(), vc.double().cpu().numpy()
    out_q = q if in_place else torch.full((b * rows, wq), 7.0, dtype=dtype(dt), device="cuda")
    oq0 = out_q.double().cpu().numpy()
    ks = torch.tensor(rng.uniform(0.01, 2.0, hk), dtype=torch.float32).cuda() if scales else None
    vs = torch.tensor(rng.uniform(0.01, 2.0, hk), dtype=torch.float32).cuda() if scales else None
    max_len = max(1, max(n + max(d, 0) for n, d in zip(lengths, dlen)))
    ctx = context(b, rows, max_len, hq, hk, dim, dt, cache, page, rot, interleaved, scaling,
                  magnitude)
    try:
        B.pld_kv_append(ctx, q if with_q else None, wq if in_place else width, k, v, width, rows,
                        torch.tensor(lengths, dtype=torch.int32).cuda(),
                        torch.tensor(dlen, dtype=torch.int32).cuda(), b,
                        torch.from_numpy(table).cuda(), table.shape[1], kc, vc, pages, ks, vs,
                        out_q if with_q else None)
        assert B.pld_sync(ctx) == B.PLD_OK, B.pld_last_error()
    finally:
        B.pld_destroy(ctx)
    gq, gk, gv = [x.double().cpu().numpy() for x in (out_q, kc, vc)]
    freq = R.rope_frequencies(rot, scaling, **ROPE)
    want_q, want_k, want_v = oq0.copy(), kc0.copy(), vc0.copy()
    tol_q, tol_k, tol_v = np.zeros_like(gq), np.zeros_like(gk), np.zeros_like(gv)
    for i in range(b):
        for t in range(R.block_rows(lengths[i], dlen[i])):
            r, p = i * rows + t, lengths[i] - 1 + t
            y, size = R.rotate(q0[r].reshape(hq, dim), p, freq, rot, interleaved, magnitude)
            if with_q:
                want_q[r] = y.reshape(-1)
                tol_q[r] = stored(dt, y, size, 2.0**-20).reshape(-1)
            y, size = R.rotate(k0[r].reshape(hk, dim), p, freq, rot, interleaved, magnitude)
            div = ks.double().cpu().numpy()[:, None] if scales else np.ones((hk, 1))
            y, size = y / div, (size + np.abs(y) * 2.0**-4) / div
            top = LARGEST[cache]
            want_k[table[i, p // page], :, p % page] = np.clip(y, -top, top)
            tol_k[table[i, p // page], :, p % page] = stored(cache, y, size, 2.0**-20)
            div = vs.double().cpu().numpy()[:, None] if scales else np.ones((hk, 1))
            y = v0[r].reshape(hk, dim) / div
            want_v[table[i, p // page], :, :, p % page] = np.clip(y, -top, top)
            if cache != dt:
                tol_v[table[i, p // page], :, :, p % page] = stored(cache, y, np.abs(y), 2.0**-24)
    for name, got, want, tol in (("q", gq, want_q, tol_q), ("k", gk, want_k, tol_k),
                                 ("v", gv, want_v, tol_v)):
        off = np.abs(got - want) - tol
        assert not np.isnan(off).any() and off.max() <= 0, (
            name, float(off.max()), np.unravel_index(np.argmax(off), off.shape))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_dims_and_layouts(dt, dim, interleaved):
    check([1, 40, 17], [5, 0, 3], 6, dim=dim, dt=dt, interleaved=interleaved, seed=dim)


@pytest.mark.parametrize("rot", [0, 2, 6, 32, 62, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_the_head(rot, interleaved):
    check([30, 5], [9, 2], 10, dim=128, rot=rot, interleaved=interleaved, seed=rot)


@pytest.mark.parametrize("scaling", sorted(SCALINGS))
@pytest.mark.parametrize("start", [1, 262100, 2097000])
def test_far_positions(scaling, start):
    # 2^21 positions: the angle's fraction keeps 52 - 21 bits in the product
    check([start], [30], 31, hq=2, hk=1, dim=64, page=256, scaling=scaling, magnitude=1.25,
          seed=start)


@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 8), (12, 4), (16, 1), (5, 5)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_heads_and_pages(hq, hk, page):
    check([250, 15, 16, 17, 63], [20, 1, 0, 15, 2], 21, hq=hq, hk=hk, page=page, seed=hq * page)


def test_empty_and_idle_requests_leave_everything():
    check([0, 5, 0, 9], [3, -1, -1, 2], 4)
    check([0, 5], [3, -1], 4)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("scales", [False, True])
def test_eight_bit_cells(dt, scales):
    check([33, 5], [15, 7], 16, dim=128, dt=dt, cache="e4m3", page=32, scales=scales, seed=4)


def test_odd_strides_and_offsets():
    check([33, 5], [15, 7], 16, pad=3, offset=1, seed=5)
    check([33, 5], [15, 7], 16, dim=96, pad=8, offset=5, seed=6)
    check([33, 5], [15, 7], 16, pad=8, offset=8, seed=7)


def test_in_place_and_without_q():
    check([33, 5], [15, 7], 16, in_place=True, seed=8)
    check([33, 5], [15, 7], 16, with_q=False, seed=9)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_prompt_in_one_call(cache):
    # many rows, starting inside a page; the last page ends inside the block
    check([10, 1, 64], [499, 63, 300], 500, hq=2, hk=2, page=64, cache=cache, seed=10)


def test_rounding_saturates_and_keeps_special_values():
    import torch
    x = torch.zeros((1, 128), dtype=torch.bfloat16)
    x[0, :8] = torch.tensor([500.0, -1e30, float("inf"), -float("inf"), float("nan"), 1e-9,
                             -448.0, 0.0175])
    k = x.cuda()
    kc = torch.zeros((1, 1, 16, 128), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc = torch.zeros((1, 1, 128, 16), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    ctx = context(1, 1, 16, 1, 1, 128, "bf16", "e4m3", 16)
    try:
        B.pld_kv_append(ctx, None, 0, k, k, 128, 1, one, one * 0, 1, one * 0, 1, kc, vc, 1)
        assert B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)
    want = torch.tensor([448.0, -448.0, 448.0, -448.0, float("nan"), 0.0, -448.0, 0.017578125])
    for got in (kc[0, 0, 0, :8].float().cpu(), vc[0, 0, :8, 0].float().cpu()):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


def test_bad_inputs_are_reported_and_leave_the_cache():
    import torch
    rng = np.random.default_rng(11)
    b, rows, hq, hk, dim, page = 6, 4, 2, 1, 64, 16
    lengths, dlen = [-1, 20, 62, 20, 20, 20], [1, 4, 3, -2, 2, 2]
    table = np.arange(b * 4, dtype=np.int32).reshape(b, 4)
    table[4, 1] = b * 4        # a page past the cache, under rows 0..2
    table[5, 1] = -7
    q = torch.randn((b * rows, (hq + 2) * dim)).bfloat16().cuda()
    args = lambda: (q, q.shape[1], q[:, hq * dim:], q[:, (hq + 1) * dim:], q.shape[1], rows)
    ctx = context(b, rows, 64, hq, hk, dim, "bf16", "bf16", page)
    try:
        for i in range(b):
            kc = torch.ones((b * 4, hk, page, dim), dtype=torch.bfloat16, device="cuda")
            vc = torch.ones((b * 4, hk, dim, page), dtype=torch.bfloat16, device="cuda")
            oq = torch.ones((b * rows, hq * dim), dtype=torch.bfloat16, device="cuda")
            ln, dl = [0] * b, [0] * b
            ln[i], dl[i] = lengths[i], dlen[i]
            B.pld_kv_append(ctx, *args(), torch.tensor(ln, dtype=torch.int32).cuda(),
                            torch.tensor(dl, dtype=torch.int32).cuda(), b,
                            torch.from_numpy(table).cuda(), 4, kc, vc, b * 4, None, None, oq)
            want = B.PLD_ECAPACITY if i == 2 else B.PLD_EINVAL
            assert B.pld_sync(ctx) == want, i
            assert bool((kc == 1).all()) and bool((vc == 1).all())
            # rows of a request with a bad page still rotate q
            assert bool((oq == 1).all()) == (i < 4)
            assert B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)


def test_position_past_the_table_is_a_bad_page():
    import torch
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    x = torch.randn((1, 192)).bfloat16().cuda()
    kc = torch.ones((4, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.ones((4, 1, 64, 16), dtype=torch.bfloat16, device="cuda")
    ctx = context(1, 1, 64, 1, 1, 64, "bf16", "bf16", 16)
    try:
        B.pld_kv_append(ctx, None, 0, x[:, 64:], x[:, 128:], 192, 1, one * 33, one * 0, 1,
                        torch.zeros(2, dtype=torch.int32, device="cuda"), 2, kc, vc, 4)
        assert B.pld_sync(ctx) == B.PLD_EINVAL and "page" in B.pld_last_error()
        assert bool((kc == 1).all()) and bool((vc == 1).all())
    finally:
        B.pld_destroy(ctx)


def test_refusals_on_a_context():
    import torch
    x = torch.randn((4, 192)).bfloat16().cuda()
    i4 = torch.ones(4, dtype=torch.int32, device="cuda")
    kc = torch.ones((4, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    ctx = context(2, 2, 64, 1, 1, 64, "bf16", "bf16", 16)
    good = dict(q=x, q_stride=192, k=x[:, 64:], v=x[:, 128:], kv_stride=192, rows=2, lengths=i4,
                draft_len=i4, batch=2, page_table=i4, table_stride=2, k_cache=kc, v_cache=kc,
                n_pages=4, out_q=torch.empty_like(x[:, :64].contiguous()))
    try:
        B.pld_kv_append(ctx, **{**good, "batch": 0})
        for field, value in [("rows", 0), ("rows", 3), ("batch", -1), ("batch", 3),
                             ("q_stride", 63), ("kv_stride", 63), ("table_stride", 0),
                             ("n_pages", -1), ("n_pages", 2**31), ("k", None), ("v", None),
                             ("q", None), ("out_q", None), ("lengths", None),
                             ("draft_len", None), ("page_table", None), ("k_cache", None),
                             ("v_cache", kc.data_ptr() + 2), ("lengths", i4.data_ptr() + 1)]:
            with pytest.raises(B.PldError) as e:
                B.pld_kv_append(ctx, **{**good, field: value})
            assert e.value.status == B.PLD_EINVAL, field
        with pytest.raises(B.PldError):
            # in place needs dense rows
            B.pld_kv_append(ctx, **{**good, "out_q": x.data_ptr()})
        plain = B.pld_create(2, 64)
        try:
            with pytest.raises(B.PldError, match="target"):
                B.pld_kv_append(plain, **good)
        finally:
            B.pld_destroy(plain)
        with pytest.raises(ValueError):
            B.pld_kv_append(ctx, **{**good, "k": x.float()})
        with pytest.raises(ValueError):
            B.pld_kv_append(ctx, **{**good, "k": x.t()})
        assert B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)
