"""The tree's calls (HIP, gfx950) where element offsets pass 2^31: pages far into
a cache, logits rows far apart. (tests/test_kv_keep_gpu.py has pld_kv_keep's.)"""

from __future__ import annotations

import numpy as np
import pytest

import tree_reference as TR
from prompt_lookup_gram_amd import binding as B
from test_attend_gpu import gpu  # noqa: F401
from test_tree_attend_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,pages,far", [(64, 40000, [39999, 33000, 32769]),
                                            (16, 160000, [159999, 131073, 140001, 150002, 159998,
                                                          131080, 155000, 133333, 158001, 144444,
                                                          159000])])
def test_attention_and_append_of_far_pages(page, pages, far):
    """8 heads of 128 dims: 2.6e9 elements a cache. 8, 24 and 48 query rows a kv
    head."""
    import torch
    hk, dim = 8, 128
    kc = torch.empty((pages, hk, page, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((pages, hk, dim, page), dtype=torch.bfloat16, device="cuda")
    for rows, hq in ((4, 16), (12, 16), (12, 32)):
        c = Case([150], [rows - 1], rows, hq=hq, hk=hk, dim=dim, page=page, seed=31)
        assert c.table.shape[1] <= len(far)
        table = np.array([far[:c.table.shape[1]]], np.int32)
        for i, p in enumerate(table[0]):
            kc[int(p)] = c.kc[int(c.table[0, i])]
            vc[int(p)] = c.vc[int(c.table[0, i])]
        ctx = c.context()
        try:
            out, lse = c.outputs()
            keep = c.kc, c.vc, c.pages
            c.kc, c.vc, c.pages = kc, vc, pages
            c.call(ctx, out, lse, table=table)
            assert B.pld_sync(ctx) == B.PLD_OK
            c.kc, c.vc, c.pages = keep
            c.compare(out, lse)
            # the writer reaches the same cells
            x = torch.full((rows, hk * dim), 3.0, dtype=torch.bfloat16, device="cuda")
            B.pld_kv_append_tree(ctx, None, 0, x, x, x.shape[1], rows, c.ln, c.dl, c.par, 1, c.tab,
                                 c.tab.shape[1], kc, vc, pages)
            assert B.pld_sync(ctx) == B.PLD_OK
            for at in (149, 149 + rows - 1):
                assert bool((kc[far[at // page], :, at % page] == 3).all())
                assert bool((vc[far[at // page], :, :, at % page] == 3).all())
        finally:
            B.pld_destroy(ctx)


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_logits_rows_far_apart(dt):
    import torch
    batch, rows, vocab, stride = 64, 40, 1000, 900_001
    rng = np.random.default_rng(9704)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(32)
    dtype = {"f32": torch.float32, "f16": torch.float16}[dt]
    near = (torch.randn((batch * rows, vocab), generator=gen, device="cuda") * 2).to(dtype)
    far = torch.empty((batch * rows, stride), dtype=dtype, device="cuda")
    far[:, :vocab] = near
    i32 = dict(dtype=torch.int32, device="cuda")
    par = torch.tensor([TR.random_tree(rng, rows - 1) for _ in range(batch)], **i32)
    draft = torch.randint(0, vocab, (batch, rows - 1), generator=gen, **i32)
    # (every row's likeliest token is a child of its node, where it has one)
    top = near.view(batch, rows, vocab).argmax(-1)
    draft[:, ::2] = top.gather(1, par.long())[:, ::2].to(torch.int32)
    dlen = torch.full((batch,), rows - 1, **i32)
    temperature = torch.full((batch,), 0.3, device="cuda")
    temperature[::4] = 0.0
    u = torch.rand((batch, rows), generator=gen, device="cuda")
    p = B.pld_target_params_default()
    p.max_batch, p.max_rows, p.vocab = batch, rows, vocab
    ctx = B.pld_create_target(p)
    got = []
    try:
        for z, step in ((near, vocab), (far, stride)):
            tok, path = (torch.empty((batch, rows), **i32) for _ in range(2))
            acc, cnt = (torch.empty(batch, **i32) for _ in range(2))
            logp = torch.empty((batch, rows), device="cuda")
            B.pld_verify_tree(ctx, z, step, rows, draft, dlen, par, temperature, u, batch, tok, path,
                              acc, cnt, logp)
            assert B.pld_sync(ctx) == B.PLD_OK
            got.append((tok, path, acc, cnt, logp))
        assert int(got[0][2].sum()) > 0
        for a, b in zip(*got):
            assert torch.equal(a, b)
    finally:
        B.pld_destroy(ctx)
