"""The whole verify step as a decode loop runs it, on one history store: draft
from the store, the block's keys and values into the paged cache, attention
of the block, verification of the draft against the model's logits, the
committed tokens appended and the next draft made in one launch. Everything
stays on the device; lengths and draft lengths go from call to call as the
calls leave them.

The model is one attention layer with random weights over a small vocabulary,
so that its text repeats itself and lookup drafts are often right. Because a
greedy step commits exactly the model's own greedy tokens, whatever was
drafted, the loop is compared with the same model decoding one token at a time
through the same calls (rows = 1), and that with a plain 64-bit decode."""

from __future__ import annotations

import numpy as np
import pytest

import target_reference as R
from prompt_lookup_gram_amd import binding as B

pytestmark = pytest.mark.gpu

V, HQ, HK, D, PAGE, K_MAX = 40, 4, 2, 64, 16, 7


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.load()
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


class Model:
    """Embedding, one attention layer, output projection."""

    def __init__(self, seed):
        import torch
        gen = torch.Generator().manual_seed(seed)
        dim = 64
        self.emb = torch.randn(V, dim, generator=gen).cuda()
        self.qkv = (torch.randn(dim, (HQ + 2 * HK) * D, generator=gen) / 8).cuda()
        self.out = (torch.randn(HQ * D, V, generator=gen) / 4).cuda()
        self.res = (torch.randn(dim, V, generator=gen) / 4).cuda()

    def project(self, tokens):
        return (self.emb[tokens.long()] @ self.qkv).bfloat16()

    def logits(self, tokens, attended):
        return attended.float() @ self.out + self.emb[tokens.long()] @ self.res


class Loop:
    """The step's buffers for a batch."""

    def __init__(self, model, batch, k_max, max_len, temperature, seed):
        import torch
        self.m, self.b, self.k, self.rows = model, batch, k_max, k_max + 1
        p = B.pld_target_params_default()
        p.max_batch, p.max_rows, p.max_len = batch, max(self.rows, max_len), max_len + 64
        p.q_heads, p.kv_heads, p.head_dim, p.page_tokens, p.vocab = HQ, HK, D, PAGE, V
        p.rope.rot_dim = 32
        self.target = B.pld_create_target(p)
        self.store = B.pld_create(batch, max_len + 64, own_store=True)
        per = -(-(max_len + 64) // PAGE)
        ids = torch.randperm(batch * per, generator=torch.Generator().manual_seed(seed))
        self.table = ids.to(torch.int32).view(batch, per).cuda().contiguous()
        self.pages = batch * per
        self.kc = torch.full((self.pages, HK, PAGE, D), float("nan"), dtype=torch.bfloat16,
                             device="cuda")
        self.vc = torch.full((self.pages, HK, D, PAGE), float("nan"), dtype=torch.bfloat16,
                             device="cuda")
        self.temp = torch.full((batch,), temperature, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.tokens = torch.empty((batch, self.rows), **i32)
        self.accepted, self.counts = torch.empty(batch, **i32), torch.empty(batch, **i32)
        self.draft = torch.full((batch, max(1, k_max)), -1, **i32)
        self.dlen, self.match = torch.zeros(batch, **i32), torch.zeros(batch, **i32)
        self.hist, self.lengths = B.pld_histories(self.store)

    def close(self):
        B.pld_destroy(self.target)
        B.pld_destroy(self.store)

    def forward(self, block, rows, lengths, dlen):
        """One pass of the model over a block: its logits."""
        qkv = self.m.project(block).view(self.b * rows, -1)
        import torch
        w = qkv.shape[1]
        q = torch.empty((self.b * rows, HQ * D), dtype=torch.bfloat16, device="cuda")
        B.pld_kv_append(self.target, qkv, w, qkv[:, HQ * D:], qkv[:, (HQ + HK) * D:], w, rows,
                        lengths, dlen, self.b, self.table, self.table.shape[1], self.kc, self.vc,
                        self.pages, None, None, q)
        o = torch.zeros_like(q)
        B.pld_attend(self.target, q, HQ * D, rows, lengths, dlen, 0, self.b, self.table,
                     self.table.shape[1], self.kc, self.vc, self.pages, None, None, 0.0, 0, o)
        return self.m.logits(block, o.view(self.b, rows, -1)).contiguous()

    def start(self, prompts):
        """Prompts into the store and, but for their last token, the cache."""
        import torch
        width = max(len(p) for p in prompts)
        tok = np.zeros((self.b, width), np.int32)
        for i, p in enumerate(prompts):
            tok[i, :len(p)] = p
        tok = torch.from_numpy(tok).cuda()
        cnt = torch.tensor([len(p) for p in prompts], dtype=torch.int32).cuda()
        B.pld_append(self.store, tok, width, cnt, self.b)
        one = torch.ones(self.b, dtype=torch.int32, device="cuda")
        self.forward(tok, width, one, cnt - 2)   # rows 0 .. n - 2, from position 0 on
        self.last = torch.tensor([p[-1] for p in prompts], dtype=torch.int32).cuda()

    def step(self, uniform):
        """Verify the current draft, commit, draft again."""
        import torch
        block = torch.cat((self.last[:, None], self.draft[:, :self.k].clamp(min=0)), 1)
        logits = self.forward(block, self.rows, self.lengths, self.dlen)
        B.pld_verify(self.target, logits, V, self.rows, self.draft if self.k else None, self.dlen,
                     None, None, 0, self.temp, uniform, self.b, self.tokens, self.accepted,
                     self.counts)
        if self.k:
            B.pld_append_draft_store(self.store, self.tokens, self.rows, self.counts, self.b, 1, 8,
                                     self.k, self.draft, self.dlen, self.match)
        else:
            B.pld_append(self.store, self.tokens, self.rows, self.counts, self.b)
        self.last = self.tokens.gather(1, (self.counts - 1).long()[:, None])[:, 0]
        assert B.pld_sync(self.target) == B.PLD_OK and B.pld_sync(self.store) == B.PLD_OK
        return self.tokens.cpu().numpy(), self.counts.cpu().numpy()


def generate(model, prompts, k_max, steps, temperature, seed=0, uniforms=None):
    import torch
    batch = len(prompts)
    loop = Loop(model, batch, k_max, max(len(p) for p in prompts) + steps * (k_max + 1),
                temperature, seed)
    gen = torch.Generator().manual_seed(seed)
    text, taken = [list(p) for p in prompts], 0
    try:
        loop.start(prompts)
        for s in range(steps):
            u = torch.rand((batch, loop.rows), generator=gen).cuda()
            tok, cnt = loop.step(u)
            for b in range(batch):
                text[b] += tok[b, :cnt[b]].tolist()
                taken += int(cnt[b]) - 1
    finally:
        loop.close()
    return text, taken


def prompts_for(seed, batch):
    rng = np.random.default_rng([9401, seed])
    out = []
    for b in range(batch):
        phrase = rng.integers(0, V, 9)
        out.append(np.concatenate([phrase, rng.integers(0, V, 5 + b), phrase]).tolist())
    return out


def test_drafted_greedy_decode_equals_plain_greedy_decode():
    model, prompts = Model(3), prompts_for(0, 5)
    plain, _ = generate(model, prompts, 0, 60, 0.0)
    fast, taken = generate(model, prompts, K_MAX, 40, 0.0, seed=1)
    for a, b in zip(plain, fast):
        n = min(len(a), len(b))
        assert n > 60 and a[:n] == b[:n]
    assert taken > 60, "the drafts should be taken often"


def test_plain_greedy_decode_is_the_models():
    """The one-row loop against a 64-bit decode of the same model. The
    reference takes the loop's own text as its history, so that one step's
    rounding cannot part the two; a step whose two best logits lie within the
    bf16 cache's rounding may choose either."""
    model, prompts = Model(4), prompts_for(1, 3)
    text, _ = generate(model, prompts, 0, 25, 0.0)
    freq = R.rope_frequencies(32)
    qkv = model.qkv.double().cpu().numpy()
    emb = model.emb.double().cpu().numpy()
    out, res = model.out.double().cpu().numpy(), model.res.double().cpu().numpy()
    sure = 0
    for b, p in enumerate(prompts):
        x = emb[text[b]] @ qkv
        k = np.stack([R.rotate(x[i, HQ * D:(HQ + HK) * D].reshape(HK, D), i, freq, 32, False,
                               1.0)[0] for i in range(len(x))])
        v = x[:, (HQ + HK) * D:].reshape(-1, HK, D)
        for i in range(len(p) - 1, len(text[b]) - 1):
            q = R.rotate(x[i, :HQ * D].reshape(HQ, D), i, freq, 32, False, 1.0)[0]
            o = []
            for h in range(HQ):
                s = k[:i + 1, h // 2] @ q[h] / np.sqrt(D)
                e = np.exp(s - s.max())
                o.append(e / e.sum() @ v[:i + 1, h // 2])
            logits = np.concatenate(o) @ out + emb[text[b][i]] @ res
            top = np.sort(logits)[::-1]
            best = int(np.argmax(logits))
            if top[0] - top[1] > 0.25:
                assert text[b][i + 1] == best
                sure += 1
            else:
                assert logits[text[b][i + 1]] > top[0] - 0.25
    assert sure > 40


def test_sampled_decode_runs_with_ragged_drafts():
    model, prompts = Model(5), prompts_for(2, 6)
    text, taken = generate(model, prompts, K_MAX, 30, 0.5)
    assert all(len(t) >= len(p) + 30 for t, p in zip(text, prompts))
    assert all(0 <= x < V for t in text for x in t) and taken > 0


def test_fused_block_is_verified_with_its_sources():
    """pld_draft_fuse_batch's block and source mask as pld_verify takes them:
    lookup positions are point masses, the drafter's have q."""
    import torch
    rng = np.random.default_rng(9402)
    batch, head, long = 4, 3, 6
    hist = [np.tile(rng.integers(0, V, 6), 6).astype(np.int32) for _ in range(batch)]
    db = B.DeviceBatch(hist)
    params = B.pld_fuse_params_default()
    params.head, params.positions_long, params.entry_steps = head, long, 0
    params.replace_min, params.agree_min, params.agree_tokens = 64, 64, 1
    ctx = B.pld_create(batch, 64)
    p = B.pld_target_params_default()
    p.max_batch, p.max_rows, p.vocab = batch, long + 1, V
    target = B.pld_create_target(p)
    i32 = dict(dtype=torch.int32, device="cuda")
    try:
        d, l, m = torch.empty((batch, 8), **i32), torch.empty(batch, **i32), torch.empty(batch, **i32)
        drafter = torch.from_numpy(rng.integers(0, V, (batch, head)).astype(np.int32)).cuda()
        acc, state = torch.zeros(batch, **i32), torch.zeros((batch, 4), **i32)
        block, pos = torch.empty((batch, long), **i32), torch.empty(batch, **i32)
        src = torch.empty(batch, dtype=torch.int64, device="cuda")
        B.pld_draft_fuse_batch(ctx, db.rows, db.lengths, batch, 4, 12, 8, d, l, m, params, drafter,
                               acc, state, block, pos, src)
        z = torch.from_numpy(rng.standard_normal((batch, long + 1, V))).float().cuda()
        q = torch.softmax(torch.from_numpy(rng.standard_normal((batch, head, V))).float(), -1).cuda()
        u = torch.from_numpy(rng.random((batch, long + 1)).astype(np.float32)).cuda() * 0.05
        tok, ac, cn = torch.empty((batch, long + 1), **i32), torch.empty(batch, **i32), torch.empty(
            batch, **i32)
        B.pld_verify(target, z, V, long + 1, block, pos, src, q, head, None, u, batch, tok, ac, cn)
        assert B.pld_sync(ctx) == B.PLD_OK and B.pld_sync(target) == B.PLD_OK
        zs, qs, us = z.double().cpu().numpy(), q.double().cpu().numpy(), u.cpu().numpy()
        for b in range(batch):
            n, mask = int(pos[b]), int(src[b])
            assert n == long and mask == 0b111000
            want, _ = R.verify_one(zs[b], block[b].tolist(), n, [t < head for t in range(long)],
                                   qs[b], 1.0, us[b], us[b, -1])
            assert tok[b, :len(want)].tolist() == want and int(cn[b]) == len(want)
            assert int(ac[b]) == len(want) - 1
        # the accepted counts are what the next fusion step takes
        B.pld_fuse(ctx, params, d, 8, l, m, drafter, ac, state, batch, block, pos, src)
        assert B.pld_sync(ctx) == B.PLD_OK
    finally:
        B.pld_destroy(ctx)
        B.pld_destroy(target)


def test_the_step_in_a_graph():
    """Append, attention, verification and the next draft captured once and
    replayed, against the same calls made eagerly."""
    import torch
    model, prompts = Model(6), prompts_for(3, 4)

    def make():
        loop = Loop(model, 4, K_MAX, 300, 0.7, 2)
        loop.start(prompts)
        return loop
    uniform = torch.rand((12, 4, K_MAX + 1), generator=torch.Generator().manual_seed(8)).cuda()
    eager, graphed = make(), make()
    try:
        want = []
        for s in range(12):
            want.append([x.copy() for x in eager.step(uniform[s])])
        u = torch.empty_like(uniform[0])
        last = graphed.last.clone()

        def body():
            block = torch.cat((last[:, None], graphed.draft.clamp(min=0)), 1)
            logits = graphed.forward(block, graphed.rows, graphed.lengths, graphed.dlen)
            B.pld_verify(graphed.target, logits, V, graphed.rows, graphed.draft, graphed.dlen,
                         None, None, 0, graphed.temp, u, 4, graphed.tokens, graphed.accepted,
                         graphed.counts)
            B.pld_append_draft_store(graphed.store, graphed.tokens, graphed.rows, graphed.counts,
                                     4, 1, 8, K_MAX, graphed.draft, graphed.dlen, graphed.match)
            last.copy_(graphed.tokens.gather(1, (graphed.counts - 1).long()[:, None])[:, 0])
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mm(torch.ones(8, 8, device="cuda"), torch.ones(8, 8, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            body()
        for s in range(12):
            u.copy_(uniform[s])
            graph.replay()
            torch.cuda.synchronize()
            assert np.array_equal(graphed.counts.cpu().numpy(), want[s][1]), s
            assert np.array_equal(graphed.tokens.cpu().numpy(), want[s][0]), s
        assert B.pld_sync(graphed.target) == B.PLD_OK and B.pld_sync(graphed.store) == B.PLD_OK
    finally:
        eager.close()
        graphed.close()
