"""A tree's whole step as a decode loop runs it: two drafters' chains (the
lookup over the history, and the successor counts) stand side by side below
the last token, the tree goes into the paged cache, is attended, verified
against the model's logits, the accepted path's cells are kept, and the
committed tokens go to both drafters. Everything stays on the device.

The model is one attention layer with norms on the heads of its queries and
keys and random weights over a small vocabulary. What the loop commits is held
against a 64-bit decode of the same model over the loop's own text: a cell in
the wrong place, a wrong position or a wrong branch would change its logits by
far more than the bf16 cache's rounding."""

from __future__ import annotations

import numpy as np
import pytest

import target_reference as R
import tree_reference as TR
from prompt_lookup_gram_amd import binding as B
from test_verify_step_gpu import D, HK, HQ, PAGE, V, Model, gpu, prompts_for  # noqa: F401

pytestmark = pytest.mark.gpu

K, EPS, ROT = 5, 1e-6, 32  # tokens of a drafter's chain


class Loop:
    def __init__(self, model, prompts, steps, temperature, layers=2):
        import torch
        self.m, self.b, self.rows, self.layers = model, len(prompts), 2 * K + 1, layers
        long = max(len(p) for p in prompts)
        size = long + steps * (K + 1) + 64
        p = B.pld_target_params_default()
        p.max_batch, p.max_rows, p.max_len = self.b, max(self.rows, long), size
        p.q_heads, p.kv_heads, p.head_dim, p.page_tokens, p.vocab = HQ, HK, D, PAGE, V
        p.rope.rot_dim = ROT
        self.target = B.pld_create_target(p)
        self.lookup = B.pld_create(self.b, size, own_store=True)
        self.counts_ctx = B.pld_create_ngram(self.b, size)
        per = -(-size // PAGE)
        gen = torch.Generator().manual_seed(5)
        self.pages = self.b * per
        self.table = torch.randperm(self.pages, generator=gen).to(torch.int32).view(self.b, per)
        self.table = self.table.cuda().contiguous()
        nan = dict(dtype=torch.bfloat16, device="cuda")
        self.kc = torch.full((layers, self.pages, HK, PAGE, D), float("nan"), **nan)
        self.vc = torch.full((layers, self.pages, HK, D, PAGE), float("nan"), **nan)
        self.nq = torch.linspace(0.6, 1.4, D).cuda()
        self.nk = torch.linspace(1.3, 0.7, D).cuda()
        self.temp = torch.full((self.b,), temperature, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.draft = torch.zeros((self.b, 2 * K), **i32)
        self.parent = torch.zeros((self.b, 2 * K), **i32)
        self.dlen = torch.zeros(self.b, **i32)
        self.one, self.two = (torch.zeros((self.b, K), **i32) for _ in range(2))
        self.n1, self.n2, self.match = (torch.zeros(self.b, **i32) for _ in range(3))
        self.tokens = torch.zeros((self.b, self.rows), **i32)
        self.path = torch.zeros((self.b, self.rows), **i32)
        self.accepted, self.committed = torch.zeros(self.b, **i32), torch.zeros(self.b, **i32)
        _, self.lengths = B.pld_histories(self.lookup)
        self.u = torch.zeros((self.b, self.rows), device="cuda")
        # prompts: into both drafters and, but for the last token, the caches
        tok = np.zeros((self.b, long), np.int32)
        for i, x in enumerate(prompts):
            tok[i, :len(x)] = x
        tok = torch.from_numpy(tok).cuda()
        cnt = torch.tensor([len(x) for x in prompts], **i32)
        B.pld_append(self.lookup, tok, long, cnt, self.b)
        B.pld_append(self.counts_ctx, tok, long, cnt, self.b)
        self.forward(tok, long, torch.ones_like(cnt), cnt - 2, None)
        self.last = torch.tensor([x[-1] for x in prompts], **i32)

    def close(self):
        for ctx in (self.target, self.lookup, self.counts_ctx):
            B.pld_destroy(ctx)

    def forward(self, block, rows, lengths, dlen, parent):
        """A pass of the model (every layer the same) over a block: logits."""
        import torch
        qkv = self.m.project(block).view(self.b * rows, -1)
        w = qkv.shape[1]
        q = torch.empty((self.b * rows, HQ * D), dtype=torch.bfloat16, device="cuda")
        o = torch.zeros_like(q)
        for i in range(self.layers):
            B.pld_kv_append_tree(self.target, qkv, w, qkv[:, HQ * D:], qkv[:, (HQ + HK) * D:], w,
                                 rows, lengths, dlen, parent, self.b, self.table,
                                 self.table.shape[1], self.kc[i], self.vc[i], self.pages, None,
                                 None, self.nq, self.nk, EPS, q)
            B.pld_attend_tree(self.target, q, HQ * D, rows, lengths, dlen, parent, 0, self.b,
                              self.table, self.table.shape[1], self.kc[i], self.vc[i], self.pages,
                              None, None, 0.0, 0, o)
        return self.m.logits(block, o.view(self.b, rows, -1)).contiguous()

    def plant(self):
        """The drafters' chains as one tree: nodes 1..n1, then n1 + 1.. below
        the root again."""
        import torch
        B.pld_draft_ngram(self.counts_ctx, B.pld_ngram_params_default(), self.b, K, self.two,
                          self.n2)
        t = torch.arange(1, 2 * K + 1, dtype=torch.int32, device="cuda")[None, :]
        n1 = self.n1[:, None]
        first = self.one.gather(1, (t - 1).clamp(max=K - 1).long().expand(self.b, -1))
        second = self.two.gather(1, (t - 1 - n1).clamp(0, K - 1).long())
        self.draft.copy_(torch.where(t <= n1, first, second).clamp(min=0))
        self.parent.copy_(torch.where(t == n1 + 1, 0, t - 1))
        self.dlen.copy_(self.n1 + self.n2)

    def step(self):
        import torch
        self.plant()
        block = torch.cat((self.last[:, None], self.draft), 1)
        logits = self.forward(block, self.rows, self.lengths, self.dlen, self.parent)
        B.pld_verify_tree(self.target, logits, V, self.rows, self.draft, self.dlen, self.parent,
                          self.temp, self.u, self.b, self.tokens, self.path, self.accepted,
                          self.committed)
        B.pld_kv_keep(self.target, self.lengths, self.dlen, self.path, self.accepted, self.rows,
                      self.b, self.table, self.table.shape[1], self.kc, self.vc, self.pages,
                      self.layers, self.kc.stride(0), self.vc.stride(0))
        B.pld_append(self.counts_ctx, self.tokens, self.rows, self.committed, self.b)
        B.pld_append_draft_store(self.lookup, self.tokens, self.rows, self.committed, self.b, 1, 8,
                                 K, self.one, self.n1, self.match)
        self.last.copy_(self.tokens.gather(1, (self.committed - 1).long()[:, None])[:, 0])

    def sync(self):
        for ctx in (self.target, self.lookup, self.counts_ctx):
            assert B.pld_sync(ctx) == B.PLD_OK, B.pld_last_error()


def logits_of(loop, text):
    """The model over a text in 64 bits: a row of logits a position."""
    m = loop.m
    freq = R.rope_frequencies(ROT)
    emb = m.emb.double().cpu().numpy()
    x = emb[text] @ m.qkv.double().cpu().numpy()
    nq, nk = loop.nq.double().cpu().numpy(), loop.nk.double().cpu().numpy()
    q, k = [], []
    for i in range(len(text)):
        y = TR.normed(x[i, :HQ * D].reshape(HQ, D), nq, EPS)
        q.append(R.rotate(y, i, freq, ROT, False, 1.0)[0])
        y = TR.normed(x[i, HQ * D:(HQ + HK) * D].reshape(HK, D), nk, EPS)
        k.append(R.rotate(y, i, freq, ROT, False, 1.0)[0])
    q, k = np.stack(q), np.stack(k)
    v = x[:, (HQ + HK) * D:].reshape(-1, HK, D)
    out, res = m.out.double().cpu().numpy(), m.res.double().cpu().numpy()
    rows = []
    for i in range(len(text)):
        o = []
        for h in range(HQ):
            s = k[:i + 1, h // (HQ // HK)] @ q[i, h] / np.sqrt(D)
            e = np.exp(s - s.max())
            o.append(e / e.sum() @ v[:i + 1, h // (HQ // HK)])
        rows.append(np.concatenate(o) @ out + emb[text[i]] @ res)
    return np.stack(rows)


def test_a_greedy_trees_text_is_the_models():
    """Every committed token is the argmax of the model over the text before
    it; where the two best logits lie within the bf16 cache's rounding either
    may be. Both drafters' branches are taken at times."""
    model, prompts = Model(7), prompts_for(4, 5)
    loop = Loop(model, prompts, 40, 0.0)
    text, branches, kept = [list(p) for p in prompts], [0, 0], 0
    try:
        for _ in range(40):
            loop.step()
            loop.sync()
            tok, n = loop.tokens.cpu().numpy(), loop.committed.cpu().numpy()
            path, dlen = loop.path.cpu().numpy(), loop.dlen.cpu().numpy()
            parent = loop.parent.cpu().numpy()
            for b in range(loop.b):
                text[b] += tok[b, :n[b]].tolist()
                way = path[b, :n[b]]
                assert way[0] == 0 and (path[b, n[b]:] == -1).all() and way[-1] <= dlen[b]
                assert all(parent[b, y - 1] == x for x, y in zip(way, way[1:]))
                if len(way) > 1:
                    branches[int(way[1] != 1)] += 1
                    kept += int(way[1] != 1)
    finally:
        sure = 0
        for b, t in enumerate(text):
            z = logits_of(loop, t)
            for i in range(len(prompts[b]) - 1, len(t) - 1):
                top = np.sort(z[i])[::-1]
                if top[0] - top[1] > 0.25:
                    assert t[i + 1] == int(np.argmax(z[i])), (b, i)
                    sure += 1
                else:
                    assert z[i][t[i + 1]] > top[0] - 0.25, (b, i)
        loop.close()
    assert sure > 100 and branches[0] > 10 and kept > 0


def test_the_step_in_a_graph():
    """The whole step captured once and replayed, against the same calls made
    eagerly, with sampling."""
    import torch
    model, prompts = Model(8), prompts_for(5, 4)
    u = torch.rand((10, 4, 2 * K + 1), generator=torch.Generator().manual_seed(9)).cuda()
    eager, graphed = (Loop(model, prompts, 12, 0.6) for _ in range(2))
    try:
        want = []
        for s in range(10):
            eager.u.copy_(u[s])
            eager.step()
            eager.sync()
            want.append([x.cpu().numpy() for x in (eager.tokens, eager.path, eager.committed)])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mm(torch.ones(8, 8, device="cuda"), torch.ones(8, 8, device="cuda"))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            graphed.step()
        for s in range(10):
            graphed.u.copy_(u[s])
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip((graphed.tokens, graphed.path, graphed.committed), want[s]):
                assert np.array_equal(x.cpu().numpy(), y), s
        graphed.sync()
    finally:
        eager.close()
        graphed.close()
