"""The verify step's operators, as cases that can be measured.

Three operators of libpld follow the draft call of a speculative decoding
step: ``pld_kv_append`` (rotary positions, and the block's keys and values
into the paged cache), ``pld_attend`` (attention of the block's rows over that
cache) and ``pld_verify`` (acceptance of the drafted tokens from the target
model's logits and given random numbers, and the draw of the token after
them). Each case is one call of one of them.

``own`` False computes the same in elementary torch operations; ``own`` True
makes the library's calls. ``exact`` states each operator once more in 64 bits.

Shared conventions: a request has ``lengths[b]`` tokens, the last of which is
row 0 of its block, and ``draft_len[b]`` drafted tokens, rows 1.. of it; row t
stands at position lengths[b] - 1 + t. A block is padded to ``rows`` rows.
K pages are [page, kv_head, token, head_dim], V pages [page, kv_head,
head_dim, token].
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def _verify(name, batch, draft, vocab, dtype, temperature, accept, probs=0, ragged=False):
    return {"op": "verify", "name": name, "batch": batch, "draft": draft, "vocab": vocab,
            "dtype": dtype, "temperature": temperature, "accept": accept, "probs": probs,
            "ragged": ragged}


def _attend(name, batch, lo, hi, draft, heads, kv_heads, dim, dtype, cache, page, window=0,
            ragged=False):
    return {"op": "attend", "name": name, "batch": batch, "lo": lo, "hi": hi, "draft": draft,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": cache,
            "page": page, "window": window, "ragged": ragged}


def _append(name, batch, lo, hi, draft, heads, kv_heads, dim, dtype, page, rot, interleaved,
            scaling, ragged=False):
    return {"op": "append", "name": name, "batch": batch, "lo": lo, "hi": hi, "draft": draft,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "page": page,
            "rot": rot, "interleaved": interleaved, "scaling": scaling, "ragged": ragged}


def listed():
    return [
        # one request's 16 lookup tokens, small vocabulary: latency alone
        _verify("verify_b1_d16_v32000_f32", 1, 16, 32000, "f32", 1.0, 0.8),
        # a small batch's 15-token blocks while it copies a document
        _verify("verify_b8_d15_v151936_bf16", 8, 15, 151936, "bf16", 0.8, 0.9),
        # a full serving batch with ragged lookup drafts
        _verify("verify_b64_d16_v151936_bf16", 64, 16, 151936, "bf16", 1.0, 0.7, ragged=True),
        # a model drafter's 7 proposals with their probabilities, odd vocabulary
        _verify("verify_b32_d7_probs_v50257_f32", 32, 7, 50257, "f32", 0.7, 0.75, probs=7),
        # greedy decoding's acceptance
        _verify("verify_b64_d7_greedy_v151936_f16", 64, 7, 151936, "f16", 0.0, 0.8),
        # a short chat's next token, one request
        _attend("attend_b1_4096_t1", 1, 4096, 4096, 0, 32, 8, 128, "bf16", "bf16", 16),
        # the 16-row verify block over a 25,000-token document
        _attend("attend_b8_25000_t16", 8, 25000, 25000, 15, 16, 2, 128, "bf16", "bf16", 64),
        # a serving batch's single tokens over ragged contexts
        _attend("attend_b64_ragged_t1", 64, 8192, 65536, 0, 32, 8, 128, "bf16", "bf16", 64,
                ragged=True),
        # ragged lookup drafts over an 8-bit cache
        _attend("attend_b64_ragged_t8_e4m3", 64, 8192, 65536, 7, 16, 4, 128, "f16", "e4m3", 32,
                ragged=True),
        # the longest contexts with full verify blocks
        _attend("attend_b16_262144_t16", 16, 262144, 262144, 15, 16, 2, 128, "bf16", "bf16", 64),
        # a batch's verify blocks going into the cache
        _append("append_b64_t16_half", 64, 8192, 65536, 15, 32, 8, 128, "bf16", 64, 128, False,
                "plain", ragged=True),
        # a long prompt going into the cache in one call
        _append("append_b1_t65536_banded", 1, 1, 1, 65535, 32, 8, 128, "bf16", 64, 64, True,
                "banded"),
    ]


def _span(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["verify", "attend", "append"])
    if op == "verify":
        batch, draft = _span(rng, 1, 64), rng.randint(0, 16)
        vocab = _span(rng, 1000, 151936)
        greedy = rng.random() < 0.25
        probs = min(draft, 7) if rng.random() < 0.3 and not greedy else 0
        return _verify("", batch, draft, vocab, rng.choice(["f32", "bf16", "f16"]),
                       0.0 if greedy else round(rng.uniform(0.3, 1.5), 2),
                       round(rng.uniform(0.3, 0.95), 2), probs, rng.random() < 0.5)
    dim = rng.choice([64, 96, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    dtype = rng.choice(["bf16", "f16"])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.6
    if op == "attend":
        batch = _span(rng, 1, 64)
        draft = rng.choice([0, 0, 1, 3, 7, 15, rng.randint(0, 15)])
        # at most the largest listed case's cache, products and plain copies
        cost = batch * kv_heads * dim * max(1, (draft + 1) * group / 32)
        hi = _span(rng, 16, max(16, min(262144, int(2.0e9 / 2 / cost))))
        lo = _span(rng, max(1, hi // 8), hi) if ragged else hi
        window = rng.choice([0, 0, 0, 2048, _span(rng, 1, 4096)])
        return _attend("", batch, lo, hi, draft, kv_heads * group, kv_heads, dim, dtype,
                       rng.choice([dtype, dtype, "e4m3"]), page, window, ragged)
    batch = _span(rng, 1, 64)
    draft = _span(rng, 1, max(1, int(65536 * 48 * 128 / (batch * kv_heads * (group + 2) * dim)))) - 1
    draft = min(draft, 65535)
    hi = _span(rng, 1, 262144 - draft)
    lo = _span(rng, max(1, hi // 8), hi) if ragged else hi
    return _append("", batch, lo, hi, draft, kv_heads * group, kv_heads, dim, dtype, page,
                   rng.choice([dim, dim // 2, dim // 4, 0]), rng.random() < 0.5,
                   rng.choice(["plain", "linear", "banded"]), ragged)


def _rows(case):
    """Mean rows of a request's block."""
    return 1 + (case["draft"] / 2 if case["ragged"] and case["draft"] < 64 else case["draft"])


def work(case):
    b = case["batch"]
    if case["op"] == "verify":
        # rows up to the first refusal (the expected number), each once, and
        # the refused row's draft probabilities
        v, a, d = case["vocab"], case["accept"], _rows(case) - 1
        rows = b * (1 - a ** (d + 1)) / (1 - a)
        n = rows * v
        byte = n * SIZE[case["dtype"]]
        if case["probs"]:
            byte += b * (1 - a ** d) * v * 4
        return {"bytes": int(byte), "flops": int(4 * n)}
    rows = b * _rows(case)
    hq, hk, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        return {"bytes": int(rows * (hq + 2 * hk) * dim * 2 * SIZE[case["dtype"]]),
                "flops": int(rows * (hq + hk) * case["rot"] * 3 + 1)}
    mean = (case["lo"] + case["hi"]) / 2 + _rows(case) - 1
    seen = min(mean, case["window"] + _rows(case) - 1) if case["window"] else mean
    per_row = min(mean, case["window"]) if case["window"] else mean
    byte = b * seen * hk * dim * 2 * SIZE[case["cache"]] + rows * hq * (2 * dim * 2 + 4)
    return {"bytes": int(byte), "flops": int(4 * rows * per_row * hq * dim)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


class _Context:
    """A library context that goes with the state."""

    def __init__(self, handle, destroy):
        self.handle, self.destroy = handle, destroy

    def __del__(self):
        self.destroy(self.handle)


def _rope_fields(case):
    return {"rot_dim": case["rot"], "interleaved": int(case["interleaved"]),
            "scaling": {"plain": 0, "linear": 1, "banded": 2}[case["scaling"]],
            "base": 10000.0, "factor": 8.0, "original_len": 32768, "beta_fast": 32.0,
            "beta_slow": 1.0, "magnitude": 0.1 * math.log(8.0) + 1.0
            if case["scaling"] == "banded" else 1.0}


def _context(case, state):
    from prompt_lookup_gram_amd import binding as B
    p = B.pld_target_params_default()
    p.max_batch, p.max_rows = case["batch"], case["draft"] + 1
    if case["op"] == "verify":
        p.vocab = case["vocab"]
    else:
        p.max_len = state["max_len"]
        p.q_heads, p.kv_heads, p.head_dim = case["heads"], case["kv_heads"], case["dim"]
        p.dtype = B.PLD_TYPES[TYPES[case["dtype"]]]
        p.cache_dtype = B.PLD_TYPES[TYPES[case.get("cache", case["dtype"])]]
        p.page_tokens = case["page"]
        if case["op"] == "append":
            for k, v in _rope_fields(case).items():
                setattr(p.rope, k, v)
    state["B"] = B
    state["ctx"] = _Context(B.pld_create_target(p), B.pld_destroy)


def _blocks(case, rng):
    """lengths and draft_len of a batch, on the host."""
    b = case["batch"]
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(b)]
    dlen = [rng.randint(0, case["draft"]) if case["ragged"] and case["draft"] < 64
            else case["draft"] for _ in range(b)]
    return lens, dlen


def _pages(case, lens, dlen, rng):
    """A page table over randomly placed pages: (table, pages)."""
    page = case["page"]
    need = [-(-(n + d) // page) for n, d in zip(lens, dlen)]
    ids = list(range(sum(need)))
    rng.shuffle(ids)
    width = max(need)
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [0] * (width - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32, device=DEV), len(ids)


def _randn(shape, gen, dtype):
    """Normal values of a type, made a slice at a time."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEV))
    return out


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    make = {"verify": _prepare_verify, "attend": _prepare_attend, "append": _prepare_append}
    state = make[case["op"]](case, gen, rng)
    state["case"] = case
    if own:
        _context(case, state)
    return state


def _prepare_verify(case, gen, rng):
    b, d, v = case["batch"], case["draft"], case["vocab"]
    temp = case["temperature"]
    scale = temp if temp > 0 else 1.0
    dlen = [rng.randint(0, d) if case["ragged"] else d for _ in range(b)]
    logits = torch.empty((b, d + 1, v), dtype=TYPES[case["dtype"]], device=DEV)
    draft = torch.randint(0, v, (b, max(1, d)), generator=gen, device=DEV)[:, :d]
    # a request's rows: normal logits, and the drafted token at about the
    # case's acceptance (probability `accept`, spread around it)
    for i in range(b):
        z = torch.randn((d + 1, v), generator=gen, device=DEV) * 2.0
        p = case["accept"] + 0.2 * (torch.rand((d, 1), generator=gen, device=DEV) - 0.5)
        p = p.clamp(0.02, 0.98)
        if temp == 0.0:
            hit = torch.rand((d, 1), generator=gen, device=DEV) < case["accept"]
            plant = torch.where(hit, z[:d].amax(1, keepdim=True) + 2.0, -4.0)
        else:
            rest = torch.logsumexp(z[:d] / scale, 1, keepdim=True)
            plant = scale * (rest + torch.log(p / (1 - p)))
        if d:
            z[:d].scatter_(1, draft[i, :, None], plant)
        logits[i] = z.to(logits.dtype)
    state = {"logits": logits, "draft": draft.to(torch.int32).contiguous(),
             "draft_len": _ints(dlen),
             "temperature": torch.full((b,), temp, dtype=torch.float32, device=DEV),
             "uniform": torch.rand((b, d + 1), generator=gen, device=DEV), "probs": None}
    if case["probs"]:
        # the drafter's own distribution: the target's, blurred
        h = case["probs"]
        q = torch.empty((b, h, v), dtype=torch.float32, device=DEV)
        for i in range(b):
            noise = torch.randn((h, v), generator=gen, device=DEV) * 0.5
            q[i] = torch.softmax(logits[i, :h].float() / scale + noise, -1)
        state["probs"] = q
    state["out_tokens"] = torch.empty((b, d + 1), dtype=torch.int32, device=DEV)
    state["out_accepted"] = torch.empty(b, dtype=torch.int32, device=DEV)
    state["out_counts"] = torch.empty(b, dtype=torch.int32, device=DEV)
    state["out_logprobs"] = torch.empty((b, d + 1), dtype=torch.float32, device=DEV)
    return state


def _prepare_attend(case, gen, rng):
    b, rows = case["batch"], case["draft"] + 1
    hq, hk, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens, dlen = _blocks(case, rng)
    table, pages = _pages(case, lens, dlen, rng)
    dt = TYPES[case["dtype"]]
    # scores with a deviation of 3: attention that a few hundred keys carry
    state = {"lengths": _ints(lens), "draft_len": _ints(dlen), "table": table, "pages": pages,
             "max_len": max(n + d for n, d in zip(lens, dlen)),
             "k": _randn((pages, hk, page, dim), gen, TYPES[case["cache"]]),
             "v": _randn((pages, hk, dim, page), gen, TYPES[case["cache"]]),
             "q": _randn((b, rows, hq, dim), gen, dt) * 3, "k_scale": None, "v_scale": None,
             "out": torch.zeros((b, rows, hq, dim), dtype=dt, device=DEV),
             "lse": torch.zeros((b, rows, hq), dtype=torch.float32, device=DEV)}
    if case["cache"] == "e4m3":
        state["k_scale"] = 0.5 + torch.rand(hk, generator=gen, device=DEV)
        state["v_scale"] = 0.5 + torch.rand(hk, generator=gen, device=DEV)
    return state


def _prepare_append(case, gen, rng):
    b, rows = case["batch"], case["draft"] + 1
    hq, hk, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens, dlen = _blocks(case, rng)
    # a cache of the pages that the block's rows fall in; the positions
    # before them share one page that the call does not touch
    first = [(n - 1) // page for n in lens]
    last = [(n - 1 + d) // page for n, d in zip(lens, dlen)]
    width, at = max(last) + 1, 1
    ids = list(range(1, 1 + sum(y - x + 1 for x, y in zip(first, last))))
    rng.shuffle(ids)
    table = torch.zeros((b, width), dtype=torch.int32)
    for i, (x, y) in enumerate(zip(first, last)):
        table[i, x:y + 1] = torch.tensor(ids[at - 1:at + y - x], dtype=torch.int32)
        at += y - x + 1
    dt = TYPES[case["dtype"]]
    # q, k and v are slices of one projection's output
    qkv = _randn((b * rows, (hq + 2 * hk) * dim), gen, dt)
    return {"lengths": _ints(lens), "draft_len": _ints(dlen), "table": table.to(DEV), "pages": at,
            "max_len": max(n + d for n, d in zip(lens, dlen)), "qkv": qkv,
            "q": qkv[:, :hq * dim], "k_new": qkv[:, hq * dim:(hq + hk) * dim],
            "v_new": qkv[:, (hq + hk) * dim:], "k": _randn((at, hk, page, dim), gen, dt),
            "v": _randn((at, hk, dim, page), gen, dt),
            "out_q": torch.zeros((b, rows, hq, dim), dtype=dt, device=DEV)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(state):
    case = state["case"]
    if own:
        return {"verify": _own_verify, "attend": _own_attend, "append": _own_append}[case["op"]](
            case, state)
    return {"verify": _plain_verify, "attend": _plain_attend, "append": _plain_append}[
        case["op"]](case, state)


def _own_verify(case, s):
    s["B"].pld_verify(s["ctx"].handle, s["logits"], case["vocab"], case["draft"] + 1, s["draft"],
                      s["draft_len"], None, s["probs"], case["probs"], s["temperature"],
                      s["uniform"], case["batch"], s["out_tokens"], s["out_accepted"],
                      s["out_counts"], s["out_logprobs"])
    return s["out_tokens"], s["out_accepted"], s["out_counts"], s["out_logprobs"]


def _own_attend(case, s):
    s["B"].pld_attend(s["ctx"].handle, s["q"], case["heads"] * case["dim"], case["draft"] + 1,
                      s["lengths"], s["draft_len"], s["max_len"], case["batch"], s["table"],
                      s["table"].shape[1], s["k"], s["v"], s["pages"], s["k_scale"],
                      s["v_scale"], 0.0, case["window"], s["out"], s["lse"])
    return s["out"], s["lse"]


def _own_append(case, s):
    width = s["qkv"].shape[1]
    s["B"].pld_kv_append(s["ctx"].handle, s["q"], width, s["k_new"], s["v_new"], width,
                         case["draft"] + 1, s["lengths"], s["draft_len"], case["batch"],
                         s["table"], s["table"].shape[1], s["k"], s["v"], s["pages"], None, None,
                         s["out_q"])
    return s["out_q"], s["k"], s["v"]


def _plain_verify(case, s):
    logits, draft, dlen = s["logits"], s["draft"].long(), s["draft_len"].long()
    b, rows, v = logits.shape
    d = rows - 1
    temp = s["temperature"]
    greedy = case["temperature"] == 0.0
    scale = torch.where(temp > 0, temp, torch.ones_like(temp))[:, None, None]
    z = logits.float()
    top, arg = z.max(-1)
    # the first index of the largest value
    if greedy:
        arg = (z == top[..., None]).to(torch.int8).argmax(-1)
    total = torch.exp((z - top[..., None]) / scale).sum(-1, dtype=torch.float64)
    at = torch.arange(d, device=DEV)[None, :]
    zd = z[:, :d].gather(2, draft[..., None])[..., 0].double()
    weight = torch.exp((zd - top[:, :d].double()) / scale[..., 0].double())
    p = weight / total[:, :d]
    q = torch.ones_like(p)
    h = case["probs"]
    if h:
        q[:, :h] = s["probs"].gather(2, draft[:, :h, None])[..., 0].double()
    ok = (draft == arg[:, :d]) if greedy else (s["uniform"][:, :d].double() * q < p)
    refuse = (~ok) & (at < dlen[:, None])
    first = torch.where(refuse, at, d).amin(1) if d else torch.zeros_like(dlen)
    accepted = torch.minimum(first, dlen)
    refused = accepted < dlen
    pick = torch.arange(b, device=DEV)
    if greedy:
        token = arg[pick, accepted]
    else:
        # the row after the last accepted token, in 64 bits: what the draft
        # did not already claim, drawn by the running sum
        row = logits[pick, accepted].double()
        w = torch.exp((row - row.amax(1, keepdim=True)) / scale[:, 0].double())
        if d:
            x = draft[pick, accepted.clamp(max=d - 1)]
            if h:
                has = refused & (accepted < h)
                claim = s["probs"][pick, accepted.clamp(max=h - 1)].double()
                left = (w - claim * w.sum(1, keepdim=True)).clamp(min=0)
                has = has & (left.sum(1) > 0)
            else:
                has = torch.zeros_like(refused)
            point = refused & ~(accepted < h)
            only = w.scatter(1, x[:, None], 0.0)
            w = torch.where(point[:, None], only, w)
            if h:
                w = torch.where(has[:, None], left, w)
        c = w.cumsum(1)
        u = s["uniform"][:, -1].double()
        token = (c <= u[:, None] * c[:, -1:]).sum(1).clamp(max=v - 1)
    out = torch.full((b, rows), -1, dtype=torch.int64, device=DEV)
    if d:
        out[:, :d] = torch.where(at < accepted[:, None], draft, -1)
    out.scatter_(1, accepted[:, None], token[:, None])
    zt = z.gather(2, out.clamp(min=0)[..., None])[..., 0].double()
    logp = (zt - top.double()) / scale[..., 0].double() - torch.log(total)
    logp = torch.where(out >= 0, logp, torch.zeros_like(logp))
    return (out.to(torch.int32), accepted.to(torch.int32), (accepted + 1).to(torch.int32),
            logp.float())


def _plain_attend(case, s):
    hq, hk, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    g = hq // hk
    out, lse = s["out"], s["lse"]
    rows = out.shape[1]
    scale = dim ** -0.5
    for b in range(case["batch"]):
        n = min(s["max_len"], s["table"].shape[1] * page)
        ids = s["table"][b, :-(-n // page)].long()
        pos = torch.arange(ids.numel() * page, device=DEV)
        length, dlen = s["lengths"][b], s["draft_len"][b]
        at = length - 1 + torch.arange(rows, device=DEV)
        live = torch.arange(rows, device=DEV) <= dlen
        see = pos[None, :] <= at[:, None]
        if case["window"]:
            see = see & (pos[None, :] > at[:, None] - case["window"])
        see = see.repeat_interleave(g, 0)
        for h in range(hk):
            k = s["k"][ids, h].float().reshape(-1, dim)
            v = s["v"][ids, h].float().transpose(1, 2).reshape(-1, dim)
            if s["k_scale"] is not None:
                k = k * s["k_scale"][h]
                v = v * s["v_scale"][h]
            v = torch.where((pos < length + dlen)[:, None], v, 0.0)
            q = s["q"][b, :, h * g:(h + 1) * g].float().reshape(rows * g, dim)
            x = (q @ k.t()) * scale
            x = torch.where(see, x, -math.inf)
            top = x.amax(1, keepdim=True)
            e = torch.exp(x - top)
            total = e.sum(1, keepdim=True)
            o = ((e / total) @ v).reshape(rows, g, dim)
            ls = (top + torch.log(total)).reshape(rows, g)
            part = out[b, :, h * g:(h + 1) * g]
            part.copy_(torch.where(live[:, None, None], o, part.float()))
            part = lse[b, :, h * g:(h + 1) * g]
            part.copy_(torch.where(live[:, None], ls, part))
    return out, lse


def _frequencies(case):
    """Rotations per position of each pair, in 64 bits, and the factor on
    the rotated values."""
    r = _rope_fields(case)
    n = case["rot"]
    i = torch.arange(n // 2, dtype=torch.float64, device=DEV)
    f = torch.exp(i * (-2.0 * math.log(r["base"]) / max(1, n)))
    if case["scaling"] == "linear":
        f = f / r["factor"]
    elif case["scaling"] == "banded":
        def turn(beta):
            return n / 2 * math.log(r["original_len"] / (beta * 2 * math.pi)) / math.log(r["base"])
        lo = max(0, math.floor(turn(r["beta_fast"])))
        hi = min(n - 1, math.ceil(turn(r["beta_slow"])))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / r["factor"] * ramp + f * (1 - ramp)
    return f, r["magnitude"]


def _rotate(case, x, cos, sin):
    """x [tokens, heads, dim] rotated by cos and sin [tokens, 1, rot / 2]."""
    n = case["rot"]
    if n == 0:
        return x
    if case["interleaved"]:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., n:]), -1)


def _plain_append(case, s):
    hq, hk, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    b, rows = case["batch"], case["draft"] + 1
    t = torch.arange(rows, device=DEV)[None, :]
    live = (t <= s["draft_len"][:, None]).reshape(-1)
    pos = (s["lengths"][:, None].long() - 1 + t).reshape(-1)
    f, gain = _frequencies(case)
    angle = pos[:, None, None].double() * f
    cos, sin = (torch.cos(angle) * gain).float(), (torch.sin(angle) * gain).float()
    q = _rotate(case, s["q"].reshape(b * rows, hq, dim).float(), cos, sin)
    k = _rotate(case, s["k_new"].reshape(b * rows, hk, dim).float(), cos, sin)
    v = s["v_new"].reshape(b * rows, hk, dim)
    keep = torch.nonzero(live)[:, 0]
    where = pos[keep]
    ids = s["table"][keep // rows, where // page].long()
    s["out_q"].view(b * rows, hq, dim)[keep] = q[keep].to(s["out_q"].dtype)
    s["k"][ids, :, where % page] = k[keep].to(s["k"].dtype)
    s["v"][ids, :, :, where % page] = v[keep]
    return s["out_q"], s["k"], s["v"]


# ---------------------------------------------------------------------------
# the operators in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"verify": _exact_verify, "attend": _exact_attend, "append": _exact_append}[
        case["op"]](case, s)


def _exact_verify(case, s):
    b, rows, v = s["logits"].shape
    d = rows - 1
    tokens = torch.full((b, rows), -1, dtype=torch.int32)
    accepted = torch.zeros(b, dtype=torch.int32)
    logps = torch.zeros((b, rows), dtype=torch.float64)
    dlen, draft = s["draft_len"].tolist(), s["draft"].tolist()
    u, temp = s["uniform"].double().tolist(), s["temperature"].double().tolist()
    for i in range(b):
        t = 0
        while True:
            z = s["logits"][i, t].double()
            logp = torch.log_softmax(z / (temp[i] if temp[i] > 0 else 1.0), 0)
            if temp[i] == 0:
                best = int(torch.nonzero(z == z.max())[0, 0])
            last = t == dlen[i]
            if not last:
                x = draft[i][t]
                if temp[i] == 0:
                    take = x == best
                else:
                    q = float(s["probs"][i, t, x]) if t < case["probs"] else 1.0
                    take = u[i][t] * q < math.exp(float(logp[x]))
                if take:
                    tokens[i, t], logps[i, t] = x, float(logp[x])
                    t += 1
                    continue
            if temp[i] == 0:
                pick = best
            else:
                p = torch.exp(logp)
                if not last:
                    if t < case["probs"]:
                        left = (p - s["probs"][i, t].double()).clamp(min=0)
                        p = left if float(left.sum()) > 0 else p
                    else:
                        p[x] = 0.0
                c = torch.cumsum(p, 0)
                pick = int(torch.searchsorted(c, (u[i][d] * c[-1]).reshape(1), right=True)[0])
                pick = min(pick, v - 1)
            tokens[i, t], logps[i, t], accepted[i] = pick, float(logp[pick]), t
            break
    return tuple(x.to(DEV) for x in (tokens, accepted, accepted + 1, logps))


def _exact_attend(case, s):
    hq, hk, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    g = hq // hk
    out, lse = s["out"].double(), s["lse"].double()
    for b, (n, d) in enumerate(zip(s["lengths"].tolist(), s["draft_len"].tolist())):
        end = n + d
        ids = s["table"][b, :-(-end // page)].long()
        for h in range(hk):
            k = s["k"][ids, h].double().flatten(0, 1)[:end]
            v = s["v"][ids, h].double().transpose(1, 2).flatten(0, 1)[:end]
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            q = s["q"][b, :d + 1, h * g:(h + 1) * g].double()
            for t in range(d + 1):
                hi = n + t
                lo = max(0, hi - case["window"]) if case["window"] else 0
                x = torch.matmul(q[t], k[lo:hi].t()) / math.sqrt(dim)
                total = torch.logsumexp(x, 1)
                lse[b, t, h * g:(h + 1) * g] = total
                out[b, t, h * g:(h + 1) * g] = torch.matmul(torch.exp(x - total[:, None]),
                                                            v[lo:hi])
    return out, lse


def _exact_append(case, s):
    hq, hk, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    b, rows, n = case["batch"], case["draft"] + 1, case["rot"]
    out_q, k, v = s["out_q"].double(), s["k"].double(), s["v"].double()
    r = _rope_fields(case)
    freq = [r["base"] ** (-2.0 * i / n) for i in range(n // 2)]
    if case["scaling"] == "linear":
        freq = [f / r["factor"] for f in freq]
    if case["scaling"] == "banded":
        def index(beta):
            return n * math.log(r["original_len"] / (2 * math.pi * beta)) / (
                2 * math.log(r["base"]))
        lo = max(math.floor(index(r["beta_fast"])), 0) if n else 0
        hi = min(math.ceil(index(r["beta_slow"])), n - 1) if n else 0
        keep = [1 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(n // 2)]
        freq = [f * w + f / r["factor"] * (1 - w) for f, w in zip(freq, keep)]
    freq = torch.tensor(freq, dtype=torch.float64, device=DEV)
    if case["interleaved"]:
        left = torch.arange(0, n, 2, device=DEV)
        right = left + 1
    else:
        left = torch.arange(n // 2, device=DEV)
        right = left + n // 2
    def turned(x, pos):
        """x [tokens, heads, dim] as complex pairs times exp(i angle)."""
        w = torch.polar(torch.full((pos.numel(), freq.numel()), r["magnitude"],
                                   dtype=torch.float64, device=DEV), pos[:, None] * freq)
        c = torch.complex(x[..., left], x[..., right]) * w[:, None]
        y = x.clone()
        y[..., left], y[..., right] = c.real, c.imag
        return y
    for i, (length, d) in enumerate(zip(s["lengths"].tolist(), s["draft_len"].tolist())):
        for t0 in range(0, d + 1, 8192):
            t1 = min(d + 1, t0 + 8192)
            pos = torch.arange(length - 1 + t0, length - 1 + t1, dtype=torch.float64, device=DEV)
            at = slice(i * rows + t0, i * rows + t1)
            out_q[i, t0:t1] = turned(s["q"][at].double().reshape(-1, hq, dim), pos)
            cell = pos.long()
            ids = s["table"][i, cell // page].long()
            k[ids, :, cell % page] = turned(s["k_new"][at].double().reshape(-1, hk, dim), pos)
            v[ids, :, :, cell % page] = s["v_new"][at].double().reshape(-1, hk, dim)
    return out_q, k, v
