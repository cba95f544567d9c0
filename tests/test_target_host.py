"""The verify step's calls on the host: defaults, refusals before anything
touches the GPU, and the 64-bit reference against hand-derived values (no GPU
needed)."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

import target_reference as R
from prompt_lookup_gram_amd import binding as B


def params(**kw):
    p = B.pld_target_params_default()
    p.q_heads, p.kv_heads, p.vocab = 8, 2, 100
    for k, v in kw.items():
        if k.startswith("rope_"):
            setattr(p.rope, k[5:], v)
        else:
            setattr(p, k, v)
    return p


def test_defaults():
    p = B.pld_target_params_default()
    assert (p.max_batch, p.max_rows, p.max_len) == (1, 16, 32768)
    assert (p.q_heads, p.kv_heads, p.head_dim, p.vocab) == (0, 0, 128, 0)
    assert (p.dtype, p.cache_dtype, p.page_tokens) == (B.PLD_BF16, B.PLD_BF16, 64)
    r = p.rope
    assert (r.rot_dim, r.interleaved, r.scaling, r.original_len) == (0, 0, 0, 32768)
    assert (r.base, r.factor, r.beta_fast, r.beta_slow, r.magnitude) == (1e4, 1, 32, 1, 1)
    assert B.load().pld_target_params_default(None) == B.PLD_EINVAL


@pytest.mark.parametrize("field,value,word", [
    ("max_batch", 0, "max_batch"), ("max_rows", 0, "max_rows"), ("max_len", 0, "max_len"),
    ("max_len", 2**30 + 1, "max_len"), ("vocab", -1, "vocab"), ("vocab", 2**24 + 1, "vocab"),
    ("max_batch", 2**27, "max_batch"), ("max_rows", 2**29, "max_rows"), ("q_heads", 7, "q_heads"),
    ("q_heads", 0, "q_heads"), ("kv_heads", 0, "q_heads"), ("kv_heads", -2, "q_heads"),
    ("head_dim", 80, "head_dim"), ("head_dim", 512, "head_dim"), ("dtype", B.PLD_F32, "dtype"),
    ("dtype", 9, "dtype"), ("cache_dtype", B.PLD_F16, "cache_dtype"),
    ("page_tokens", 8, "page_tokens"), ("page_tokens", 48, "page_tokens"),
    ("rope_rot_dim", 3, "rot_dim"), ("rope_rot_dim", 130, "rot_dim"),
    ("rope_rot_dim", -2, "rot_dim")])
def test_create_refuses(field, value, word):
    with pytest.raises(B.PldError) as e:
        B.pld_create_target(params(**{field: value}))
    assert e.value.status == B.PLD_EINVAL and word in str(e.value)


@pytest.mark.parametrize("kw", [
    {"rope_interleaved": 2}, {"rope_scaling": 3}, {"rope_base": 1.0}, {"rope_base": math.inf},
    {"rope_magnitude": 0.0}, {"rope_magnitude": math.nan},
    {"rope_scaling": 1, "rope_factor": 0.0}, {"rope_scaling": 2, "rope_factor": -1.0},
    {"rope_scaling": 2, "rope_original_len": 0}, {"rope_scaling": 2, "rope_beta_slow": 0.0},
    {"rope_scaling": 2, "rope_beta_fast": 0.5}])
def test_create_refuses_rope(kw):
    with pytest.raises(B.PldError) as e:
        B.pld_create_target(params(rope_rot_dim=64, **kw))
    assert e.value.status == B.PLD_EINVAL and "rope" in str(e.value)


def test_create_refuses_an_empty_geometry_and_null():
    with pytest.raises(B.PldError) as e:
        B.pld_create_target(params(q_heads=0, kv_heads=0, vocab=0))
    assert e.value.status == B.PLD_EINVAL
    ctx = ctypes.c_void_p()
    assert B.load().pld_create_target(ctypes.byref(ctx), None, None) == B.PLD_EINVAL
    assert B.load().pld_create_target(None, ctypes.byref(params()), None) == B.PLD_EINVAL


def test_null_context_refused():
    f32 = ctypes.c_float(0)
    lib = B.load()
    assert lib.pld_kv_append(None, None, 0, None, None, 0, 1, None, None, 0, None, 1, None, None,
                             0, None, None, None, None) == B.PLD_EINVAL
    assert lib.pld_attend(None, None, 0, 1, None, None, 0, 0, None, 1, None, None, 0, None, None,
                          f32, 0, None, None, None) == B.PLD_EINVAL
    assert lib.pld_verify(None, None, 0, 1, 1, None, None, None, None, 0, None, None, 0, None,
                          None, None, None, None) == B.PLD_EINVAL
    assert "ctx is null" in B.pld_last_error()


def test_binding_checks_tensors_before_the_call():
    import torch
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        B.pld_attend(1, cpu.half(), 8, 1, None, None, 0, 0, None, 1, None, None, 0)
    with pytest.raises(ValueError, match="on the GPU"):
        B.pld_verify(1, cpu, 8, 1, None, None, None, None, 0, None, None, 0, None, None, None)
    with pytest.raises(TypeError, match="logits"):
        B.pld_verify(1, 1234, 8, 1, None, None, None, None, 0, None, None, 0, None, None, None)


class _Recorder:
    """Stands for the library: takes every call."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            if name == "pld_create_target":
                args[0]._obj.value = 4096
            return 0
        return call


@pytest.mark.parametrize("dt,cache", [("bfloat16", "bfloat16"), ("float16", "float16"),
                                      ("bfloat16", "float8_e4m3fn"), ("float16", "float8_e4m3fn")])
def test_binding_checks_dtypes_against_the_context(monkeypatch, dt, cache):
    """A cache or rows of another type than the context's would be read and
    written past their end, or as other numbers: refused before the call."""
    import torch
    lib = _Recorder()
    monkeypatch.setattr(B, "_lib", lib)
    # CPU tensors pass for the device's: their get_device() is -1
    monkeypatch.setattr(B, "_types", {**B._verify_types(), "gpu": True, "device": lambda: -1})
    types = {"float16", "bfloat16", "float8_e4m3fn"}
    p = params(dtype=B.PLD_TYPES[getattr(torch, dt)],
               cache_dtype=B.PLD_TYPES[getattr(torch, cache)])
    ctx = B.pld_create_target(p, 0)
    one = torch.ones(4, dtype=torch.int32)

    def tensor(name):
        return torch.zeros(64, dtype=getattr(torch, name))

    def attend(q, k, v, out):
        B.pld_attend(ctx, tensor(q), 64, 1, one, one, 0, 1, one, 1, tensor(k), tensor(v), 1,
                     out=tensor(out), stream=0)

    def append(q, k, v, kc, vc, out):
        B.pld_kv_append(ctx, tensor(q), 64, tensor(k), tensor(v), 64, 1, one, one, 1, one, 1,
                        tensor(kc), tensor(vc), 1, out_q=tensor(out), stream=0)
    for call, good in ((attend, (dt, cache, cache, dt)), (append, (dt, dt, dt, cache, cache, dt))):
        lib.calls.clear()
        call(*good)
        assert len(lib.calls) == 1
        for i, right in enumerate(good):
            for wrong in types - {right}:
                with pytest.raises(ValueError):
                    call(*good[:i], wrong, *good[i + 1:])
        assert len(lib.calls) == 1, "a call with another type reached the library"
    # the handle of a context that is gone says nothing about the next one's types
    B.pld_destroy(ctx)
    attend("bfloat16", "bfloat16", "bfloat16", "bfloat16")
    attend("float16", "float8_e4m3fn", "float8_e4m3fn", "float16")


# ---------------------------------------------------------------------------
# the reference, against values derived by hand
# ---------------------------------------------------------------------------


def test_reference_rotation():
    f = R.rope_frequencies(4, base=100.0)
    assert np.allclose(f, [1.0, 0.1])
    x = np.array([[1.0, 2.0, 3.0, 4.0, 5.0]])
    y, _ = R.rotate(x, 0, f, 4, False, 1.0)
    assert np.array_equal(y, x)
    # a quarter turn of pair 0: (x, y) -> (-y, x)
    f = np.array([math.pi / 2, 0.0])
    y, _ = R.rotate(x, 1, f, 4, False, 1.0)
    assert np.allclose(y, [[-3.0, 2.0, 1.0, 4.0, 5.0]])
    y, _ = R.rotate(x, 1, f, 4, True, 2.0)
    assert np.allclose(y, [[-4.0, 2.0, 6.0, 8.0, 5.0]])
    # scores of rotated vectors depend on the distance alone
    rng = np.random.default_rng(5)
    f = R.rope_frequencies(16)
    q, k = rng.standard_normal((2, 1, 16))
    for layout in (False, True):
        a = [R.rotate(q, p + 9, f, 16, layout, 1.0)[0] @ R.rotate(k, p, f, 16, layout, 1.0)[0].T
             for p in (0, 7, 100000)]
        assert np.allclose(a, a[0])


def test_reference_frequency_scaling():
    n, s = 32, 8.0
    plain = R.rope_frequencies(n)
    assert np.allclose(R.rope_frequencies(n, "linear", factor=s), plain / s)
    banded = R.rope_frequencies(n, "banded", factor=s, original_len=4096)
    turns = plain * 4096 / (2 * math.pi)
    assert np.allclose(banded[turns > 64], plain[turns > 64])
    assert np.allclose(banded[turns < 0.5], plain[turns < 0.5] / s)
    assert np.all(banded <= plain * (1 + 1e-12)) and np.all(banded >= plain / s * (1 - 1e-12))
    assert np.all(np.diff(banded) < 0)


def test_reference_attention():
    # two positions in one page; head 1 of 2 shares kv head 0
    kc = np.zeros((1, 1, 16, 2))
    vc = np.zeros((1, 1, 2, 16))
    kc[0, 0, 1] = [math.log(3.0), 0.0]
    vc[0, 0, :, 0], vc[0, 0, :, 1] = [1.0, 0.0], [0.0, 1.0]
    q = np.zeros((1, 2, 2, 2))
    q[0, :, 1, 0] = 1.0
    table = np.zeros((1, 1), int)
    out, lse, mass, _ = R.attend(q, kc, vc, table, [1], [1], 16, 1.0, 0)
    # row 0 sees position 0 only; row 1 weighs them 1 : 1 and 1 : 3
    assert np.allclose(out[0, 0], [[1, 0], [1, 0]])
    assert np.allclose(out[0, 1], [[0.5, 0.5], [0.25, 0.75]])
    assert np.allclose(lse[0, 1], [math.log(2), math.log(4)])
    assert np.allclose(mass, out)
    out, _, _, _ = R.attend(q, kc, vc, table, [1], [1], 16, 1.0, 1)
    assert np.allclose(out[0, 1], [[0, 1], [0, 1]])
    out, _, _, _ = R.attend(q, kc, vc, table, [0], [1], 16, 1.0, 0)
    assert np.isnan(out).all()


def test_reference_verification():
    z = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.6, 0.3], [0.2, 0.2, 0.6]]))
    no = [False, False]
    # both accepted: the draw is from the last row
    assert R.verify_one(z, [0, 1], 2, no, None, 1.0, [0.4, 0.5], 0.39)[0] == [0, 1, 1]
    # refused at row 1 (0.6 < u): drawn from [0.1, 0, 0.3]
    assert R.verify_one(z, [0, 1], 2, no, None, 1.0, [0.4, 0.7], 0.24)[0] == [0, 0]
    tok, logp = R.verify_one(z, [0, 1], 2, no, None, 1.0, [0.4, 0.7], 0.26)
    assert tok == [0, 2] and np.allclose(logp, [math.log(0.5), math.log(0.3)])
    # a drafter's q: accepted at u q < p; else from the excess over q
    q = np.array([[0.8, 0.1, 0.1]])
    assert R.verify_one(z, [0], 1, [True], q, 1.0, [0.62], 0.0)[0] == [0, 0]
    assert R.verify_one(z, [0], 1, [True], q, 1.0, [0.63], 0.0)[0] == [1]
    assert R.verify_one(z, [0], 1, [True], q, 1.0, [0.63], 0.51)[0] == [2]
    # greedy: argmax, lowest index on a tie
    g = np.array([[1.0, 1.0, 0.0], [0.0, 2.0, 2.0]])
    assert R.verify_one(g, [0], 1, no, None, 0.0, [0.9], 0.9)[0] == [0, 1]
    assert R.verify_one(g, [1], 1, no, None, 0.0, [0.0], 0.9)[0] == [0]


def test_reference_commits_the_targets_distribution():
    """Over a grid of random numbers the first committed token's frequencies
    are the target's probabilities, for a point mass and for a drafter's q."""
    p = np.array([0.45, 0.3, 0.2, 0.05])
    z = np.log(np.stack([p, p]))
    grid = (np.arange(40) + 0.5) / 40
    for probs in (None, np.array([[0.1, 0.6, 0.1, 0.2]])):
        hits = np.zeros(4)
        for x in range(4):
            w = (probs[0][x] if probs is not None else (1.0 if x == 1 else 0.0))
            if w == 0:
                continue
            for u in grid:
                for ud in grid:
                    tok, _ = R.verify_one(z, [x], 1, [probs is not None], probs, 1.0, [u], ud)
                    hits[tok[0]] += w
        # 40 steps: each acceptance edge is off by at most half a step
        assert np.abs(hits / 1600 - p).max() < 2.0 / 40
