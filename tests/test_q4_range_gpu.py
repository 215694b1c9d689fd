"""decode_q4 at the ends of its range.  All factors here are powers of two, so what is compared stands for the same
numbers: equal bits where nothing falls below the number formats' range inside, else the documented error of a score.

Inside, a score's products are held at 2^-73 of <q, k>, and the offset of a group, -8 sum(q), as three bf16 parts, the
last of them 2^-18 of it: 2^-73 * 2^3 * 32 |q| * 2^-18 = 2^-83 |q|, whole as long as its 8 bits lie above bf16's 2^-133,
that is |q| >= 2^-43."""

from __future__ import annotations

import dataclasses

import numpy as np
import pytest
import torch

from tests.helpers import f64
from tests.q4_cases import S_MAX, check, make, reference, score_error
from tests.test_q4_gpu import run_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from paged_attention_relative_attn_gb300 import build
    build.build()
    import paged_attention_relative_attn_gb300 as m
    return m


def scaled(pool, e):
    """The pool with every scale times 2^e; scales that are NaN (dead places) stay."""
    n, H, P, row = pool.shape
    D = row * 16 // 9
    out = pool.clone().view(n, H, P // 16, 9 * D)
    s = out[..., 8 * D:].contiguous().view(torch.bfloat16)
    out[..., 8 * D:] = torch.ldexp(s.double(), torch.tensor(float(e), device=s.device)).to(torch.bfloat16).view(torch.uint8)
    return out.view(pool.shape)


def inputs(q_len, D, G, window=0, q_std=1.0):
    lens = [300, 41, 1000, 17]
    inp = make([q_len] * 4, lens, 2 * G, 2, D, 16, window, 64, seed=400 + D + q_len, q_std=q_std)
    inp.q[inp.q.abs() > 4] = 4.0
    return inp


def shifted(inp, q, k):
    """(q times 2^q, K times 2^k, the scale such that the scores are the same numbers; the unscaled inputs with that
    scale).  The scale is passed in fp32, which holds one below 2^-126 with fewer bits: both get the number it holds."""
    scale = float(np.float32(inp.scale * 2.0 ** (-q - k)))
    return _times(inp, q, k, scale), dataclasses.replace(inp, scale=scale * 2.0 ** (q + k))


def _times(inp, q, k, scale):
    return dataclasses.replace(inp, q=torch.ldexp(inp.q.double(), torch.tensor(float(q), device=inp.q.device)).to(inp.q.dtype),
                               k_cache=scaled(inp.k_cache, k), scale=scale)


FORMS = [(1, 64, 2), (1, 128, 6), (4, 64, 1), (3, 128, 2)]


@pytest.mark.parametrize("q_len,D,G", FORMS)
@pytest.mark.parametrize("q,k", [(58, 0), (58, -98), (-30, 0), (0, 40), (-20, 124), (58, 66), (48, -98), (0, -45)])
def test_large_and_small_q_and_k(ops, q_len, D, G, q, k):
    """q to 2^60, K groups from 2^-99 to 2^126 and scales to 2^51: the same bits."""
    far, inp = shifted(inputs(q_len, D, G), q, k)
    want, lwant = run_decode(ops, inp, q_len)
    check(inp, want, lwant)
    out, lse = run_decode(ops, far, q_len)
    assert torch.equal(out, want) and torch.equal(lse, lwant)


@pytest.mark.parametrize("q_len,D,G", FORMS)
@pytest.mark.parametrize("q,k", [(-50, 100), (-50, -1), (-60, 115), (-80, 124), (-54, 1), (-45, 0)])
def test_small_q_against_large_factors(ops, q_len, D, G, q, k):
    """A score carries an absolute error of 2^-60 |scale| max(k, 2^-9), k being K's largest magnitude: more than fp32's
    where q is tiny and the other factors huge."""
    far, inp = shifted(inputs(q_len, D, G), q, k)
    ro, rl, size = reference(inp)
    out, lse = run_decode(ops, far, q_len)
    e = score_error(inp) + 2.0 ** -60 * far.scale * max(7 * S_MAX * 2.0 ** k, 2.0 ** -9)
    g = f64(out)
    assert np.isfinite(g).all()
    # as in check; a weight moves by a factor within exp(2 e)
    tol = 2.0 ** -8 * (np.abs(ro) + size) * (1 + 2.0 ** -7) + (np.expm1(2 * e) + 2.0 ** -20) * size
    tol += 2 * (1000 / 16 + 2) * 2.0 ** -23 * (23 * S_MAX + size)
    assert (np.abs(g - ro) <= tol).all()
    assert (np.abs(f64(lse) - rl) <= e[..., 0] + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl)).all()


@pytest.mark.parametrize("q_len,D,G", FORMS)
@pytest.mark.parametrize("e", [-35, 55])
@pytest.mark.parametrize("slope", [0.0, 0.02, -0.02])
def test_ends_of_v(ops, q_len, D, G, e, slope):
    """V groups of 2^-37 and 2^57, under scores that rise along the keys too (weights above 1 until the exponents'
    base follows): the bounds of the middle of the range."""
    inp = inputs(q_len, D, G)
    rel = inp.rel_logits + slope * torch.arange(64, device=inp.q.device)
    inp = dataclasses.replace(inp, rel_logits=rel.contiguous())
    ref = reference(inp)
    out, lse = run_decode(ops, dataclasses.replace(inp, v_cache=scaled(inp.v_cache, e)), q_len)
    check(inp, torch.ldexp(out.float(), torch.tensor(float(-e), device=out.device)), lse, ref)


def test_scales_past_the_range_are_refused(ops):
    inp = inputs(1, 64, 2)
    for scale in (2.0 ** 54, -2.0 ** 54):  # the last that are taken; q small enough for finite scores
        q = torch.ldexp(inp.q.double(), torch.tensor(-56.0, device=inp.q.device)).to(inp.q.dtype)
        out, lse = run_decode(ops, dataclasses.replace(inp, q=q, scale=scale), 1)
        assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    for scale in (2.0 ** 54 * (1 + 2.0 ** -23), 2.0 ** 55, -2.0 ** 60, float("inf"), -float("inf")):
        with pytest.raises(ops.InklingError):
            run_decode(ops, dataclasses.replace(inp, scale=scale), 1)
