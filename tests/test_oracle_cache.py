"""Pins of the oracle of quantised caches, block selection and drafted tokens: closed forms and torch's own e4m3."""

import math

import numpy as np
import pytest
import torch

from oracle import attention_ref as ar
from oracle import cache_ref as cr


def test_bf16_outwards_brackets_the_value():
    x = np.concatenate([np.random.default_rng(0).normal(size=2000), [0.0, 1.0, -1.0, 1e-40, -1e-40, 3.3895314e38]]).astype(np.float32)
    lo, hi = cr.bf16_down(x), cr.bf16_up(x)
    assert (lo <= x).all() and (hi >= x).all()
    near = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    assert ((lo == near) | (hi == near)).all()              # the nearest value is one of the two
    exact = torch.randn(500, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).float().numpy()
    assert (cr.bf16_down(exact) == exact).all() and (cr.bf16_up(exact) == exact).all()


def test_round_e4m3_is_torchs():
    y = torch.cat([torch.randn(4000, generator=torch.Generator().manual_seed(2)) * s for s in (1e-3, 0.05, 1, 100)]).clamp(-448, 448)
    halves = torch.arange(-900, 901) / 64.0                   # ties among them
    for v in (y, halves):
        assert np.array_equal(cr.round_e4m3(v.numpy()), v.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_quantised_rows(fmt):
    x = torch.randn(50, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).double().numpy()
    x[0] = 0.0
    c, s = cr.quantise(x, fmt)
    a = np.abs(x).max(-1)
    assert s[0] == 0 and not c[0].any()
    if fmt == "int8":       # half a step of the scale, and the scale's own rounding of 127 steps
        assert np.all(np.abs(c * s[:, None].astype(np.float64) - x) <= s[:, None].astype(np.float64) * (0.5 + 127 * 2.0**-24))
        assert np.all(np.abs(c[1:]).max(-1) == 127)
    else:
        assert np.all(a <= 448.0 * s) and np.all(a[1:] > 224.0 * s[1:]) and np.all(np.log2(s[1:]) % 1 == 0)
        err = np.abs(c * s[:, None].astype(np.float64) - x)
        assert np.all(err <= np.maximum(2.0**-4 * np.abs(x), 2.0**-10 * s[:, None]))
    bad = x[1].copy()
    bad[5] = math.inf
    assert math.isnan(cr.row_scale(bad, fmt))


def test_scores_bound_the_keys():
    rng = np.random.default_rng(4)
    K, q = rng.normal(size=(100, 64)).astype(np.float32), rng.normal(size=(1, 64))
    b = cr.block_summary(K, 32, 100)
    s = cr.block_scores(q, b)
    assert b.shape == (4, 2, 64)
    for j in range(4):
        assert s[j] >= (K[32 * j:32 * j + 32] @ q[0]).max()
    assert np.array_equal(b[3], cr.block_summary(K[96:], 32, 4)[0])


def test_scores_are_the_heads_bounds_where_finite():
    rng = np.random.default_rng(6)
    b, q = np.sort(rng.normal(size=(20, 2, 64)), axis=1), rng.normal(size=(3, 64))
    q[0, 5] = 0.0
    heads = np.maximum(q[:, None] * b[None, :, 0], q[:, None] * b[None, :, 1]).sum((0, 2))
    assert np.allclose(cr.block_scores(q, b), heads, rtol=1e-6, atol=1e-6)
    q[:, 7], q[:, 8], q[1, 8] = np.abs(q[:, 7]), -np.abs(q[:, 8]), 0.25
    b[0, 1, 7], b[1, 0, 7], b[2, 1, 8], b[3, 0, 8] = math.inf, -math.inf, math.inf, -math.inf
    s = cr.block_scores(q, b)
    assert s[0] == math.inf and math.isnan(s[1]) and s[2] == math.inf and s[3] == math.inf      # (a negative query, -infinity)
    q[1, 9] = math.nan
    assert np.isnan(cr.block_scores(q, b)).all()


def test_select_blocks_order():
    s = np.array([1.0, 5.0, 5.0, np.nan, 5.0, -2.0], np.float32)
    assert list(cr.select_blocks(s, 6, 2, 0, 0)) == [1, 2]
    assert list(cr.select_blocks(s, 6, 3, 1, 1)) == [0, 1, 5]
    assert list(cr.select_blocks(s, 6, 5, 0, 0)) == [0, 1, 2, 4, 5]          # NaN last
    assert list(cr.select_blocks(s, 3, 5, 1, 1)) == [0, 1, 2, -1, -1]
    assert list(cr.select_blocks(s, 0, 2, 1, 1)) == [-1, -1]


def test_attend_seen_is_the_dense_oracle():
    rng = np.random.default_rng(5)
    q, K, V = rng.normal(size=64), rng.normal(size=(30, 64)), rng.normal(size=(30, 64))
    O, A, S = cr.attend_seen(q, K, V, 0.125)
    assert np.allclose(O, ar.exact_attention(q, K, V, 0.125), rtol=1e-14)
    assert (A >= np.abs(O)).all() and S >= 0.125 * np.abs(K @ q).max()
    assert not cr.attend_seen(q, K[:0], V[:0], 0.125)[0].any()
