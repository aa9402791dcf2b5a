"""Quantised caches, block selection and drafted tokens -- float64 CPU oracle.

TEST INFRASTRUCTURE: see the package docstring for who may import this.

The definitions are those of the C header: a row's scale and codes (int8 and
e4m3), a block's summary and score, and softmax attention over the keys that a
query row sees (0 where it sees none).
"""

from __future__ import annotations

import math

import numpy as np


def bf16_down(x) -> np.ndarray:
    """The largest bf16 value that is not above f32 x, as float64."""
    x = np.asarray(x, dtype=np.float32)
    bits = x.view(np.uint32)
    cut = (bits & np.uint32(0xFFFF0000)).astype(np.uint32)
    toward_zero = cut.view(np.float32)
    away = (cut + np.uint32(0x10000)).view(np.float32)
    return np.where(toward_zero > x, away, toward_zero).astype(np.float64)


def bf16_up(x) -> np.ndarray:
    return -bf16_down(-np.asarray(x, dtype=np.float32))


def round_e4m3(y) -> np.ndarray:
    """Nearest e4m3 value (ties to even), |y| <= 448: steps of an eighth of the power of two below |y|, 2^-9 at least."""
    y = np.asarray(y, dtype=np.float64)
    e = np.frexp(np.maximum(np.abs(y), 2.0**-6))[1] - 1
    step = np.exp2(e - 3.0)
    return np.rint(y / step) * step


def row_scale(x, fmt: str) -> np.float32:
    """Scale of one row x [d] (exact values as float64)."""
    a = np.max(np.abs(x))
    if not np.all(np.isfinite(x)):
        return np.float32(np.nan)
    if a == 0:
        return np.float32(0)
    if fmt == "int8":
        return np.float32(max(a / 127.0, 2.0**-126))
    e = -126
    while a > 448.0 * 2.0**e:
        e += 1
    return np.float32(2.0**e)


def quantise(x, fmt: str):
    """Rows x [..., d] -> (codes as float64, scales float32 [...]); a value is code * scale."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, x.shape[-1])
    codes, scales = np.zeros_like(flat), np.zeros(len(flat), np.float32)
    for i, r in enumerate(flat):
        s = row_scale(r, fmt)
        scales[i] = s
        if s > 0:
            y = r / np.float64(s)
            codes[i] = np.clip(np.rint(y), -127, 127) if fmt == "int8" else round_e4m3(y)
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1])


def block_summary(K, block: int, N: int) -> np.ndarray:
    """K [N.., d] -> [ceil(N / block), 2, d]: minima rounded down and maxima rounded up to bf16, of the first N keys."""
    K = np.asarray(K, dtype=np.float32)
    out = []
    for j in range(-(-N // block)):
        part = K[j * block:min(N, (j + 1) * block)]
        out.append(np.stack((bf16_down(np.fmin.reduce(part)), bf16_up(np.fmax.reduce(part)))))
    return np.stack(out)


def block_scores(Qg, bsum) -> np.ndarray:
    """Group scores [NB] (float32) of summaries [NB, 2, d] for the group's query rows Qg [G, d]."""
    q = np.asarray(Qg, dtype=np.float64)
    b = np.asarray(bsum, dtype=np.float64)
    neg, pos = np.minimum(q, 0.0).sum(0), np.maximum(q, 0.0).sum(0)
    with np.errstate(invalid="ignore", over="ignore"):       # 0 * infinity is NaN; sums may leave f32
        return (neg * b[:, 0] + pos * b[:, 1]).sum(-1).astype(np.float32)


def select_blocks(scores, nb: int, k: int, n_first: int, n_last: int) -> np.ndarray:
    """The k chosen of the first nb blocks, ascending, then -1."""
    def rank(j):
        forced = j < n_first or j >= nb - n_last
        s = float(scores[j])
        return (not forced, math.inf if math.isnan(s) else -s, math.isnan(s), j)
    chosen = sorted(sorted(range(nb), key=rank)[:k])
    return np.array(chosen + [-1] * (k - len(chosen)), dtype=np.int32)


def attend_seen(q, K, V, scale: float):
    """softmax(q . K^T * scale) . V over the rows given, 0 for none; also the bound's parts (see below).

    Returns (O [d], A [d], S): A = sum_i p_i |v_i|, S = the largest scale * sum_c |q_c k_ic|. An f32 evaluation with
    relative error u per operation is off by at most about A * 2 * (d + 8) * S * u (the logits) + A * 2 * (n + 64) * u
    (the sums).
    """
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    if len(K) == 0:
        return np.zeros(V.shape[-1]), np.zeros(V.shape[-1]), 0.0
    a = (K @ q) * scale
    w = np.exp(a - a.max())
    p = w / w.sum()
    return p @ V, p @ np.abs(V), scale * float((np.abs(K) @ np.abs(q)).max())
