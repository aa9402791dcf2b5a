"""Edges of the operators over quantised, block-selected and drafted caches: choices where scores lie close together or are
not finite, numbers near the ends of their types, codes that are no numbers. Tolerances: test_gpu_cache_ops.py."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import cache_ref as cr
from tests.test_gpu_cache_ops import DEV, FMT, QT, api, choose, hold, lib, make_cache, oracle, query, rows, status, up  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- the choice of blocks
def planted(values):
    """f32 scores [B, Hkv, nb] -> (Q, bsum) that have them: three bf16 terms of each value in channels whose query is 1."""
    B, Hkv, nb = values.shape
    bsum = torch.zeros(B, Hkv, nb, 2, 64)
    left = values.clone()
    for c in range(3):
        term = (left.view(torch.int32) & -65536).view(torch.float32)         # cut off to bf16: exact, and so is what is left
        bsum[..., c] = term[..., None]
        left = left - term
    assert (left == 0).all()
    Q = torch.zeros(B, Hkv, 64)
    Q[..., :3] = 1.0
    return Q.to(DEV), bsum.to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("nb, k", [(1000, 100), (1500, 62), (4500, 300)])
@pytest.mark.parametrize("base", [700.0, 1000.0, -3.0])
def test_block_select_over_every_width_of_range(api, nb, k, base):
    """Distinct scores, and many equal ones, in a range of 2^w steps of an f32, w from 1 to 23: each pass of the search, and
    the second look at scores that f32 sums cannot tell apart, over ranges that are no multiple of a pass's bins."""
    g = torch.Generator().manual_seed(nb + k)
    for w in range(1, 24):
        start = torch.tensor(base).view(torch.int32) - (1 << (w - 1))
        v = (start + torch.randint(0, 1 << w, (2, 2, nb), generator=g, dtype=torch.int32)).view(torch.float32)
        v[1, 0, ::2] = v[1, 0, nb // 2]                                      # half of them equal
        v[1, 1] = v[1, 1].sort()[0]
        Q, bsum = planted(v)
        choose(api, Q, bsum, 16 * nb, 16, k, 1, 1)


@pytest.mark.parametrize("block, N, k, spread", [(64, 131072, 100, 5.0), (64, 32768, 62, 5.0), (32, 102400, 97, 16.0), (16, 16000, 100, 1.0)])
def test_block_select_of_scores_with_a_common_part(api, block, N, k, spread):
    """Summaries that share a large channel, as keys with one strong channel do: all scores within part of one power of two."""
    B, Hkv, G, d, nb = 2, 4, 8, 128, N // block
    g = torch.Generator().manual_seed(N + k)
    b = (torch.randn(B, Hkv, nb, 2, d, generator=g).sort(3)[0]).to(torch.bfloat16)
    Q = query(k, "bf16", B, Hkv * G, d)
    s = np.stack([cr.block_scores(Q[0, :G].double().cpu().numpy(), b[0, 0].double().numpy())])
    Q = (Q.float() * (spread / float(s.std()))).to(torch.bfloat16)
    b[..., 0], Q[..., 0] = 11.0, 8.0                                         # 8 heads x 88
    choose(api, Q, b.to(DEV), N, block, k, 1, 1)


def test_block_select_of_queries_that_are_no_numbers(api):
    """A NaN in a query makes every score of its group NaN: the lowest blocks, and the forced ones."""
    g = torch.Generator().manual_seed(9)
    b = torch.randn(1, 2, 300, 2, 64, generator=g).sort(3)[0].to(torch.bfloat16).to(DEV)
    for q in QT:
        Q = query(3, q, 1, 8, 64)
        Q[0, 2, 17] = math.nan                                               # the first group's
        choose(api, Q, b, 4800, 16, 20, 1, 2)
        idx = torch.empty(1, 2, 20, dtype=torch.int32, device=DEV)
        api.block_select(Q, b, 4800, 4800, 16, 1, 2, idx)
        assert idx[0, 0].tolist() == [*range(18), 298, 299]
    Q[0, 2, 17] = math.inf
    choose(api, Q, b, 4800, 16, 20, 1, 2)


@pytest.mark.parametrize("G, d", [(1, 64), (4, 128), (8, 64)])
def test_block_select_of_infinite_summaries(api, G, d):
    """Infinite minima and maxima under queries of either sign, some of them 0: the definition's values, as they are."""
    g = torch.Generator().manual_seed(G)
    B, Hkv, nb = 2, 2, 120
    Q = query(G, "bf16", B, Hkv * G, d)
    Q[0, :, 3] = Q[0, :, 3].abs()
    Q[0, :, 4] = -Q[0, :, 4].abs()
    Q[1, :, 5] = 0.0
    for n in (1, 10, 60, 120):
        b = torch.randn(B, Hkv, nb, 2, d, generator=g).sort(3)[0].to(torch.bfloat16)
        hit = torch.randperm(nb, generator=g)[:n]
        for i, j in enumerate(hit.tolist()):
            c = (3, 4, 5, 7)[i % 4]
            b[:, :, j, 0 if i % 3 else 1, c] = -math.inf if i % 3 else math.inf
            if i % 7 == 0:
                b[:, :, j, :, 9] = torch.tensor([-math.inf, math.inf])
        choose(api, Q, b.to(DEV), 16 * nb, 16, 25, 1, 1)


# ---------------------------------------------------------------- numbers near the ends of their types, and codes that are none
@pytest.mark.parametrize("fmt, q, d, G, T, out", [("int8", "bf16", 128, 4, 4, "f32"), ("e4m3", "f32", 64, 3, 1, "f32"), ("int8", "f32", 128, 8, 3, "bf16"),
                                                  ("e4m3", "bf16", 128, 4, 20, "f32"), ("int8", "bf16", 64, 8, 20, "bf16")])
def test_key_scales_of_any_size(api, fmt, q, d, G, T, out):
    """Scales of seen keys up to 2^115, with queries that bring the logits back to ordinary size, and with ordinary ones, under
    which the largest logit has all the weight."""
    B, Hkv, N = 1, 2, 300
    K, V, sc, Kd, Vd = make_cache(fmt, 97, B, Hkv, up(N + T), d)
    base, k0 = query(9, "f32", B, T, Hkv * G, d), sc[..., 0].clone()
    for qsize, ksize in ((2.0**-112, 2.0**112), (2.0**-100, 2.0**118), (2.0**110, 2.0**-110), (2.0**-20, 2.0**112), (1.0, 2.0**112)):
        Q = (base * qsize).to(QT[q])
        sc[..., 0] = k0 * ksize
        scale = 0.1 if qsize * ksize < 2.0**30 else 1.0
        if qsize * ksize == 2.0**18:
            scale *= 2.0**-18
        seen = lambda b, h, t: slice(0, N + t + 1)                           # noqa: E731
        want, A, S = oracle(Q, Kd * ksize, Vd, seen, scale)
        if S.max() > 1e6:                                                    # one key has all the weight, by far
            for hq in range(Hkv * G):
                x = np.sort(Q[0, -1, hq].double().cpu().numpy() @ (Kd[0, hq // G] * ksize)[:N + T].T)
                assert x[-1] - x[-2] > 2.0**-12 * S[0, -1, hq]
            S = np.zeros_like(S)
        O = torch.empty(B, T, Hkv * G, d, dtype=QT[out], device=DEV)
        api.tree_decode(Q, K, V, N, scale, O, scales=sc)
        if S.max() == 0:
            hold(O[:, -1:], want[:, -1:], A[:, -1:], S[:, -1:], d, N + T, out)
            assert torch.isfinite(O.float()).all()
        else:
            hold(O, want, A, S, d, N + T, out)
        O1 = torch.empty(B, Hkv * G, d, device=DEV)
        api.quant_decode(Q[:, -1].contiguous(), K, V, sc, N + T, scale, O1)
        hold(O1[:, None], want[:, -1:], A[:, -1:], S[:, -1:], d, N + T)


@pytest.mark.parametrize("T, G, d, q, out", [(20, 1, 128, "bf16", "bf16"), (20, 4, 64, "bf16", "f32"), (7, 2, 128, "bf16", "f32"), (20, 8, 128, "bf16", "bf16"),
                                             (100, 8, 128, "bf16", "bf16"), (40, 4, 128, "bf16", "f32"), (20, 4, 128, "f32", "f32"), (100, 1, 64, "f32", "bf16")])
def test_drafts_whose_codes_are_no_numbers(api, lib, T, G, d, q, out):
    """e4m3 codes 0x7f and 0xff in drafted rows: the tokens that see the row have NaN in that channel, nobody else has one."""
    B, Hkv, N = 2, 2, 150
    K, V, sc, Kd, Vd = make_cache("e4m3", 98, B, Hkv, up(N + T), d)
    lens = torch.tensor([N, N - 90], dtype=torch.int32, device=DEV)
    seen = torch.zeros(B, T, T, dtype=torch.bool)
    seen[:, :, ::2] = torch.tril(torch.ones(T, T, dtype=torch.bool))[:, ::2]
    seen[:, 5, 5] = True
    Kd, Vd = Kd.copy(), Vd.copy()
    for b in range(B):
        for i in range(1, T, 2):                                             # nobody sees the odd drafts, but for number 5
            r = int(lens[b]) + i
            V.view(torch.uint8)[b, :, r, i % d] = 0x7F
            V.view(torch.uint8)[b, :, r, (3 * i + 64) % d] = 0xFF
            Vd[b, :, r, i % d] = Vd[b, :, r, (3 * i + 64) % d] = np.nan
            if i != 5:
                K.view(torch.uint8)[b, :, r, (7 * i) % d] = 0xFF
                Kd[b, :, r, (7 * i) % d] = np.nan
    Q = query(10, q, B, T, Hkv * G, d)
    O = torch.empty(B, T, Hkv * G, d, dtype=QT[out], device=DEV)
    api.tree_decode(Q, K, V, N, 0.1, O, mask=api.tree_mask(seen).to(DEV), scales=sc, lens=lens)
    want, A, S = oracle(Q, Kd, Vd, lambda b, h, t: list(range(int(lens[b]))) + [int(lens[b]) + i for i in range(T) if seen[b, t, i]], 0.1)
    none = np.isnan(want)
    assert none[:, 5].sum() == 2 * B * Hkv * G and none.sum() == none[:, 5].sum()
    assert np.array_equal(torch.isnan(O).cpu().numpy(), none)
    hold(torch.nan_to_num(O.float()), np.nan_to_num(want), np.nan_to_num(A), S, d, N + T, out)
    assert status(lib) == 0


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_infinite_values_that_are_seen(api, kv):
    """They show in their channel (infinite or NaN over bf16 caches, infinite over f32 ones) and in no other."""
    B, Hkv, G, d, N, T = 1, 2, 4, 128, 300, 12
    K, V, _, Kd, Vd = make_cache(kv, 99, B, Hkv, up(N + T), d)
    V[0, :, 40, 7], V[0, :, N + 2, 9] = math.inf, -math.inf                  # a cached row, and a draft
    Vd[0, :, 40, 7], Vd[0, :, N + 2, 9] = 0.0, 0.0
    Q = query(11, kv, B, T, Hkv * G, d)
    O = torch.empty(B, T, Hkv * G, d, device=DEV)
    api.tree_decode(Q, K, V, N, 0.1, O)
    want, A, S = oracle(Q, Kd, Vd, lambda b, h, t: slice(0, N + t + 1), 0.1)
    bad = torch.zeros_like(O, dtype=torch.bool)
    bad[..., 7] = True
    bad[:, 2:, :, 9] = True
    assert torch.equal(~torch.isfinite(O), bad)
    assert (O[:, 2:, :, 9] == -math.inf).all()
    if kv == "f32":
        assert (O[..., 7] == math.inf).all()
    at = bad.cpu().numpy()
    hold(O.masked_fill(bad, 0.0), np.where(at, 0.0, want), np.where(at, 0.0, A), S, d, N + T)
    bl = torch.tensor([1, 4], dtype=torch.int32, device=DEV).expand(B, Hkv, 2).contiguous()
    O1 = torch.empty(B, Hkv * G, d, device=DEV)
    api.block_attend(Q[:, 0].contiguous(), K, V, N, 32, bl, 0.1, O1)
    want, A, S = oracle(Q[:, :1], Kd, Vd, lambda b, h, t: [*range(32, 64), *range(128, 160)], 0.1)
    assert torch.equal(~torch.isfinite(O1), bad[:, 0])
    hold(O1[:, None].masked_fill(bad[:, :1], 0.0), np.where(at[:, :1], 0.0, want), np.where(at[:, :1], 0.0, A), S, d, 64)


# ---------------------------------------------------------------- layouts
def test_append_of_a_row_with_odd_strides(api):
    """The stride of a dimension of one says nothing: a row that was computed as a column."""
    Kq, Vq, sc = api.empty_quant(1, 1, 64, 128)
    col = rows(1, 128, 1).to(DEV)
    new = col.T[None, None]
    assert new.stride()[:3] == (1, 1, 1)
    api.quant_append(new, new, Kq, Vq, sc, n_begin=9)
    c, s = cr.quantise(col[:, 0].double().cpu().numpy(), "int8")
    for x, z in ((Kq, 0), (Vq, 1)):
        assert np.array_equal(x[0, 0, 9].double().cpu().numpy(), c) and float(sc[0, 0, 9, z]) == float(s)


# ---------------------------------------------------------------- errors
def test_a_failed_launch_is_reported_once(api, lib):
    """A launch into a capture that has become invalid fails; the calls after it do not report it again."""
    driver = ctypes.CDLL("libcuda.so.1")
    Kq, Vq, sc = api.empty_quant(1, 1, 64, 128)
    new = rows(1, 1, 1, 2, 128).to(DEV)
    O, Q = torch.empty(1, 1, 128, device=DEV), query(1, "bf16", 1, 1, 128)
    ws = torch.empty(api.workspace_bytes(api.OP_QUANT_DECODE, 1, 1, 1, 64, 2, 128), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
    assert driver.cuStreamBeginCapture_v2(handle, 2) == 0
    assert driver.cuStreamSynchronize(handle) == 900                         # not allowed there: the capture is invalid now
    with torch.cuda.stream(s):
        with pytest.raises(RuntimeError, match="quant_append"):
            api.quant_append(new, new, Kq, Vq, sc)
        assert driver.cuStreamEndCapture(handle, ctypes.byref(graph)) == 901
        api.quant_append(new, new, Kq, Vq, sc)
        api.quant_decode(Q, Kq, Vq, sc, 2, 0.1, O, ws=ws)
    s.synchronize()
    assert (sc[0, 0, :2] > 0).all() and status(lib) == 0
