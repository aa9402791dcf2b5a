"""Quantised caches, block selection and drafted tokens against the float64 oracle, through the binding.

Tolerances. Codes, scales, summaries and chosen blocks are equal. An attention output in f32 is held to
    A * (2 (d + 8) S + 2 (n + 64)) * 2^-23 + A * 2^-20
with A = sum_i p_i |v_i| and S = max_i scale sum_c |q_c k_ic| of its row (oracle/cache_ref.py): a logit is d products
and a few scalings, each off by at most S 2^-23 (tensor-core sums may truncate: a whole step, not half), which moves
weights and their sum; the sums over n keys, chained in any order, and their joins; 2^-20 covers exp2 (2 steps on either
side) and weights split into two or three 16-bit terms. With bf16 outputs the weights and the result are rounded to
bf16: 2^-8 A and 2^-8 |O| more.
"""

import math

import numpy as np
import pytest
import torch

from oracle import cache_ref as cr

pytestmark = pytest.mark.gpu

DEV = "cuda"
FMT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
QT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def api():
    from hash_scored_top_b200 import build
    build.build()
    from hash_scored_top_b200 import api as _api
    return _api


@pytest.fixture(scope="module")
def lib(api):
    from hash_scored_top_b200 import _lib
    return _lib


def status(lib):
    return lib.lib.sk_check_status(None)


def up(x):
    return -(-x // 32) * 32


def rows(seed, *shape, spread=0.4):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(spread * torch.randn(*shape[:-1], 1, generator=g))
    return x.to(torch.bfloat16)


def make_cache(kv, seed, B, Hkv, Ncap, d):
    """(K, V, scales or None on the GPU, K and V as float64 numpy)."""
    K, V = rows(seed, B, Hkv, Ncap, d, spread=0.2), rows(seed + 1, B, Hkv, Ncap, d)
    if kv in QT:
        K, V = K.to(QT[kv]), V.to(QT[kv])
        if kv == "f32":
            g = torch.Generator().manual_seed(seed + 2)
            K = K * (1 + 2.0**-12 * torch.rand(K.shape, generator=g))
        return K.to(DEV), V.to(DEV), None, K.double().numpy(), V.double().numpy()
    (kc, ks), (vc, vs) = cr.quantise(K.double().numpy(), kv), cr.quantise(V.double().numpy(), kv)
    s = torch.from_numpy(np.stack((ks, vs), -1)).to(DEV)
    code = [torch.from_numpy(c).to(torch.float32).to(FMT[kv]).to(DEV) for c in (kc, vc)]
    return (*code, s.contiguous(), kc * ks[..., None].astype(np.float64), vc * vs[..., None].astype(np.float64))


def poison(K, V, scales, b, rows_):
    """NaN and infinities in rows that nobody may see."""
    if scales is None:
        K[b, :, rows_], V[b, :, rows_] = math.nan, math.inf
        V[b, :, rows_, ::2] = math.nan
    else:
        scales[b, :, rows_, 0], scales[b, :, rows_, 1] = math.inf, math.nan


def hold(O, want, A, S, d, n, out="f32", floor=0.0):
    """O against the oracle's row by row: arrays [..., d] and S [...]. floor: see test_large_queries_and_keys."""
    O = O.double().cpu().numpy()
    tol = A * ((2 * (d + 8) * S[..., None] + 2 * (n + 64)) * 2.0**-23 + 2.0**-20) + floor
    if out == "bf16":
        tol = tol + 2.0**-8 * (A + np.abs(want))
    bad = np.abs(O - want) > tol
    assert not bad.any() and np.isfinite(O).all(), (float(np.abs(O - want).max()), float((np.abs(O - want) / (tol + 1e-300)).max()))


def oracle(Q, K, V, seen_of, scale):
    """Q [B, T, Hq, d]; seen_of(b, h, t) -> rows of pair (b, h) that token t sees. Returns O, A, S."""
    B, T, Hq, d = Q.shape
    G = Hq // K.shape[1]
    O, A, S = np.zeros((B, T, Hq, d)), np.zeros((B, T, Hq, d)), np.zeros((B, T, Hq))
    Qd = Q.double().cpu().numpy()
    for b in range(B):
        for hq in range(Hq):
            for t in range(T):
                r = seen_of(b, hq // G, t)
                O[b, t, hq], A[b, t, hq], S[b, t, hq] = cr.attend_seen(Qd[b, t, hq], K[b, hq // G][r], V[b, hq // G][r], scale)
    return O, A, S


def query(seed, q, *shape):
    g = torch.Generator().manual_seed(seed)
    return (1.5 * torch.randn(*shape, generator=g)).to(QT[q]).to(DEV)


# ---------------------------------------------------------------- quantised rows
HARD_ROWS = {
    "zeros": lambda d: torch.zeros(d),
    "one": lambda d: torch.eye(d)[3] * 5.0,
    "tiny": lambda d: torch.linspace(-1, 1, d) * 2.0**-120,
    "subnormal": lambda d: torch.linspace(-1, 1, d) * 2.0**-128,
    "huge": lambda d: torch.linspace(-1, 1, d) * 3.0e38,
    "inf": lambda d: torch.cat([torch.tensor([math.inf]), torch.ones(d - 1)]),
    "neg_inf": lambda d: torch.cat([torch.ones(d - 1), torch.tensor([-math.inf])]),
    "nan": lambda d: torch.cat([torch.ones(d // 2), torch.tensor([math.nan]), torch.ones(d - d // 2 - 1)]),
    "ties": lambda d: torch.cat([torch.tensor([127.0]), torch.arange(d - 1) - (d - 1) // 2 + 0.5]),
    "edge448": lambda d: torch.cat([torch.tensor([448.0]), torch.arange(d - 1) * 3.5]),
    "over448": lambda d: torch.cat([torch.tensor([450.0]), torch.arange(d - 1) * 3.25]),
    "steps": lambda d: torch.cat([torch.tensor([256.0]), torch.arange(d - 1) / 512.0]),
}


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 5, 33, 130])
def test_append_and_read(api, lib, fmt, src, d, n):
    B, Hkv, begin = 2, 3, 7
    Ncap = up(n + begin + 9)
    x = [rows(10 + i, B, n, Hkv, d).float() for i in range(2)]
    if src == "f32":
        x = [v * 1.0001 for v in x]
    for i, f in enumerate(HARD_ROWS.values()):
        x[i % 2].view(-1, d)[(5 * i) % (B * n * Hkv)] = f(d)
    x = [v.to(QT[src]) for v in x]
    Kq, Vq, sc = api.empty_quant(B, Hkv, Ncap, d, FMT[fmt])
    Kq.view(torch.uint8).fill_(77), Vq.view(torch.uint8).fill_(78), sc.fill_(-3.0)
    new = [v.to(DEV).transpose(1, 2) for v in x]                            # token-major memory, strided view
    api.quant_append(*new, Kq, Vq, sc, n_begin=begin)
    assert status(lib) == 0
    K, V = (torch.empty(B, Hkv, n, d, dtype=QT[src], device=DEV) for _ in range(2))
    api.quant_read(Kq, Vq, sc, K, V, n_begin=begin)
    for i, (code, back) in enumerate(((Kq, K), (Vq, V))):
        want_c, want_s = cr.quantise(x[i].double().transpose(1, 2).numpy(), fmt)
        got_s = sc[:, :, begin:begin + n, i].cpu().numpy()
        assert np.array_equal(got_s, want_s, equal_nan=True)
        assert np.array_equal(code[:, :, begin:begin + n].float().double().cpu().numpy(), want_c)
        value = torch.from_numpy((want_c * want_s[..., None].astype(np.float64))).to(torch.float32).to(QT[src])
        assert np.array_equal(back.float().cpu().numpy(), value.float().numpy(), equal_nan=True)
        raw = code.view(torch.uint8)
        assert (raw[:, :, :begin] == 77 + i).all() and (raw[:, :, begin + n:] == 77 + i).all()
    assert (sc[:, :, :begin] == -3).all() and (sc[:, :, begin + n:] == -3).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_ragged_append(api, lib, fmt):
    """starts and lens: rows behind a length are left out silently, rows outside the cache are reported."""
    B, Hkv, d, n, Ncap = 5, 2, 64, 40, 64
    x = rows(20, B, Hkv, n, d).to(DEV)
    y = rows(21, B, Hkv, n, d).to(DEV)
    starts = torch.tensor([0, 10, 60, 24, 5], dtype=torch.int32, device=DEV)
    lens = torch.tensor([40, 13, 64, 24, 0], dtype=torch.int32, device=DEV)
    Kq, Vq, sc = api.empty_quant(B, Hkv, Ncap, d, FMT[fmt])
    sc.fill_(-1.0)
    api.quant_append(x, y, Kq, Vq, sc, starts=starts, lens=lens)
    assert status(lib) == 0
    K, V = torch.full((B, Hkv, n, d), 9.0, device=DEV), torch.full((B, Hkv, n, d), 9.0, device=DEV)
    api.quant_read(Kq, Vq, sc, K, V, starts=starts, lens=lens)
    for b in range(B):
        s, e = int(starts[b]), int(lens[b])
        cnt = max(0, min(n, e - s))
        c, ws = cr.quantise(x[b, :, :cnt].double().cpu().numpy(), fmt)
        assert np.array_equal(sc[b, :, s:s + cnt, 0].cpu().numpy(), ws)
        assert np.array_equal(K[b, :, :cnt].cpu().numpy(), (c * ws[..., None].astype(np.float64)).astype(np.float32))
        assert (K[b, :, cnt:] == 9).all() and (V[b, :, cnt:] == 9).all()
        keep = torch.ones(Ncap, dtype=torch.bool)
        keep[s:s + cnt] = False
        assert (sc[b][:, keep] == -1).all()
    # without lens, sequence 2's rows 64 .. and a negative start have no place
    api.quant_append(x, y, Kq, Vq, sc, starts=starts)
    assert status(lib) == 1 and "outside [0, Ncap)" in lib.last_error()
    assert status(lib) == 0
    api.quant_append(x[:, :, :2], y[:, :, :2], Kq, Vq, sc, starts=torch.tensor([-1, 0, 0, 0, 0], dtype=torch.int32, device=DEV))
    assert status(lib) == 1
    assert status(lib) == 0


# ---------------------------------------------------------------- attention over a quantised cache
@pytest.mark.parametrize("N", [1, 15, 16, 17, 100, 1000, 2049])
@pytest.mark.parametrize("fmt, q, d, G", [("int8", "bf16", 128, 4), ("e4m3", "bf16", 128, 8), ("int8", "f32", 64, 3),
                                          ("e4m3", "f32", 128, 1), ("int8", "bf16", 64, 7), ("e4m3", "bf16", 64, 2),
                                          ("int8", "f32", 128, 8)])
def test_quant_decode(api, lib, fmt, q, d, G, N):
    B, Hkv = 3, 2
    Ncap = up(N + 40)
    Kq, Vq, sc, K, V = make_cache(fmt, 100 + N, B, Hkv, Ncap, d)
    Q = query(N, q, B, Hkv * G, d)
    lens = torch.tensor([N, 0, max(1, N // 3)], dtype=torch.int32, device=DEV)
    for b in range(B):
        poison(Kq, Vq, sc, b, slice(int(lens[b]), None))
    scale = 1.0 / math.sqrt(d)
    O = torch.full((B, Hkv * G, d), 5.0, device=DEV)
    api.quant_decode(Q, Kq, Vq, sc, N, scale, O, lens=lens)
    want, A, S = oracle(Q[:, None], K, V, lambda b, h, t: slice(0, int(lens[b])), scale)
    hold(O[:, None], want, A, S, d, N)
    assert (O[1] == 0).all()
    if N <= 100:        # no lens: every sequence has N keys
        sc2 = make_cache(fmt, 100 + N, B, Hkv, Ncap, d)[2]
        api.quant_decode(Q, Kq, Vq, sc2, N, scale, O)
        want, A, S = oracle(Q[:, None], K, V, lambda b, h, t: slice(0, N), scale)
        hold(O[:, None], want, A, S, d, N)
    assert status(lib) == 0


def test_quant_decode_lens_are_clamped(api):
    B, Hkv, d, N = 2, 1, 64, 50
    Kq, Vq, sc, K, V = make_cache("int8", 7, B, Hkv, 64, d)
    Q = query(1, "bf16", B, 4, d)
    O = torch.empty(B, 4, d, device=DEV)
    api.quant_decode(Q, Kq, Vq, sc, N, 0.125, O, lens=torch.tensor([1000, -5], dtype=torch.int32, device=DEV))
    want, A, S = oracle(Q[:, None], K, V, lambda b, h, t: slice(0, N if b == 0 else 0), 0.125)
    hold(O[:, None], want, A, S, d, N)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_scales_of_any_size(api, fmt):
    """Rows of very different magnitude in one cache, up to f32's range: the weights' product with a scale must not leave it."""
    B, Hkv, d, N = 1, 2, 128, 200
    Kq, Vq, sc, K, V = make_cache(fmt, 8, B, Hkv, up(N), d)
    f = np.exp2(np.linspace(-100, 80, up(N)).round()).astype(np.float32)
    sc[..., 1] *= torch.from_numpy(f).to(DEV)
    V = V * f[None, None, :, None].astype(np.float64)
    Q = query(2, "bf16", B, Hkv * 4, d)
    O = torch.empty(B, Hkv * 4, d, device=DEV)
    api.quant_decode(Q, Kq, Vq, sc, N, 0.05, O)
    want, A, S = oracle(Q[:, None], K, V, lambda b, h, t: slice(0, N), 0.05)
    hold(O[:, None], want, A, S, d, N)


@pytest.mark.parametrize("k", [1, 5, 16, 100, 333])
@pytest.mark.parametrize("fmt, q, d, G", [("int8", "bf16", 128, 4), ("e4m3", "f32", 64, 8), ("e4m3", "bf16", 128, 1)])
def test_quant_sparse_attend(api, lib, fmt, q, d, G, k):
    B, Hkv, N = 2, 3, 640
    Kq, Vq, sc, K, V = make_cache(fmt, 30, B, Hkv, N, d)
    Q = query(k, q, B, Hkv * G, d)
    g = torch.Generator().manual_seed(k)
    idx = torch.stack([torch.randperm(N, generator=g)[:k] for _ in range(B * Hkv)]).view(B, Hkv, k).int()
    if k >= 5:
        idx[0, 0, 1], idx[0, 0, 3], idx[0, 0, 4] = -1, N, 2**31 - 1         # left out
        idx[1, 2, 1] = idx[1, 2, 0]                                          # counts twice
    idx[1, 1] = -1                                                           # nothing listed
    dead = sorted(set(range(N)) - set(idx.flatten().tolist()))
    for b in range(B):
        poison(Kq, Vq, sc, b, dead)
    O = torch.empty(B, Hkv * G, d, device=DEV)
    api.quant_sparse_attend(Q, Kq, Vq, sc, idx.to(DEV), 0.09, O)
    want, A, S = oracle(Q[:, None], K, V, lambda b, h, t: [r for r in idx[b, h].tolist() if 0 <= r < N], 0.09)
    hold(O[:, None], want, A, S, d, k)
    assert (O[1, G:2 * G] == 0).all() and status(lib) == 0


@pytest.mark.parametrize("fmt, N, k", [("int8", 1000, 64), ("e4m3", 4096, 128)])
def test_socket_decode_quant(api, lib, fmt, N, k):
    B, Hkv, G, d, L, P, tau = 2, 2, 4, 128, 8, 4, 0.5
    Kq, Vq, sc, K, V = make_cache(fmt, 40, B, Hkv, up(N), d)
    Kb, Vb = torch.from_numpy(K).to(torch.bfloat16).to(DEV), torch.from_numpy(V).to(torch.bfloat16).to(DEV)
    R = torch.randn(L * P, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    ids, norms = api.empty_ids(B, Hkv, up(N), L), api.empty_norms(B, Hkv, up(N))
    api.socket_hash_keys(Kb, Vb, R, L, P, ids, norms)
    Q = query(3, "bf16", B, Hkv * G, d)
    O, O2 = torch.empty(B, Hkv * G, d, device=DEV), torch.empty(B, Hkv * G, d, device=DEV)
    idx, idx2 = (torch.empty(B, Hkv, k, dtype=torch.int32, device=DEV) for _ in range(2))
    api.socket_decode_quant(Q, Kq, Vq, sc, R, ids, norms, N, L, P, tau, k, 0.09, O, idx_out=idx)
    api.socket_select(Q, R, ids, norms, N, L, P, tau, k, idx2)
    api.quant_sparse_attend(Q, Kq, Vq, sc, idx2, 0.09, O2)
    assert torch.equal(idx, idx2) and torch.equal(O, O2)
    want, A, S = oracle(Q[:, None], K, V, lambda b, h, t: idx[b, h].tolist(), 0.09)
    hold(O[:, None], want, A, S, d, k)
    O.zero_()
    api.socket_decode_quant(Q, Kq, Vq, sc, R, ids, norms, N, L, P, tau, k, 0.09, O)      # the list stays inside
    assert torch.equal(O, O2) and status(lib) == 0


# ---------------------------------------------------------------- blocks
@pytest.mark.parametrize("kv", ["bf16", "f32", "int8", "e4m3"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_block_summarize(api, kv, block, d):
    B, Hkv, N = 2, 2, 205
    Ncap = up(N)
    K, _, sc, Kd, _ = make_cache(kv, 50, B, Hkv, Ncap, d)
    poison(K, K.clone(), sc, slice(None), slice(N, None))
    Kf = Kd.astype(np.float32)
    bsum = api.empty_block_summaries(B, Hkv, Ncap, d, block)
    bsum.fill_(7.0)
    api.block_summarize(K, block, bsum, n_count=N, scales=sc)
    nb = -(-N // block)
    for b in range(B):
        for h in range(Hkv):
            assert np.array_equal(bsum[b, h, :nb].double().cpu().numpy(), cr.block_summary(Kf[b, h], block, N))
    assert (bsum[:, :, nb:] == 7).all()
    # row by row, from every start, to the same summaries; ragged sequences
    part = api.empty_block_summaries(B, Hkv, Ncap, d, block)
    part.fill_(7.0)
    for n in (0, 1, 15, 16, 17, 130, N - 1):
        starts = torch.tensor([n, max(0, n - 9)], dtype=torch.int32, device=DEV)
        lens = starts + 1
        api.block_summarize(K, block, part, n_count=3, scales=sc, starts=starts, lens=lens)
        for b in range(B):
            j = int(starts[b]) // block
            want = cr.block_summary(Kf[b, 1], block, int(lens[b]))[j]
            assert np.array_equal(part[b, 1, j].double().cpu().numpy(), want)
    before = part.clone()
    api.block_summarize(K, block, part, n_count=5, scales=sc, starts=torch.tensor([N, 40], dtype=torch.int32, device=DEV),
                        lens=torch.tensor([N, 40], dtype=torch.int32, device=DEV))       # no rows
    assert torch.equal(part, before)


def test_block_summarize_passes_over_nan(api):
    K = rows(51, 1, 1, 64, 64).to(DEV)
    Kf = K[0, 0].float().cpu().numpy().copy()
    K[0, 0, 3, 5] = math.nan
    Kf[3, 5] = np.nan
    K[0, 0, 40, 2], Kf[40, 2] = math.inf, np.inf
    bsum = api.empty_block_summaries(1, 1, 64, 64, 32)
    api.block_summarize(K, 32, bsum)
    assert np.array_equal(bsum[0, 0].double().cpu().numpy(), cr.block_summary(Kf, 32, 64))


@pytest.mark.parametrize("block, N, k, first, last", [(16, 1, 1, 0, 0), (16, 40, 2, 1, 1), (16, 500, 8, 1, 1), (32, 2000, 17, 0, 2),
                                                      (64, 700, 11, 2, 0), (64, 700, 20, 1, 1), (128, 5000, 3, 0, 0), (16, 20000, 300, 1, 4)])
@pytest.mark.parametrize("q, d, G", [("bf16", 128, 4), ("f32", 64, 8), ("bf16", 64, 1)])
def test_block_select(api, block, N, k, first, last, q, d, G):
    B, Hkv = 3, 2
    Ncap = up(N + 70)
    NB = -(-Ncap // block)
    g = torch.Generator().manual_seed(N)
    a, b_ = torch.randn(2, B, Hkv, NB, d, generator=g)
    bsum = torch.stack((torch.minimum(a, b_), torch.maximum(a, b_)), 3).to(torch.bfloat16)
    if NB > 6:
        bsum[:, :, 5] = bsum[:, :, 3]                                        # equal scores: the lower block
        bsum[:, :, 4, 1, 0] = math.nan
        bsum[0, 0, 2, 1] = math.inf
    Q = query(N + 1, q, B, Hkv * G, d)
    lens = torch.tensor([N, max(0, N // 2 - 3), 0], dtype=torch.int32, device=DEV)
    idx = torch.empty(B, Hkv, k, dtype=torch.int32, device=DEV)
    api.block_select(Q, bsum.to(DEV), Ncap, N, block, first, last, idx, lens=lens)
    Qd = Q.double().cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            with np.errstate(invalid="ignore"):
                s = cr.block_scores(Qd[b, h * G:(h + 1) * G], bsum[b, h].double().numpy())
            if NB > 6:
                s[4] = np.nan
                if b == 0 and h == 0:
                    q_ = Qd[b, :G]
                    s[2] = np.inf if (np.maximum(q_, 0).sum(0) > 0).all() else np.nan          # 0 * inf
            want = cr.select_blocks(s, -(-int(lens[b]) // block), k, first, last)
            assert np.array_equal(idx[b, h].cpu().numpy(), want), (b, h)


def test_block_select_all_equal(api):
    """Every score the same: the lowest blocks, and the forced ones."""
    B, Hkv, d, N, block, k = 1, 1, 64, 4000, 16, 9
    bsum = torch.ones(B, Hkv, 250, 2, d, dtype=torch.bfloat16, device=DEV)
    idx = torch.empty(B, Hkv, k, dtype=torch.int32, device=DEV)
    api.block_select(query(1, "bf16", B, 4, d), bsum, N, N, block, 0, 2, idx)
    assert idx[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 248, 249]


@pytest.mark.parametrize("kv, q, d, G, block", [("bf16", "bf16", 128, 4, 32), ("bf16", "bf16", 64, 8, 16), ("f32", "f32", 128, 2, 64),
                                                ("int8", "bf16", 128, 5, 16), ("e4m3", "f32", 64, 4, 128), ("int8", "f32", 64, 1, 32),
                                                ("bf16", "bf16", 128, 1, 128), ("e4m3", "bf16", 128, 8, 64)])
@pytest.mark.parametrize("k", [1, 3, 10])
def test_block_attend(api, lib, kv, q, d, G, block, k):
    B, Hkv, N = 3, 2, 1003
    Ncap = up(N)
    K, V, sc, Kd, Vd = make_cache(kv, 60, B, Hkv, Ncap, d)
    lens = torch.tensor([N, 333, 0], dtype=torch.int32, device=DEV)
    for b in range(B):
        poison(K, V, sc, b, slice(int(lens[b]), None))
    nb = -(-N // block)
    g = torch.Generator().manual_seed(k)
    idx = torch.stack([torch.randperm(nb, generator=g)[:k] if k <= nb else torch.arange(k) % nb for _ in range(B * Hkv)]).view(B, Hkv, k).int()
    idx[0, 0, 0] = nb - 1                                                    # the partly filled block
    if k == 10:
        idx[0, 1, 2], idx[0, 1, 3], idx[0, 1, 4] = -1, nb + 5, 2**31 - 1      # left out
        idx[1, 0, 1] = idx[1, 0, 0]
    Q = query(k, q, B, Hkv * G, d)
    O = torch.empty(B, Hkv * G, d, device=DEV)
    api.block_attend(Q, K, V, N, block, idx.to(DEV), 0.1, O, scales=sc, lens=lens)

    def seen(b, h, t):
        n = int(lens[b])
        return [r for j in idx[b, h].tolist() if j >= 0 for r in range(j * block, min(n, (j + 1) * block))]
    want, A, S = oracle(Q[:, None], Kd, Vd, seen, 0.1)
    hold(O[:, None], want, A, S, d, k * block)
    assert (O[2] == 0).all() and status(lib) == 0


@pytest.mark.parametrize("kv", ["bf16", "f32", "int8", "e4m3"])
def test_block_decode(api, lib, kv):
    B, Hkv, G, d, N, block, k = 2, 3, 4, 128, 1500, 32, 9
    K, V, sc, Kd, Vd = make_cache(kv, 70, B, Hkv, up(N), d)
    q = "f32" if kv == "f32" else "bf16"
    Q = query(4, q, B, Hkv * G, d)
    lens = torch.tensor([N, 700], dtype=torch.int32, device=DEV)
    bsum = api.empty_block_summaries(B, Hkv, up(N), d, block)
    api.block_summarize(K, block, bsum, n_count=N, scales=sc, lens=lens)
    O, O2 = torch.empty(B, Hkv * G, d, device=DEV), torch.empty(B, Hkv * G, d, device=DEV)
    idx, idx2 = (torch.empty(B, Hkv, k, dtype=torch.int32, device=DEV) for _ in range(2))
    api.block_decode(Q, K, V, bsum, N, block, k, 1, 1, 0.08, O, scales=sc, lens=lens, idx_out=idx)
    api.block_select(Q, bsum, up(N), N, block, 1, 1, idx2, lens=lens)
    api.block_attend(Q, K, V, N, block, idx2, 0.08, O2, scales=sc, lens=lens)
    assert torch.equal(idx, idx2) and torch.equal(O, O2)

    def seen(b, h, t):
        return [r for j in idx[b, h].tolist() for r in range(j * block, min(int(lens[b]), (j + 1) * block))]
    want, A, S = oracle(Q[:, None], Kd, Vd, seen, 0.08)
    hold(O[:, None], want, A, S, d, k * block)
    assert status(lib) == 0


# ---------------------------------------------------------------- drafted tokens
def random_tree(seed, B, T):
    g = torch.Generator().manual_seed(seed)
    seen = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            p = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            if p >= 0:
                seen[b, t] = seen[b, p]
            seen[b, t, t] = True
    return seen


TREES = [(kv, q, d, G, T, N, out) for kv, q, d, G in (("bf16", "bf16", 128, 4), ("bf16", "bf16", 64, 1), ("f32", "f32", 64, 2),
                                                      ("int8", "bf16", 128, 8), ("e4m3", "f32", 64, 5), ("int8", "f32", 64, 3),
                                                      ("bf16", "bf16", 128, 8), ("e4m3", "bf16", 128, 1))
         for T, N, out in ((1, 128, "f32"), (2, 0, "f32"), (7, 300, "bf16"), (33, 1, "f32"), (16, 129, "bf16"), (40, 513, "f32"))]
TREES += [("bf16", "bf16", 128, 4, 100, 200, "bf16"), ("bf16", "bf16", 64, 8, 70, 77, "f32"), ("int8", "bf16", 64, 2, 256, 40, "bf16"),
          ("bf16", "bf16", 64, 2, 256, 260, "bf16"), ("bf16", "bf16", 128, 4, 5, 3000, "f32"), ("e4m3", "bf16", 128, 4, 24, 1500, "f32")]


TREES += [("int8", "f32", 128, 4, 16, 700, "f32"), ("e4m3", "f32", 128, 8, 40, 333, "bf16"), ("int8", "f32", 64, 2, 5, 4000, "f32"),
          ("e4m3", "f32", 64, 8, 100, 90, "bf16"), ("int8", "f32", 128, 1, 1, 4097, "f32")]


@pytest.mark.parametrize("kv, q, d, G, T, N, out", TREES)
def test_tree_decode(api, lib, kv, q, d, G, T, N, out):
    B, Hkv = 2, 2
    Ncap = up(N + T + 1)
    K, V, sc, Kd, Vd = make_cache(kv, 80 + T, B, Hkv, Ncap, d)
    lens = torch.tensor([N, N // 3], dtype=torch.int32, device=DEV)
    for b in range(B):
        poison(K, V, sc, b, slice(int(lens[b]) + T, None))
    seen = random_tree(T, B, T)
    seen[1, T - 1] = False                                                   # a token that sees no draft, not even itself
    Q = query(T, q, B, T, Hkv * G, d)
    O = torch.full((B, T, Hkv * G, d), 3.0, dtype=QT[out], device=DEV)
    mask = api.tree_mask(seen)
    if T % 32:
        mask[..., -1] |= -1 << (T % 32)                                      # bits past T are ignored
    api.tree_decode(Q, K, V, N, 0.11, O, mask=mask.to(DEV), scales=sc, lens=lens)

    def rows_of(b, h, t):
        n = int(lens[b])
        return list(range(n)) + [n + i for i in range(T) if seen[b, t, i]]
    want, A, S = oracle(Q, Kd, Vd, rows_of, 0.11)
    hold(O, want, A, S, d, N + T, out)
    if N // 3 == 0:
        assert (O[1, T - 1] == 0).all()
    assert status(lib) == 0


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_tree_decode_chain_and_hidden_drafts(api, kv):
    """No mask: a chain. A draft of NaN and infinities reaches the tokens that see it and no other."""
    B, Hkv, G, d, T, N = 1, 2, 4, 128, 20, 150
    K, V, sc, Kd, Vd = make_cache(kv, 90, B, Hkv, up(N + T), d)
    Q = query(5, "bf16", B, T, Hkv * G, d)
    O = torch.empty(B, T, Hkv * G, d, device=DEV)
    poison(K, V, sc, 0, slice(N + 12, None))
    api.tree_decode(Q, K, V, N, 0.1, O, scales=sc)
    want, A, S = oracle(Q[:, :12], Kd, Vd, lambda b, h, t: slice(0, N + t + 1), 0.1)
    hold(O[:, :12], want, A, S, d, N + T)
    assert torch.isnan(O[:, 12:]).any(-1).all()


@pytest.mark.parametrize("T, G, out", [(20, 1, "bf16"), (20, 4, "bf16"), (20, 8, "bf16"), (40, 8, "bf16"), (20, 4, "f32"), (7, 2, "f32"),
                                       (30, 5, "f32")])
@pytest.mark.parametrize("kv", ["bf16", "int8", "e4m3"])
def test_tree_decode_hidden_drafts_of_any_size(api, kv, T, G, out, q="bf16"):
    """Drafts 2^100 times the others' size do not change what the tokens that do not see them get."""
    B, Hkv, d, N = 1, 2, 128, 150
    K, V, sc, Kd, Vd = make_cache(kv, 95, B, Hkv, up(N + T), d)
    big = slice(N + 1, N + T, 2)                                             # the odd drafts
    if sc is None:
        K[:, :, big] *= 2.0**100
        V[:, :, big] *= 2.0**100
    else:
        sc[:, :, big] *= 2.0**100
    Q = query(8, q, B, T, Hkv * G, d)
    seen = torch.zeros(B, T, T, dtype=torch.bool)
    seen[:, :, ::2] = torch.tril(torch.ones(T, T, dtype=torch.bool))[:, ::2]
    O = torch.empty(B, T, Hkv * G, d, dtype=QT[out], device=DEV)
    api.tree_decode(Q, K, V, N, 0.1, O, scales=sc, mask=api.tree_mask(seen).to(DEV))
    want, A, S = oracle(Q, Kd, Vd, lambda b, h, t: list(range(N)) + [N + i for i in range(T) if seen[b, t, i]], 0.1)
    hold(O, want, A, S, d, N + T, out)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
def test_tree_decode_hidden_drafts_under_f32_queries(api, kv):
    test_tree_decode_hidden_drafts_of_any_size(api, kv, 20, 4, "f32", q="f32")


def test_tree_of_one_token_is_quant_decode(api):
    B, Hkv, G, d, N = 2, 2, 4, 128, 777
    K, V, sc, Kd, Vd = make_cache("int8", 91, B, Hkv, up(N), d)
    Q = query(6, "bf16", B, 1, Hkv * G, d)
    O1, O2 = torch.empty(B, 1, Hkv * G, d, device=DEV), torch.empty(B, Hkv * G, d, device=DEV)
    api.tree_decode(Q, K, V, N - 1, 0.1, O1, scales=sc)
    api.quant_decode(Q[:, 0], K, V, sc, N, 0.1, O2)
    want, A, S = oracle(Q, Kd, Vd, lambda b, h, t: slice(0, N), 0.1)
    hold(O1, want, A, S, d, N)
    hold(O2[:, None], want, A, S, d, N)


# ---------------------------------------------------------------- together, graphs, streams, sizes
def test_a_serving_loop(api, lib):
    """A prompt, then steps of append, summarise and block decode, then a drafted tree, all on one quantised cache."""
    B, Hkv, G, d, block, k = 2, 2, 4, 64, 16, 6
    n0, steps, T = [70, 33], 5, 6
    Ncap = 128
    Kt, Vt = rows(200, B, Hkv, Ncap, d), rows(201, B, Hkv, Ncap, d)
    qk, ks = cr.quantise(Kt.double().numpy(), "int8")
    qv, vs = cr.quantise(Vt.double().numpy(), "int8")
    Kd, Vd = qk * ks[..., None].astype(np.float64), qv * vs[..., None].astype(np.float64)
    Kq, Vq, sc = api.empty_quant(B, Hkv, Ncap, d)
    bsum = api.empty_block_summaries(B, Hkv, Ncap, d, block)
    Kt, Vt = Kt.to(DEV), Vt.to(DEV)
    lens = torch.tensor(n0, dtype=torch.int32, device=DEV)
    api.quant_append(Kt[:, :, :max(n0)], Vt[:, :, :max(n0)], Kq, Vq, sc, lens=lens)
    api.block_summarize(Kq, block, bsum, n_count=max(n0), scales=sc, lens=lens)
    O = torch.empty(B, Hkv * G, d, device=DEV)
    idx = torch.empty(B, Hkv, k, dtype=torch.int32, device=DEV)
    at = torch.arange(B, device=DEV)
    for s in range(steps):
        new_k, new_v = (x[at, :, lens.long()][:, :, None].contiguous() for x in (Kt, Vt))
        starts, lens = lens, lens + 1
        api.quant_append(new_k, new_v, Kq, Vq, sc, starts=starts)
        api.block_summarize(Kq, block, bsum, n_count=1, scales=sc, starts=starts, lens=lens)
        Q = query(300 + s, "bf16", B, Hkv * G, d)
        api.block_decode(Q, Kq, Vq, bsum, Ncap, block, k, 1, 1, 0.125, O, scales=sc, lens=lens, idx_out=idx)
        Qd = Q.double().cpu().numpy()
        for b in range(B):
            n = int(lens[b])
            for h in range(Hkv):
                sums = cr.block_summary(Kd[b, h].astype(np.float32), block, n)
                assert np.array_equal(bsum[b, h, :len(sums)].double().cpu().numpy(), sums)
                want = cr.select_blocks(cr.block_scores(Qd[b, h * G:(h + 1) * G], sums), len(sums), k, 1, 1)
                assert np.array_equal(idx[b, h].cpu().numpy(), want)

        def seen(b, h, t):
            return [r for j in idx[b, h].tolist() if j >= 0 for r in range(j * block, min(int(lens[b]), (j + 1) * block))]
        want, A, S = oracle(Q[:, None], Kd, Vd, seen, 0.125)
        hold(O[:, None], want, A, S, d, k * block)
    drafts = torch.stack([torch.arange(int(lens[b]), int(lens[b]) + T) for b in range(B)]).to(DEV)
    api.quant_append(*(torch.stack([x[b, :, drafts[b]] for b in range(B)]) for x in (Kt, Vt)), Kq, Vq, sc, starts=lens)
    tree = random_tree(9, B, T)
    Q = query(400, "bf16", B, T, Hkv * G, d)
    Ot = torch.empty(B, T, Hkv * G, d, device=DEV)
    api.tree_decode(Q, Kq, Vq, Ncap - T, 0.125, Ot, mask=api.tree_mask(tree).to(DEV), scales=sc, lens=lens)
    want, A, S = oracle(Q, Kd, Vd, lambda b, h, t: list(range(int(lens[b]))) + [int(lens[b]) + i for i in range(T) if tree[b, t, i]], 0.125)
    hold(Ot, want, A, S, d, Ncap)
    assert status(lib) == 0


def test_captured_steps(api, lib):
    """Two graphs (a decode step and a drafted step) that share one workspace, replayed with other lengths and inputs."""
    B, Hkv, G, d, block, k, T, Ncap = 2, 2, 4, 128, 32, 4, 9, 512
    K, V, sc, Kd, Vd = make_cache("e4m3", 500, B, Hkv, Ncap, d)
    Kb, Vb = (torch.from_numpy(x).to(torch.bfloat16).to(DEV) for x in (Kd, Vd))      # exact: the codes times a power of two
    Kq, Vq, s2 = api.empty_quant(B, Hkv, Ncap, d, torch.float8_e4m3fn)
    bsum = api.empty_block_summaries(B, Hkv, Ncap, d, block)
    lens, starts = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    new = [torch.zeros(B, Hkv, 1, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    Q, Qt = query(1, "bf16", B, Hkv * G, d), query(2, "bf16", B, T, Hkv * G, d)
    Od, Ob = torch.empty(B, Hkv * G, d, device=DEV), torch.empty(B, Hkv * G, d, device=DEV)
    Ot = torch.empty(B, T, Hkv * G, d, device=DEV)
    tree = random_tree(3, B, T)
    mask = api.tree_mask(tree).to(DEV)
    size = max(api.workspace_bytes(api.OP_QUANT_DECODE, B, Hkv * G, Hkv, Ncap, Ncap, d),
               api.workspace_bytes(api.OP_BLOCK_DECODE, B, Hkv * G, Hkv, Ncap, Ncap, d, block, 0, k),
               api.workspace_bytes(api.OP_TREE_DECODE, B, Hkv * G, Hkv, Ncap, Ncap - T, d, 0, 0, T))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)             # a workspace of NaN

    def step():
        api.quant_append(*new, Kq, Vq, s2, starts=starts)
        api.block_summarize(Kq, block, bsum, n_count=1, scales=s2, starts=starts, lens=lens)
        api.quant_decode(Q, Kq, Vq, s2, Ncap, 0.09, Od, lens=lens, ws=ws)
        api.block_decode(Q, Kq, Vq, bsum, Ncap, block, k, 1, 1, 0.09, Ob, scales=s2, lens=lens, ws=ws)

    def drafted():
        api.tree_decode(Qt, K, V, Ncap - T, 0.09, Ot, mask=mask, scales=sc, lens=lens, ws=ws)

    graphs = []
    for f in (step, drafted):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            f()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    at = torch.arange(B, device=DEV)
    n = torch.tensor([130, 96], dtype=torch.int32, device=DEV)
    api.quant_append(Kb[:, :, :130], Vb[:, :, :130], Kq, Vq, s2, lens=n)
    api.block_summarize(Kq, block, bsum, n_count=130, scales=s2, lens=n)
    for r in range(3):
        starts.copy_(n + r)
        lens.copy_(n + r + 1)
        for x, src in zip(new, (Kb, Vb)):
            x.copy_(src[at, :, starts.long()][:, :, None])
        Q.copy_(query(20 + r, "bf16", B, Hkv * G, d))
        Qt.copy_(query(30 + r, "bf16", B, T, Hkv * G, d))
        graphs[0].replay()
        graphs[1].replay()
        ln = lens.tolist()
        want, A, S = oracle(Q[:, None], Kd, Vd, lambda b, h, t: slice(0, ln[b]), 0.09)
        hold(Od[:, None], want, A, S, d, Ncap)
        Qd = Q.double().cpu().numpy()

        def seen(b, h, t):
            sums = cr.block_summary(Kd[b, h].astype(np.float32), block, ln[b])
            ids = cr.select_blocks(cr.block_scores(Qd[b, h * G:(h + 1) * G], sums), len(sums), k, 1, 1)
            return [i for j in ids if j >= 0 for i in range(j * block, min(ln[b], (j + 1) * block))]
        want, A, S = oracle(Q[:, None], Kd, Vd, seen, 0.09)
        hold(Ob[:, None], want, A, S, d, Ncap)
        want, A, S = oracle(Qt, Kd, Vd, lambda b, h, t: list(range(ln[b])) + [ln[b] + i for i in range(T) if tree[b, t, i]], 0.09)
        hold(Ot, want, A, S, d, Ncap)
    assert status(lib) == 0


def test_repeats_and_other_streams_give_the_same_bits(api):
    B, Hkv, G, d, N, T = 2, 4, 4, 128, 3000, 12
    K, V, sc, _, _ = make_cache("int8", 600, B, Hkv, up(N + T), d)
    Kb, Vb, _, _, _ = make_cache("bf16", 601, B, Hkv, up(N + T), d)
    Q, Qt = query(1, "bf16", B, Hkv * G, d), query(2, "bf16", B, T, Hkv * G, d)
    bsum = api.empty_block_summaries(B, Hkv, up(N + T), d, 16)
    api.block_summarize(Kb, 16, bsum, n_count=N)

    def all_of():
        outs = [torch.empty(B, Hkv * G, d, device=DEV) for _ in range(2)] + [torch.empty(B, T, Hkv * G, d, device=DEV) for _ in range(2)]
        api.quant_decode(Q, K, V, sc, N, 0.1, outs[0])
        api.block_decode(Q, Kb, Vb, bsum, N, 16, 20, 1, 1, 0.1, outs[1])
        api.tree_decode(Qt, K, V, N, 0.1, outs[2], scales=sc)
        api.tree_decode(Qt, Kb, Vb, N, 0.1, outs[3])
        return outs
    first = all_of()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:                       # both at once, each with workspaces of its own
        with torch.cuda.stream(s):
            for _ in range(3):
                got.append(all_of())
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(first, outs):
            assert torch.equal(a, b)


def test_offsets_past_32_bits(api, lib):
    """A cache of more than 2^32 bytes: the last row of the last pair carries all the weight."""
    B, Hkv, G, d, T = 1, 3, 2, 128, 3
    Ncap = 11534336                                                          # 3 pairs x 11.5 M rows x 128 B = 4.4 GB
    if torch.cuda.get_device_properties(0).total_memory < 24 << 30:
        pytest.skip("needs 24 GB")
    Kq, Vq, sc = api.empty_quant(B, Hkv, Ncap, d)
    hot = torch.ones(B, Hkv, 1, d, dtype=torch.bfloat16, device=DEV)
    val = rows(700, B, Hkv, 1, d).to(DEV)
    N = Ncap - 40 - T
    api.quant_append(20 * hot, val, Kq, Vq, sc, n_begin=N - 1)
    want = torch.empty(B, Hkv, 1, d, device=DEV)
    api.quant_read(Kq, Vq, sc, torch.empty_like(want), want, n_begin=N - 1)
    ref = cr.quantise(val.double().cpu().numpy(), "int8")
    assert np.array_equal(want.cpu().numpy(), (ref[0] * ref[1][..., None].astype(np.float64)).astype(np.float32))
    Q = torch.ones(B, Hkv * G, d, dtype=torch.bfloat16, device=DEV)
    O = torch.empty(B, Hkv * G, d, device=DEV)
    expect = want.repeat_interleave(G, 1)[:, :, 0]

    def same():     # weight of the other keys: N e^-226; the sum of 128 products and the weights are exact here but for exp2's steps
        assert (O - expect).abs().max() <= 2.0**-20 * expect.abs().max()
        O.zero_()
    api.quant_decode(Q, Kq, Vq, sc, N, 1 / math.sqrt(d), O)
    same()
    api.quant_sparse_attend(Q, Kq, Vq, sc, torch.tensor([[[0, N - 1, 5]] * Hkv], dtype=torch.int32, device=DEV), 1 / math.sqrt(d), O)
    same()
    bl = torch.tensor([[[1, (N - 1) // 64]] * Hkv], dtype=torch.int32, device=DEV)
    api.block_attend(Q, Kq, Vq, N, 64, bl, 1 / math.sqrt(d), O, scales=sc)
    same()
    bsum = api.empty_block_summaries(B, Hkv, Ncap, d, 64)
    api.block_summarize(Kq, 64, bsum, n_count=N, scales=sc)
    idx = torch.empty(B, Hkv, 2, dtype=torch.int32, device=DEV)
    api.block_decode(Q, Kq, Vq, bsum, N, 64, 2, 0, 0, 1 / math.sqrt(d), O, scales=sc, idx_out=idx)
    same()
    assert idx[0, :, 1].tolist() == [(N - 1) // 64] * Hkv
    Ot = torch.empty(B, T, Hkv * G, d, device=DEV)
    api.tree_decode(Q[:, None].expand(B, T, Hkv * G, d).contiguous(), Kq, Vq, N, 1 / math.sqrt(d), Ot, scales=sc)
    for t in range(T):
        O.copy_(Ot[:, t])
        same()
    assert status(lib) == 0


# ---------------------------------------------------------------- the choice of blocks where it is hard
def choose(api, Q, bsum, N, block, k, first=0, last=0):
    B, Hkv = bsum.shape[:2]
    idx = torch.full((B, Hkv, k), -7, dtype=torch.int32, device=DEV)
    api.block_select(Q, bsum, N, N, block, first, last, idx)
    Qd, G = Q.double().cpu().numpy(), Q.shape[1] // Hkv
    b = bsum.double().cpu().numpy()
    for i in range(B):
        for h in range(Hkv):
            with np.errstate(invalid="ignore"):
                s = cr.block_scores(Qd[i, h * G:(h + 1) * G], b[i, h])
            want = cr.select_blocks(s, -(-N // block), k, first, last)
            assert np.array_equal(idx[i, h].cpu().numpy(), want), (i, h)


@pytest.mark.parametrize("N, block, k", [(102400, 16, 500), (1048576, 16, 77), (1048576, 16, 70000), (70016, 16, 4376)])
def test_block_select_of_many_blocks(api, N, block, k):
    """More blocks than registers hold, than shared memory holds, and k beyond them all."""
    g = torch.Generator(device=DEV).manual_seed(k)
    b = torch.randn(1, 1, N // block, 2, 64, generator=g, device=DEV).sort(3)[0].to(torch.bfloat16)
    choose(api, query(1, "bf16", 1, 2, 64), b, N, block, k, 1, 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k", [3, 64, 100, 255])
def test_block_select_near_ties(api, d, k):
    """Scores that differ by less than f32 sums can tell, and equal ones: the choice is the exact sums'."""
    B, Hkv, nb = 2, 2, 256
    g = torch.Generator().manual_seed(k)
    base = torch.randn(B, Hkv, 1, 2, d, generator=g).sort(3)[0].expand(B, Hkv, nb, 2, d).to(torch.bfloat16).clone()
    # the last bit of a few small channels, in some blocks
    bits = base.view(torch.int16)
    small = base.float().abs().flatten(3).argsort(-1)[..., :3]
    flip = torch.randint(0, 2, small.shape, generator=g).to(torch.int16)
    flat = bits.view(B, Hkv, nb, 2 * d)
    flat.scatter_(3, small, flat.gather(3, small) ^ flip)
    choose(api, query(k, "f32", B, Hkv * 3, d), base.to(DEV), 16 * nb, 16, k, 1, 0)


def test_block_select_infinite_and_nan(api):
    """More NaN scores, and more infinite ones, than blocks to choose; and fewer."""
    g = torch.Generator().manual_seed(5)
    Q = query(2, "bf16", 1, 4, 64).abs() + 0.1
    for n_nan, n_inf, k in ((30, 0, 20), (30, 0, 38), (0, 30, 12), (20, 20, 25), (40, 0, 7), (0, 0, 40)):
        b = torch.randn(1, 1, 40, 2, 64, generator=g).sort(3)[0].to(torch.bfloat16)
        p = torch.randperm(40, generator=g)
        b[0, 0, p[:n_nan], 1, 3] = math.nan
        b[0, 0, p[n_nan:n_nan + n_inf], 1, 5] = math.inf
        choose(api, Q, b.to(DEV), 640, 16, k)
    b[..., :] = -math.inf
    b[0, 0, 7] = 1.0
    choose(api, Q, b.to(DEV), 640, 16, 5)


def test_block_select_large_and_small_numbers(api):
    """Sums that leave f32, subnormal ones, and zeros."""
    g = torch.Generator().manual_seed(6)
    for size in (2.0**120, 2.0**-120, 0.0):
        b = (torch.randn(1, 1, 100, 2, 64, generator=g).sort(3)[0] * size).to(torch.bfloat16)
        choose(api, query(3, "bf16", 1, 8, 64), b.to(DEV), 1600, 16, 9)
        choose(api, (query(4, "bf16", 1, 8, 64).float() * 2.0**60).to(torch.bfloat16), b.to(DEV), 1600, 16, 9)


def test_nothing_to_append(api, lib):
    Kq, Vq, sc = api.empty_quant(1, 1, 64, 64)
    e = torch.empty(1, 1, 0, 64, device=DEV)
    api.quant_append(e, e, Kq, Vq, sc)
    api.quant_read(Kq, Vq, sc, e, e)
    assert status(lib) == 0


@pytest.mark.parametrize("kv", ["bf16", "int8", "f32"])
def test_negative_and_zero_scale(api, kv):
    """softmax(-x) and equal weights are softmaxes too."""
    B, Hkv, G, d, N, T = 1, 2, 4, 64, 150, 40
    K, V, sc, Kd, Vd = make_cache(kv, 95, B, Hkv, up(N + T), d)
    q = "f32" if kv == "f32" else "bf16"
    Q = query(7, q, B, T, Hkv * G, d)
    tree = random_tree(1, B, T)
    bl = torch.arange(3, dtype=torch.int32, device=DEV).expand(B, Hkv, 3).contiguous()
    for scale in (-0.2, 0.0):
        O = torch.empty(B, T, Hkv * G, d, device=DEV)
        api.tree_decode(Q, K, V, N, scale, O, mask=api.tree_mask(tree).to(DEV), scales=sc)
        want, A, S = oracle(Q, Kd, Vd, lambda b, h, t: list(range(N)) + [N + i for i in range(T) if tree[b, t, i]], scale)
        hold(O, want, A, np.abs(S), d, N + T)
        O1 = torch.empty(B, Hkv * G, d, device=DEV)
        api.block_attend(Q[:, 0].contiguous(), K, V, N, 32, bl, scale, O1, scales=sc)
        want, A, S = oracle(Q[:, :1], Kd, Vd, lambda b, h, t: slice(0, 96), scale)
        hold(O1[:, None], want, A, np.abs(S), d, 96)


@pytest.mark.parametrize("kv, q", [("bf16", "bf16"), ("int8", "bf16"), ("e4m3", "f32"), ("f32", "f32")])
def test_large_queries_and_keys(api, kv, q):
    """Logits of hundreds (one key has all the weight), and queries near the ends of their type.

    Weights of an 8-bit cache are f16 terms of w = x * vs * 2^(13 - E): x = 1 or more for the row's heaviest key, vs a
    key's value scale and 2^E <= the largest of them. The second term leaves at most half of f16's smallest step,
    2^-25, of a weight however small, which is 2^-25 * 2^(E - 13) * |code| <= 2^-38 * (largest scale) * 448 of a value:
    over n keys n * 2^-38 * max |v|, divided by a sum of weights of at least 1. Where the heavy key's value is 0,
    nothing else of the bound is left.
    """
    B, Hkv, G, d, N = 1, 2, 4, 128, 300
    K, V, sc, Kd, Vd = make_cache(kv, 96, B, Hkv, up(N), d)
    floor = 0.0 if sc is None else N * 2.0**-38 * 448 * float(sc[..., 1].max())
    for size, scale in ((30.0, 1.0), (2.0**100, 2.0**-100), (2.0**-110, 2.0**100)):
        Q = (query(8, "f32", B, 1, Hkv * G, d) * size).to(QT[q])
        O = torch.empty(B, 1, Hkv * G, d, device=DEV)
        api.tree_decode(Q, K, V, N - 1, scale, O, scales=sc)
        want, A, S = oracle(Q, Kd, Vd, lambda b, h, t: slice(0, N), scale)
        hold(O, want, A, S, d, N, floor=floor)
        if sc is not None:
            O1 = torch.empty(B, Hkv * G, d, device=DEV)
            api.quant_decode(Q[:, 0].contiguous(), K, V, sc, N, scale, O1)
            hold(O1[:, None], want, A, S, d, N, floor=floor)


@pytest.mark.parametrize("kv, d, G, T, N, out", [("bf16", 64, 2, 3, 200003, "f32"), ("bf16", 128, 4, 12, 150001, "f32"), ("bf16", 128, 4, 40, 100001, "f32"),
                                                 ("bf16", 64, 4, 33, 150000, "f32"), ("bf16", 128, 4, 40, 100001, "bf16"), ("int8", 64, 2, 3, 200003, "f32"),
                                                 ("e4m3", 128, 4, 20, 100001, "f32"), ("int8", 128, 4, 12, 150001, "bf16")])
def test_long_runs_of_tiles(api, lib, kv, d, G, T, N, out):
    """Caches long enough that a block takes tens of tiles: the accumulators' changes within a run.

    The bound's chain: f32 outputs add the products of 8 tiles (at most 192 of them) before a plain sum, a run has at
    most 150 tiles with one sum of weights each beside 64 within a tile, and at most 150 partials are joined: 500 steps.
    bf16 outputs let a run's products follow one another: 150 tiles of 8.
    """
    B, Hkv = 1, 2
    Ncap = up(N + T)
    g = torch.Generator(device=DEV).manual_seed(T)
    K, V = (torch.randn(B, Hkv, Ncap, d, generator=g, device=DEV) for _ in range(2))
    V *= 1 + torch.arange(Ncap, device=DEV)[:, None] % 7                       # no run like another
    sc = None
    if kv == "bf16":
        K, V = K.to(torch.bfloat16), V.to(torch.bfloat16)
        Kd, Vd = K.double().cpu().numpy(), V.double().cpu().numpy()
    else:
        Kq, Vq, sc = api.empty_quant(B, Hkv, Ncap, d, FMT[kv])
        api.quant_append(K, V, Kq, Vq, sc)
        Kr, Vr = torch.empty_like(K), torch.empty_like(V)
        api.quant_read(Kq, Vq, sc, Kr, Vr)
        K, V, Kd, Vd = Kq, Vq, Kr.double().cpu().numpy(), Vr.double().cpu().numpy()
    seen = random_tree(T, B, T)
    Q = query(T, "bf16", B, T, Hkv * G, d)
    # logits that rise along the cache: the maximum grows in every run
    Q[..., 0], ramp = 8.0, torch.linspace(-3, 3, Ncap, device=DEV)
    if kv == "bf16":
        K[..., 0] = ramp.to(torch.bfloat16)
        Kd = K.double().cpu().numpy()
    O = torch.empty(B, T, Hkv * G, d, dtype=QT[out], device=DEV)
    api.tree_decode(Q, K, V, N, 0.11, O, mask=api.tree_mask(seen).to(DEV), scales=sc)
    pick = sorted({0, T // 2, T - 1})                                        # some tokens, all heads
    want, A, S = oracle(Q[:, pick], Kd, Vd, lambda b, h, t: np.array(list(range(N)) + [N + i for i in range(T) if seen[b, pick[t], i]]), 0.11)
    hold(O[:, pick], want, A, S, d, 500 if out == "f32" else 1500, out)
    if sc is not None:
        O1 = torch.empty(B, Hkv * G, d, device=DEV)
        api.quant_decode(Q[:, 0].contiguous(), K, V, sc, N, 0.11, O1)
        want, A, S = oracle(Q[:, :1], Kd, Vd, lambda b, h, t: slice(0, N), 0.11)
        hold(O1[:, None], want, A, S, d, 500)
    assert status(lib) == 0
