"""Refusals of the entry points over quantised, block-selected and drafted caches (host checks: nothing is launched, no
GPU needed), their workspace sizes, and the binding's own checks."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from hash_scored_top_b200 import build
    build.build()
    from hash_scored_top_b200 import _lib
    return _lib


P = ctypes.c_void_p(256)         # never dereferenced: validation fails first
ODD = ctypes.c_void_p(264)       # 8-byte aligned only
BIG = 1 << 30
F32, BF16, INT8, E4M3 = 0, 1, 2, 3

# name -> a call that every check but the workspace's passes, as keyword arguments in the order of the C signature
GOOD = {
    "quant_append": dict(K_new=P, V_new=P, src=BF16, stride_b=0, stride_h=128, stride_n=128, starts=None, lens=None, B=1, Hkv=1,
                         Ncap=64, n_begin=0, n_count=1, d=128, Kq=P, Vq=P, kv=INT8, scales=P, stream=None),
    "quant_read": dict(Kq=P, Vq=P, kv=INT8, scales=P, starts=None, lens=None, B=1, Hkv=1, Ncap=64, n_begin=0, n_count=1, d=128,
                       K=P, V=P, dst=BF16, stream=None),
    "quant_decode": dict(Q=P, q=BF16, Kq=P, Vq=P, kv=INT8, scales=P, lens=None, B=1, Hq=4, Hkv=1, Ncap=64, N=64, d=128, scale=0.1,
                         O=P, ws=None, ws_bytes=0, stream=None),
    "quant_sparse_attend": dict(Q=P, q=BF16, Kq=P, Vq=P, kv=INT8, scales=P, idx=P, B=1, Hq=4, Hkv=1, Ncap=64, d=128, k=8,
                                scale=0.1, O=P, ws=None, ws_bytes=0, stream=None),
    "socket_decode_quant": dict(Q=P, q=BF16, Kq=P, Vq=P, kv=INT8, scales=P, R=P, ids=P, norms=P, B=1, Hq=4, Hkv=1, Ncap=64, N=64,
                                d=128, L=8, P=4, tau=0.5, k=8, scale=0.1, O=P, idx_out=None, ws=None, ws_bytes=0, stream=None),
    "block_summarize": dict(K=P, kv=BF16, scales=None, starts=None, lens=None, B=1, Hkv=1, Ncap=64, n_begin=0, n_count=64, d=128,
                            block=16, bsum=P, stream=None),
    "block_select": dict(Q=P, q=BF16, bsum=P, lens=None, B=1, Hq=4, Hkv=1, Ncap=64, N=64, d=128, block=16, k=3, n_first=1,
                         n_last=1, idx=P, ws=None, ws_bytes=0, stream=None),
    "block_attend": dict(Q=P, q=BF16, K=P, V=P, kv=BF16, scales=None, lens=None, idx=P, B=1, Hq=4, Hkv=1, Ncap=64, N=64, d=128,
                         block=16, k=3, scale=0.1, O=P, ws=None, ws_bytes=0, stream=None),
    "block_decode": dict(Q=P, q=BF16, K=P, V=P, kv=BF16, scales=None, bsum=P, lens=None, B=1, Hq=4, Hkv=1, Ncap=64, N=64, d=128,
                         block=16, k=3, n_first=1, n_last=1, scale=0.1, O=P, idx_out=None, ws=None, ws_bytes=0, stream=None),
    "tree_decode": dict(Q=P, q=BF16, K=P, V=P, kv=BF16, scales=None, lens=None, mask=None, B=1, T=4, Hq=4, Hkv=1, Ncap=64, N=60,
                        d=128, scale=0.1, O=P, o=F32, ws=None, ws_bytes=0, stream=None),
}
ATTENDS = ("quant_decode", "quant_sparse_attend", "socket_decode_quant", "block_attend", "block_decode", "tree_decode")
QUERIES = ATTENDS + ("block_select",)
QUANTISED = ("quant_append", "quant_read", "quant_decode", "quant_sparse_attend", "socket_decode_quant")

REFUSALS = (
    [(n, {a: None}, 1, f"{a} is NULL") for n in ATTENDS for a in ("Q", "O")]
    + [(n, {"Q": ODD}, 1, "Q must be 16-byte aligned") for n in QUERIES]
    + [(n, {"Hq": 3, "Hkv": 2}, 1, "multiple") for n in QUERIES]
    + [(n, {"Hq": 9}, 2, "G=9") for n in QUERIES]
    + [(n, {"d": 96}, 2, "d=96") for n in GOOD]
    + [(n, {"B": 0}, 1, "B, Hq, Hkv") for n in GOOD]
    + [(n, {"B": 70000}, 2, "65535") for n in GOOD]
    + [(n, {"Ncap": 40, "N": 40}, 1, "Ncap=40") for n in GOOD]
    + [(n, {}, 5, "workspace") for n in QUERIES]
    + [(n, {"ws": P, "ws_bytes": 16}, 5, "workspace") for n in QUERIES]
    + [(n, {"ws": ODD, "ws_bytes": BIG}, 1, "ws must be 16-byte aligned") for n in QUERIES]
    + [(n, {"kv": BF16}, 1, "SK_INT8 or SK_E4M3") for n in QUANTISED]
    + [(n, {"kv": 9}, 1, "dtype") for n in GOOD if "kv" in GOOD[n]]
    + [(n, {"q": INT8}, 1, "dtype") for n in QUERIES]
    + [(n, {"scales": None}, 1, "scales is NULL") for n in QUANTISED]
    + [(n, {"kv": E4M3}, 1, "scales is NULL") for n in ("block_summarize", "block_attend", "block_decode", "tree_decode")]
    + [(n, {"q": F32}, 1, "must be the same") for n in ("block_attend", "block_decode", "tree_decode")]
    + [(n, {"N": 65}, 1, "N=65") for n in ("quant_decode", "block_select", "block_attend", "block_decode", "socket_decode_quant")]
    + [(n, {"N": 0}, 1, "N=0") for n in ("quant_decode", "block_select", "block_attend", "block_decode")]
    + [(n, {"n_count": -1}, 1, "n_count") for n in ("quant_append", "quant_read", "block_summarize")]
    + [(n, {"n_begin": 60, "n_count": 5}, 1, "range") for n in ("quant_append", "quant_read", "block_summarize")]
    + [(n, {"n_begin": -1}, 1, "range") for n in ("quant_append", "quant_read", "block_summarize")]
    + [(n, {"n_count": (1 << 30) + 1, "starts": P}, 1, "n_count") for n in ("quant_append", "quant_read", "block_summarize")]
    + [(n, {"Ncap": 2**31 - 32}, 2, "rows per pair") for n in GOOD]
    + [(n, {"block": 24}, 2, "block=24") for n in ("block_summarize", "block_select", "block_attend", "block_decode")]
    + [(n, {"k": 0}, 1, "k=0") for n in ("quant_sparse_attend", "block_select", "block_attend", "block_decode")]
    + [(n, {"k": 1 << 28}, 1, "blocks of") for n in ("block_select", "block_attend", "block_decode")]
    + [(n, {"n_first": 2, "n_last": 2}, 1, "n_first=2") for n in ("block_select", "block_decode")]
    + [(n, {"n_first": -1}, 1, "n_first=-1") for n in ("block_select", "block_decode")]
    + [("quant_append", {"stride_n": 100}, 1, "strides"), ("quant_append", {"src": E4M3}, 1, "dtype"),
       ("quant_append", {"K_new": ODD}, 1, "K_new must be 16-byte aligned"), ("quant_append", {"scales": ctypes.c_void_p(260)}, 1, "scales"),
       ("quant_read", {"dst": INT8}, 1, "dtype"), ("quant_sparse_attend", {"idx": None}, 1, "idx is NULL"),
       ("block_select", {"idx": None}, 1, "idx is NULL"), ("block_attend", {"idx": None}, 1, "idx is NULL"),
       ("socket_decode_quant", {"k": 65}, 1, "k=65"), ("socket_decode_quant", {"tau": 0.0}, 1, "tau"),
       ("tree_decode", {"T": 0}, 2, "T=0"), ("tree_decode", {"T": 257}, 2, "T=257"), ("tree_decode", {"N": 61}, 1, "do not fit"),
       ("tree_decode", {"N": -1}, 1, "do not fit"), ("tree_decode", {"N": 2**31 - 2}, 1, "do not fit"), ("tree_decode", {"o": INT8}, 1, "dtype")]
)


@pytest.mark.parametrize("name, change, status, words", REFUSALS, ids=lambda v: str(v)[:40])
def test_refused(lib, name, change, status, words):
    args = {**GOOD[name], **{k: v for k, v in change.items() if k in GOOD[name]}}
    rc = getattr(lib.lib, name)(*args.values())
    assert rc == status and words in lib.last_error(), (rc, lib.last_error())


def test_nothing_to_do_is_no_error(lib):
    for name in ("quant_append", "quant_read", "block_summarize"):
        assert getattr(lib.lib, name)(*{**GOOD[name], "n_count": 0}.values()) == 0


def test_older_entry_points_refuse_quantised_dtypes(lib):
    for code in (INT8, E4M3):
        assert lib.lib.dense_decode(P, P, P, code, 1, 4, 1, 64, 64, 128, 0.1, P, P, BIG, None) == 1
        assert "dtype" in lib.last_error()


def test_workspace_sizes(lib):
    from hash_scored_top_b200 import api
    for op in (api.OP_QUANT_DECODE, api.OP_QUANT_SPARSE_ATTEND, api.OP_BLOCK_ATTEND, api.OP_BLOCK_DECODE, api.OP_TREE_DECODE):
        assert api.workspace_bytes(op, 2, 16, 4, 1024, 1000, 128, 32, 0, 8) > 0
    assert api.workspace_bytes(api.OP_BLOCK_SELECT, 2, 16, 4, 1024, 1000, 128, 32, 0, 8) >= 8 * 32 * 4
    assert (api.workspace_bytes(api.OP_SOCKET_DECODE_QUANT, 2, 16, 4, 1024, 1000, 128, 8, 4, 64)
            >= api.workspace_bytes(api.OP_QUANT_SPARSE_ATTEND, 2, 16, 4, 1024, 1000, 128, 0, 0, 64))
    for op, kw in ((api.OP_QUANT_DECODE, dict(d=96)), (api.OP_BLOCK_DECODE, dict(L=24)), (api.OP_TREE_DECODE, dict(k=300)),
                   (api.OP_QUANT_DECODE, dict(Hq=9, Hkv=1))):
        with pytest.raises(ValueError):
            api.workspace_bytes(op, **{**dict(B=1, Hq=4, Hkv=1, Ncap=64, N=64, d=128, L=16, P=0, k=4), **kw})


def test_binding_checks(lib):
    from hash_scored_top_b200 import api
    K = torch.zeros(1, 1, 64, 128, dtype=torch.int8)
    s = torch.zeros(1, 1, 64, 2)
    Q, O = torch.zeros(1, 4, 128), torch.zeros(1, 4, 128)
    with pytest.raises(ValueError, match="CUDA device"):
        api.quant_decode(Q, K, K, s, 64, 0.1, O)
    with pytest.raises(TypeError, match="cache dtype"):
        api.quant_decode(Q, K.float(), K.float(), s, 64, 0.1, O)
    with pytest.raises(ValueError, match="needs them"):
        api.tree_decode(Q[:, None], K, K, 32, 0.1, O[:, None])
    with pytest.raises(ValueError, match="has none"):
        api.tree_decode(Q[:, None], K.float(), K.float(), 32, 0.1, O[:, None], scales=s)
    with pytest.raises(ValueError, match="scales"):
        api.quant_decode(Q, K, K, s[:, :, :32], 64, 0.1, O)
    with pytest.raises(TypeError, match="lens"):
        api.quant_decode(Q, K, K, s, 64, 0.1, O, lens=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="K_new"):
        api.quant_append(torch.zeros(1, 1, 3, 64), torch.zeros(1, 1, 3, 64), K, K, s)
    with pytest.raises(ValueError, match="strides"):
        api.quant_append(torch.zeros(1, 1, 3, 128), torch.zeros(1, 1, 6, 128)[:, :, ::2], K, K, s)
    with pytest.raises(ValueError, match="bsum"):
        api.block_summarize(K.float(), 16, torch.zeros(1, 1, 3, 2, 128, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="int8 or float8"):
        api.empty_quant(1, 1, 64, 128, dtype=torch.float16)


def test_tree_mask_words():
    from hash_scored_top_b200 import api
    g = torch.Generator().manual_seed(3)
    seen = torch.rand(2, 70, 70, generator=g) < 0.5
    w = api.tree_mask(seen)
    assert w.shape == (2, 70, 3) and w.dtype == torch.int32
    i = torch.arange(70)
    assert torch.equal(((w[:, :, i // 32] >> (i % 32)) & 1).bool(), seen)
