"""Python binding of libhash_scored_top.so (argument marshalling only).

Every function here checks tensor devices, dtypes and shapes, passes raw
pointers and sizes to the C entry point of the same name, and raises
``RuntimeError`` with the library's message on a non-zero status. All
compute happens in the library's CUDA kernels on the current torch stream;
torch only provides device memory (outputs and workspaces) and the stream.
Without a ``ws`` argument a workspace of the size sk_workspace_bytes gives is
allocated for the call; a ``ws`` that is passed goes to the library as it is
(no size query on the host), which rejects one that is too small.
There is no CPU fallback: if the library is missing the import of
``_lib`` fails loudly.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib

SK_F32, SK_BF16, SK_INT8, SK_E4M3 = 0, 1, 2, 3
(OP_HASH_KEYS, OP_SCORE, OP_TOPK, OP_SPARSE_ATTEND, OP_DECODE, OP_HATA_HASH, OP_HATA_DECODE, OP_DENSE_DECODE,
 OP_SELECT, OP_SOFT_COUNT, OP_DECODE_HEADS, OP_DECODE_ADAPTIVE, OP_DECODE_ADAPTIVE_HEADS, OP_SPARSE_ATTEND_PAGED,
 OP_DECODE_PAGED, OP_QUANT_DECODE, OP_QUANT_SPARSE_ATTEND, OP_SOCKET_DECODE_QUANT, OP_BLOCK_SELECT, OP_BLOCK_ATTEND,
 OP_BLOCK_DECODE, OP_TREE_DECODE) = range(22)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SK_F32
    if t.dtype == torch.bfloat16:
        return SK_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _pool_ptr(t):
    """A K/V pool: device memory, or pinned host memory that the device reads directly."""
    if t.is_cuda:
        return _ptr(t)
    if not (t.is_pinned() and t.is_contiguous()):
        raise ValueError("host pools must be pinned and contiguous (the device reads them directly)")
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(rc: int, what: str):
    if rc != 0:
        raise RuntimeError(f"{what} failed (status {rc}): {_lib.last_error()}")


def _want(t: torch.Tensor, dtype, shape, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _workspace(nbytes: int, device, ws):
    if nbytes == 0:
        return ws
    if ws is None or ws.numel() * ws.element_size() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws


def _ws_bytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


# ---------------------------------------------------------------- cache allocation / layout
def ids_bytes_per_key(L: int) -> int:
    """Bytes per key of the bucket-ID cache (see the C header)."""
    return 16 if L <= 16 else 32 if L <= 32 else 48 if L <= 48 else 64


def _chunk_size(L: int, chunk: int) -> int:
    if chunk == 0:
        return 16 if L <= 16 else 32
    return 16 if L <= 48 else 32


def _byte_positions(L: int, n: int, device) -> torch.Tensor:
    """pos[i, l]: byte of key i (i < n) that holds table l's ID (the rotated layout)."""
    r = torch.arange(n, device=device)[:, None] % 32
    ll = torch.arange(L, device=device)[None, :]
    c = (ll >= 32).long()
    S = torch.where(c == 1, _chunk_size(L, 1), _chunk_size(L, 0))
    return 32 * c + torch.remainder(ll - 32 * c - r, S)


def empty_ids(B: int, Hkv: int, Ncap: int, L: int, device="cuda") -> torch.Tensor:
    """Bucket-ID cache [B, Hkv, Ncap, ids_bytes_per_key(L)] uint8 (rotated key-major layout)."""
    return torch.zeros(B, Hkv, Ncap, ids_bytes_per_key(L), dtype=torch.uint8, device=device)


def empty_norms(B: int, Hkv: int, Ncap: int, device="cuda") -> torch.Tensor:
    return torch.zeros(B, Hkv, Ncap, dtype=torch.float16, device=device)


def empty_codes(B: int, Hkv: int, Ncap: int, device="cuda") -> torch.Tensor:
    """Hard-hash code cache [B, Hkv, Ncap, 16] uint8: byte j of key n holds code byte (j + n) mod 16."""
    return torch.zeros(B, Hkv, Ncap, 16, dtype=torch.uint8, device=device)


def ids_to_natural(ids: torch.Tensor, L: int) -> torch.Tensor:
    """Cache layout -> [B, Hkv, Ncap, L] with [.., n, l] the ID of table l (a byte gather, no arithmetic)."""
    B, H, n, _ = ids.shape
    pos = _byte_positions(L, n, ids.device).expand(B, H, n, L)
    return torch.gather(ids, -1, pos)


def natural_to_ids(nat: torch.Tensor) -> torch.Tensor:
    """[B, Hkv, Ncap, L] -> cache layout (inverse of ids_to_natural; padding bytes are 0)."""
    B, H, n, L = nat.shape
    out = torch.zeros(B, H, n, ids_bytes_per_key(L), dtype=nat.dtype, device=nat.device)
    pos = _byte_positions(L, n, nat.device).expand(B, H, n, L)
    return out.scatter_(-1, pos, nat)


# ---------------------------------------------------------------- entry points
def workspace_bytes(op: int, B, Hq, Hkv, Ncap, N, d, L=0, P=0, k=0) -> int:
    n = _lib.lib.sk_workspace_bytes(op, B, Hq, Hkv, Ncap, N, d, L, P, k)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid shapes for workspace query")
    return n


def socket_hash_keys(K, V, R, L: int, P: int, ids, norms, n_begin: int = 0, n_count: int | None = None):
    """SOCKET step 1 for keys [n_begin, n_begin + n_count) of every pair (see the C header)."""
    B, Hkv, Ncap, d = K.shape
    n_count = Ncap - n_begin if n_count is None else n_count
    _want(V, K.dtype, K.shape, "V")
    _want(R, torch.bfloat16, (L * P, d), "R")
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(norms, torch.float16, (B, Hkv, Ncap), "norms")
    rc = _lib.lib.socket_hash_keys(_ptr(K), _ptr(V), _dtype_code(K), _ptr(R), B, Hkv, Ncap, n_begin, n_count, d, L, P,
                                   _ptr(ids), _ptr(norms), _stream())
    _check(rc, "socket_hash_keys")


def socket_score(Q, R, ids, norms, N: int, L: int, P: int, tau: float, scores, ws=None):
    """SOCKET steps 2-3: scores [B, Hkv, Ncap] f32 for keys < N."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = ids.shape
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(scores, torch.float32, (B, Hkv, Ncap), "scores")
    _want(R, torch.bfloat16, (L * P, d), "R")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_SCORE, B, Hq, Hkv, Ncap, N, d, L, P, 0), Q.device, ws)
    rc = _lib.lib.socket_score(_ptr(Q), _dtype_code(Q), _ptr(R), _ptr(ids), _ptr(norms), B, Hq, Hkv, Ncap, N, d, L, P,
                               ctypes.c_float(tau), _ptr(scores), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "socket_score")


def socket_topk(scores, N: int, k: int, idx):
    """SOCKET step 4 (selection): idx [B, Hkv, k] int32 ascending."""
    B, Hkv, Ncap = scores.shape
    _want(scores, torch.float32, scores.shape, "scores")
    _want(idx, torch.int32, (B, Hkv, k), "idx")
    rc = _lib.lib.socket_topk(_ptr(scores), B, Hkv, Ncap, N, k, _ptr(idx), None, 0, _stream())
    _check(rc, "socket_topk")


def socket_sparse_attend(Q, K, V, idx, scale: float, O, ws=None):
    """SOCKET step 4 (attention over idx): O [B, Hq, d] f32."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    k = idx.shape[-1]
    _want(K, Q.dtype, K.shape, "K")
    _want(V, Q.dtype, K.shape, "V")
    _want(idx, torch.int32, (B, Hkv, k), "idx")
    _want(O, torch.float32, (B, Hq, d), "O")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_SPARSE_ATTEND, B, Hq, Hkv, Ncap, k, d, 0, 0, k), Q.device, ws)
    rc = _lib.lib.socket_sparse_attend(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K), _ptr(idx), B, Hq, Hkv, Ncap, d, k,
                                       ctypes.c_float(scale), _ptr(O), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "socket_sparse_attend")


def socket_sparse_attend_noalloc(Q, K, V, idx, scale: float, O):
    """socket_sparse_attend for callers that cannot allocate device memory.

    The library keeps a fixed static device scratch (``noalloc_scratch_bytes()``
    bytes per GPU) for the attention partials, so this call allocates nothing;
    shapes that do not fit raise RuntimeError. All calls on a GPU share that
    scratch: calls that overlap on the GPU race. The first call on a device
    looks up the scratch address; make it before any stream capture.
    """
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    k = idx.shape[-1]
    _want(K, Q.dtype, K.shape, "K")
    _want(V, Q.dtype, K.shape, "V")
    _want(idx, torch.int32, (B, Hkv, k), "idx")
    _want(O, torch.float32, (B, Hq, d), "O")
    rc = _lib.lib.socket_sparse_attend_noalloc(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K), _ptr(idx), B, Hq, Hkv,
                                               Ncap, d, k, ctypes.c_float(scale), _ptr(O), _stream())
    _check(rc, "socket_sparse_attend_noalloc")


def noalloc_scratch_bytes() -> int:
    """Bytes of the static scratch socket_sparse_attend_noalloc uses."""
    return int(_lib.lib.sk_noalloc_scratch_bytes())


def socket_decode(Q, K, V, R, ids, norms, N: int, L: int, P: int, tau: float, k: int, scale: float, O, idx_out=None,
                  ws=None):
    """The fused decode step (SOCKET steps 2-4)."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    _want(K, Q.dtype, K.shape, "K")
    _want(V, Q.dtype, K.shape, "V")
    _want(R, torch.bfloat16, (L * P, d), "R")
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(norms, torch.float16, (B, Hkv, Ncap), "norms")
    _want(O, torch.float32, (B, Hq, d), "O")
    if idx_out is not None:
        _want(idx_out, torch.int32, (B, Hkv, k), "idx_out")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_DECODE, B, Hq, Hkv, Ncap, N, d, L, P, k), Q.device, ws)
    rc = _lib.lib.socket_decode(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K), _ptr(R), _ptr(ids), _ptr(norms), B, Hq, Hkv,
                                Ncap, N, d, L, P, ctypes.c_float(tau), k, ctypes.c_float(scale), _ptr(O),
                                _ptr(idx_out), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "socket_decode")


def socket_decode_heads(Q, K, V, R, ids, norms, N: int, L: int, P: int, tau: float, k: int, scale: float, O,
                        idx_out=None, ws=None):
    """The decode step with one index set per query head; idx_out: [B, Hq, k]."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    _want(K, Q.dtype, K.shape, "K")
    _want(V, Q.dtype, K.shape, "V")
    _want(R, torch.bfloat16, (L * P, d), "R")
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(norms, torch.float16, (B, Hkv, Ncap), "norms")
    _want(O, torch.float32, (B, Hq, d), "O")
    if idx_out is not None:
        _want(idx_out, torch.int32, (B, Hq, k), "idx_out")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_DECODE_HEADS, B, Hq, Hkv, Ncap, N, d, L, P, k), Q.device, ws)
    rc = _lib.lib.socket_decode_heads(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K), _ptr(R), _ptr(ids), _ptr(norms), B,
                                      Hq, Hkv, Ncap, N, d, L, P, ctypes.c_float(tau), k, ctypes.c_float(scale),
                                      _ptr(O), _ptr(idx_out), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "socket_decode_heads")


def socket_decode_adaptive(Q, K, V, R, ids, norms, N: int, L: int, P: int, tau: float, mass: float, k_min: int,
                           k_max: int, scale: float, O, idx, kcount, per_head: bool = False, ws=None):
    """The decode step with the adaptive k; idx: [B, U, k_max], kcount: [B, U] (U = Hkv, or Hq per head)."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    U = Hq if per_head else Hkv
    _want(K, Q.dtype, K.shape, "K")
    _want(V, Q.dtype, K.shape, "V")
    _want(R, torch.bfloat16, (L * P, d), "R")
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(norms, torch.float16, (B, Hkv, Ncap), "norms")
    _want(O, torch.float32, (B, Hq, d), "O")
    _want(idx, torch.int32, (B, U, k_max), "idx")
    _want(kcount, torch.int32, (B, U), "kcount")
    op = OP_DECODE_ADAPTIVE_HEADS if per_head else OP_DECODE_ADAPTIVE
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(op, B, Hq, Hkv, Ncap, N, d, L, P, k_max), Q.device, ws)
    rc = _lib.lib.socket_decode_adaptive(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K), _ptr(R), _ptr(ids), _ptr(norms),
                                         B, Hq, Hkv, Ncap, N, d, L, P, ctypes.c_float(tau), int(bool(per_head)),
                                         ctypes.c_float(mass), k_min, k_max, ctypes.c_float(scale), _ptr(O),
                                         _ptr(idx), _ptr(kcount), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "socket_decode_adaptive")


def _want_pool(K_pool, V_pool, dtype, d):
    if K_pool.dtype != dtype or V_pool.dtype != dtype:
        raise TypeError(f"pools: dtypes {K_pool.dtype}, {V_pool.dtype}, expected {dtype}")
    if K_pool.dim() != 3 or tuple(K_pool.shape) != tuple(V_pool.shape) or K_pool.shape[2] != d:
        raise ValueError(f"pools: shapes {tuple(K_pool.shape)}, {tuple(V_pool.shape)}, expected [pages, page_size, {d}]")
    if not (K_pool.is_contiguous() and V_pool.is_contiguous()):
        raise ValueError("pools must be contiguous")
    if K_pool.device.type == "cpu" and not (K_pool.is_pinned() and V_pool.is_pinned()):
        raise ValueError("host pools must be pinned (the device reads them directly)")


def socket_sparse_attend_paged(Q, K_pool, V_pool, page_table, idx, scale: float, O, ws=None):
    """Sparse attention with K/V in a paged pool (device or pinned host memory).

    K_pool, V_pool: [num_pages, page_size, d]; page_table: [B, Hkv, max_pages] int32 (device);
    idx: [B, Hkv, k] int32 (device)."""
    B, Hq, d = Q.shape
    _, Hkv, max_pages = page_table.shape
    num_pages, page_size, _ = K_pool.shape
    k = idx.shape[-1]
    _want_pool(K_pool, V_pool, Q.dtype, d)
    _want(page_table, torch.int32, (B, Hkv, max_pages), "page_table")
    _want(idx, torch.int32, (B, Hkv, k), "idx")
    _want(O, torch.float32, (B, Hq, d), "O")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_SPARSE_ATTEND_PAGED, B, Hq, Hkv, 32, k, d, 1, 1, k), Q.device, ws)
    rc = _lib.lib.socket_sparse_attend_paged(_ptr(Q), _pool_ptr(K_pool), _pool_ptr(V_pool), _dtype_code(Q),
                                             _ptr(page_table), max_pages, page_size, num_pages, _ptr(idx), B, Hq,
                                             Hkv, d, k, ctypes.c_float(scale), _ptr(O), _ptr(ws), _ws_bytes(ws),
                                             _stream())
    _check(rc, "socket_sparse_attend_paged")


def socket_decode_paged(Q, K_pool, V_pool, page_table, R, ids, norms, N: int, L: int, P: int, tau: float, k: int,
                        scale: float, O, idx_out=None, ws=None):
    """The decode step with a paged K/V cache; ids and norms are the contiguous hashed-key cache."""
    B, Hq, d = Q.shape
    _, Hkv, max_pages = page_table.shape
    num_pages, page_size, _ = K_pool.shape
    Ncap = ids.shape[2]
    _want_pool(K_pool, V_pool, Q.dtype, d)
    _want(page_table, torch.int32, (B, Hkv, max_pages), "page_table")
    _want(R, torch.bfloat16, (L * P, d), "R")
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(norms, torch.float16, (B, Hkv, Ncap), "norms")
    _want(O, torch.float32, (B, Hq, d), "O")
    if idx_out is not None:
        _want(idx_out, torch.int32, (B, Hkv, k), "idx_out")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_DECODE_PAGED, B, Hq, Hkv, Ncap, N, d, L, P, k), Q.device, ws)
    rc = _lib.lib.socket_decode_paged(_ptr(Q), _pool_ptr(K_pool), _pool_ptr(V_pool), _dtype_code(Q),
                                      _ptr(page_table), max_pages, page_size, num_pages, _ptr(R), _ptr(ids),
                                      _ptr(norms), B, Hq, Hkv, Ncap, N, d, L, P, ctypes.c_float(tau), k,
                                      ctypes.c_float(scale), _ptr(O), _ptr(idx_out), _ptr(ws), _ws_bytes(ws),
                                      _stream())
    _check(rc, "socket_decode_paged")


def socket_decode_append(Q, K, V, R, ids, norms, N: int, L: int, P: int, tau: float, k: int, scale: float, O,
                         idx_out=None, ws=None):
    """One decoder step: hash key N - 1 into (ids, norms), then the decode over N keys."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    _want(K, Q.dtype, K.shape, "K")
    _want(V, Q.dtype, K.shape, "V")
    _want(R, torch.bfloat16, (L * P, d), "R")
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(norms, torch.float16, (B, Hkv, Ncap), "norms")
    _want(O, torch.float32, (B, Hq, d), "O")
    if idx_out is not None:
        _want(idx_out, torch.int32, (B, Hkv, k), "idx_out")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_DECODE, B, Hq, Hkv, Ncap, N, d, L, P, k), Q.device, ws)
    rc = _lib.lib.socket_decode_append(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K), _ptr(R), _ptr(ids), _ptr(norms), B,
                                       Hq, Hkv, Ncap, N, d, L, P, ctypes.c_float(tau), k, ctypes.c_float(scale),
                                       _ptr(O), _ptr(idx_out), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "socket_decode_append")


def _host_ptr(t, name):
    if t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous host tensor (pinned for asynchronous copies)")
    return ctypes.c_void_p(t.data_ptr())


def socket_decode_step_host(Q_host, K_new_host, V_new_host, Q, K, V, R, ids, norms, N: int, L: int, P: int,
                            tau: float, k: int, scale: float, O, O_host, ws=None):
    """One decode step from host buffers: Q_host [B, Hq, d] and the new token's rows K_new_host, V_new_host
    [B, Hkv, d] (pinned, K's dtype) are copied in (the rows to position N - 1 of K and V), the step runs as
    socket_decode_append, and O [B, Hq, d] float32 is copied to O_host (pinned). All on the current stream:
    O_host holds the result once the stream has synchronised."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    _want(Q, K.dtype, (B, Hq, d), "Q")
    _want(V, K.dtype, K.shape, "V")
    _want(R, torch.bfloat16, (L * P, d), "R")
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(norms, torch.float16, (B, Hkv, Ncap), "norms")
    _want(O, torch.float32, (B, Hq, d), "O")
    _want(Q_host, K.dtype, (B, Hq, d), "Q_host")
    _want(K_new_host, K.dtype, (B, Hkv, d), "K_new_host")
    _want(V_new_host, K.dtype, (B, Hkv, d), "V_new_host")
    _want(O_host, torch.float32, (B, Hq, d), "O_host")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_DECODE, B, Hq, Hkv, Ncap, N, d, L, P, k), Q.device, ws)
    rc = _lib.lib.socket_decode_step_host(_host_ptr(Q_host, "Q_host"), _host_ptr(K_new_host, "K_new_host"),
                                          _host_ptr(V_new_host, "V_new_host"), _ptr(Q), _ptr(K), _ptr(V),
                                          _dtype_code(K), _ptr(R), _ptr(ids), _ptr(norms), B, Hq, Hkv, Ncap, N, d, L,
                                          P, ctypes.c_float(tau), k, ctypes.c_float(scale), _ptr(O),
                                          _host_ptr(O_host, "O_host"), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "socket_decode_step_host")


def socket_select(Q, R, ids, norms, N: int, L: int, P: int, tau: float, k: int, idx, ws=None):
    """SOCKET steps 2-4 without the attention: idx [B, Hkv, k] int32 ascending."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = ids.shape
    _want(R, torch.bfloat16, (L * P, d), "R")
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(norms, torch.float16, (B, Hkv, Ncap), "norms")
    _want(idx, torch.int32, (B, Hkv, k), "idx")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_SELECT, B, Hq, Hkv, Ncap, N, d, L, P, k), Q.device, ws)
    rc = _lib.lib.socket_select(_ptr(Q), _dtype_code(Q), _ptr(R), _ptr(ids), _ptr(norms), B, Hq, Hkv, Ncap, N, d, L,
                                P, ctypes.c_float(tau), k, _ptr(idx), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "socket_select")


def hata_hash_keys(K, R128, codes, n_begin: int = 0, n_count: int | None = None):
    """128-bit sign codes of keys [n_begin, n_begin + n_count) of every pair."""
    B, Hkv, Ncap, d = K.shape
    n_count = Ncap - n_begin if n_count is None else n_count
    _want(R128, torch.bfloat16, (128, d), "R128")
    _want(codes, torch.uint8, (B, Hkv, Ncap, 16), "codes")
    rc = _lib.lib.hata_hash_keys(_ptr(K), _dtype_code(K), _ptr(R128), B, Hkv, Ncap, n_begin, n_count, d, _ptr(codes),
                                 _stream())
    _check(rc, "hata_hash_keys")


def hata_decode(Q, K, V, R128, codes, N: int, k: int, scale: float, O, idx_out=None, ws=None):
    """Hard-hash decode step: Hamming scores, exact top-k, attention over the selection."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    _want(K, Q.dtype, K.shape, "K")
    _want(V, Q.dtype, K.shape, "V")
    _want(R128, torch.bfloat16, (128, d), "R128")
    _want(codes, torch.uint8, (B, Hkv, Ncap, 16), "codes")
    _want(O, torch.float32, (B, Hq, d), "O")
    if idx_out is not None:
        _want(idx_out, torch.int32, (B, Hkv, k), "idx_out")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_HATA_DECODE, B, Hq, Hkv, Ncap, N, d, 16, 8, k), Q.device, ws)
    rc = _lib.lib.hata_decode(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K), _ptr(R128), _ptr(codes), B, Hq, Hkv, Ncap, N,
                              d, k, ctypes.c_float(scale), _ptr(O), _ptr(idx_out), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "hata_decode")


def dense_decode(Q, K, V, N: int, scale: float, O, ws=None):
    """Dense decode attention over the first N cached keys."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    _want(K, Q.dtype, K.shape, "K")
    _want(V, Q.dtype, K.shape, "V")
    _want(O, torch.float32, (B, Hq, d), "O")
    if ws is None:                # a caller's workspace is passed as it is: the library checks its size
        ws = _workspace(workspace_bytes(OP_DENSE_DECODE, B, Hq, Hkv, Ncap, N, d), Q.device, ws)
    rc = _lib.lib.dense_decode(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K), B, Hq, Hkv, Ncap, N, d, ctypes.c_float(scale),
                               _ptr(O), _ptr(ws), _ws_bytes(ws), _stream())
    _check(rc, "dense_decode")


def socket_soft_count_attend(Q, V, R, ids, idx, L: int, P: int, tau: float, O, ws=None):
    """The soft-count attention estimator over the selected keys idx (see the C header)."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = V.shape
    k = idx.shape[-1]
    _want(V, Q.dtype, V.shape, "V")
    _want(R, torch.bfloat16, (L * P, d), "R")
    _want(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _want(idx, torch.int32, (B, Hkv, k), "idx")
    _want(O, torch.float32, (B, Hq, d), "O")
    if ws is None:              # a caller's workspace is passed as it is: the library checks its size
        if ws is None:                # a caller's workspace is passed as it is: the library checks its size
            ws = _workspace(workspace_bytes(OP_SOFT_COUNT, B, Hq, Hkv, Ncap, k, d, L, P, k), Q.device, ws)
    rc = _lib.lib.socket_soft_count_attend(_ptr(Q), _ptr(V), _dtype_code(V), _ptr(R), _ptr(ids), _ptr(idx), B, Hq,
                                           Hkv, Ncap, d, L, P, ctypes.c_float(tau), k, _ptr(O), _ptr(ws),
                                           _ws_bytes(ws), _stream())
    _check(rc, "socket_soft_count_attend")


def check_status():
    """Synchronises the current stream and raises if a kernel flagged an error."""
    _check(_lib.lib.sk_check_status(_stream()), "sk_check_status")


# ---------------------------------------------------------------- quantised caches, blocks, drafted tokens
_CACHE_CODES = {torch.float32: SK_F32, torch.bfloat16: SK_BF16, torch.int8: SK_INT8, torch.float8_e4m3fn: SK_E4M3}


def empty_quant(B: int, Hkv: int, Ncap: int, d: int, dtype=torch.int8, device="cuda"):
    """A quantised cache (Kq, Vq, scales): two [B, Hkv, Ncap, d] of int8 or float8_e4m3fn and [B, Hkv, Ncap, 2] f32."""
    if dtype not in (torch.int8, torch.float8_e4m3fn):
        raise TypeError(f"unsupported cache dtype {dtype} (int8 or float8_e4m3fn)")
    Kq, Vq = (torch.zeros(B, Hkv, Ncap, d, dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
    return Kq, Vq, torch.zeros(B, Hkv, Ncap, 2, dtype=torch.float32, device=device)


def empty_block_summaries(B: int, Hkv: int, Ncap: int, d: int, block: int, device="cuda") -> torch.Tensor:
    """Block summaries [B, Hkv, ceil(Ncap / block), 2, d] bf16: the keys' minima, then their maxima."""
    return torch.zeros(B, Hkv, -(-Ncap // block), 2, d, dtype=torch.bfloat16, device=device)


def tree_mask(seen: torch.Tensor) -> torch.Tensor:
    """[B, T, T] bool (token t sees drafted key i) -> the words of tree_decode's mask [B, T, ceil(T / 32)] int32."""
    B, T, _ = seen.shape
    bits = torch.nn.functional.pad(seen, (0, -T % 32)).view(B, T, -1, 32).long()
    w = (bits << torch.arange(32, device=seen.device)).sum(-1)
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32).contiguous()


def _cache_code(t: torch.Tensor, quantised: bool = False) -> int:
    code = _CACHE_CODES.get(t.dtype)
    if code is None or (quantised and code < SK_INT8):
        raise TypeError(f"unsupported cache dtype {t.dtype}")
    return code


def _addresses(device: int, *tensors):
    """Addresses of contiguous tensors on one CUDA device (None for None)."""
    if device < 0:
        raise ValueError("tensors must live on a CUDA device")
    out = []
    for t in tensors:
        if t is not None:
            if t.get_device() != device:
                raise ValueError(f"tensors on cuda:{device} and {t.device}: one device expected")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
            t = t.data_ptr()
        out.append(t)
    return out


def _run(device: int, what: str, *args):
    """The entry point `what` on the device's current stream, with that device current; raises the library's message."""
    fn = getattr(_lib.lib, what)
    if device == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if rc != 0:
        _check(rc, what)


def _need(t, dtype, shape, name):
    """_want, quick where nothing is wrong."""
    if t.dtype is not dtype or t.shape != shape:
        _want(t, dtype, shape, name)


def _want_cache(K, V, scales, shape, quantised: bool = False):
    """Checks K, V (if any) and their scales against the cache's shape; returns the cache's dtype code."""
    code = _cache_code(K, quantised)
    _need(K, K.dtype, shape, "K")
    if V is not None:
        _need(V, K.dtype, shape, "V")
    if code >= SK_INT8:
        if scales is None:
            raise ValueError("scales: a quantised cache needs them")
        _need(scales, torch.float32, (shape[0], shape[1], shape[2], 2), "scales")
    elif scales is not None:
        raise ValueError(f"scales: a {K.dtype} cache has none")
    return code


def _want_lens(lens, B, name="lens"):
    if lens is not None:
        _need(lens, torch.int32, (B,), name)


def _ws_arg(ws, op, Q, *shape):
    """The workspace: the caller's as it is, or one of the size the library asks for."""
    return ws if ws is not None else torch.empty(workspace_bytes(op, *shape), dtype=torch.uint8, device=Q.device)


def quant_append(K_new, V_new, Kq, Vq, scales, n_begin: int = 0, starts=None, lens=None):
    """Quantises K_new, V_new [B, Hkv, n, d] (f32 or bf16; the last dimension contiguous, the others' strides multiples of 16
    bytes) into rows n_begin .. (or starts[b] ..) of a quantised cache (see the C header)."""
    B, Hkv, Ncap, d = Kq.shape
    n = K_new.shape[2]
    code = _want_cache(Kq, Vq, scales, (B, Hkv, Ncap, d), quantised=True)
    _need(K_new, K_new.dtype, (B, Hkv, n, d), "K_new")
    _need(V_new, K_new.dtype, (B, Hkv, n, d), "V_new")
    _want_lens(starts, B, "starts")
    _want_lens(lens, B)
    strides = K_new.stride()
    if V_new.stride() != strides:         # (that of a dimension of one is arbitrary)
        if any(x != y and size > 1 for x, y, size in zip(V_new.stride(), strides, K_new.shape)):
            raise ValueError(f"V_new: strides {V_new.stride()}, expected K_new's {strides}")
    sb, sh, sn, sd = strides
    if sd != 1:
        raise ValueError("K_new, V_new: the last dimension must be contiguous")
    if B == 1:
        sb = 0
    if Hkv == 1:
        sh = 0
    if n == 1:
        sn = 0
    i = Kq.get_device()
    pk, pv, ps, p_starts, p_lens = _addresses(i, Kq, Vq, scales, starts, lens)
    if K_new.get_device() != i or V_new.get_device() != i:
        raise ValueError(f"tensors on {Kq.device}, {K_new.device} and {V_new.device}: one device expected")
    _run(i, "quant_append", K_new.data_ptr(), V_new.data_ptr(), _dtype_code(K_new), sb, sh, sn, p_starts, p_lens, B, Hkv, Ncap,
         n_begin, n, d, pk, pv, code, ps)


def quant_read(Kq, Vq, scales, K, V, n_begin: int = 0, starts=None, lens=None):
    """Reads rows n_begin .. (or starts[b] ..) of a quantised cache back into K, V [B, Hkv, n, d] (f32 or bf16)."""
    B, Hkv, Ncap, d = Kq.shape
    n = K.shape[2]
    code = _want_cache(Kq, Vq, scales, (B, Hkv, Ncap, d), quantised=True)
    _need(K, K.dtype, (B, Hkv, n, d), "K")
    _need(V, K.dtype, (B, Hkv, n, d), "V")
    _want_lens(starts, B, "starts")
    _want_lens(lens, B)
    i = Kq.get_device()
    pkq, pvq, ps, p_starts, p_lens, pk, pv = _addresses(i, Kq, Vq, scales, starts, lens, K, V)
    _run(i, "quant_read", pkq, pvq, code, ps, p_starts, p_lens, B, Hkv, Ncap, n_begin, n, d, pk, pv, _dtype_code(K))


def quant_decode(Q, Kq, Vq, scales, N: int, scale: float, O, lens=None, ws=None):
    """Dense decode attention over a quantised cache: O [B, Hq, d] f32 (see the C header)."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = Kq.shape
    code = _want_cache(Kq, Vq, scales, (B, Hkv, Ncap, d), quantised=True)
    _need(O, torch.float32, (B, Hq, d), "O")
    _want_lens(lens, B)
    i = Q.get_device()
    ws = _ws_arg(ws, OP_QUANT_DECODE, Q, B, Hq, Hkv, Ncap, N, d)
    pq, pk, pv, ps, pl, po, pw = _addresses(i, Q, Kq, Vq, scales, lens, O, ws)
    _run(i, "quant_decode", pq, _dtype_code(Q), pk, pv, code, ps, pl, B, Hq, Hkv, Ncap, N, d, scale, po, pw, _ws_bytes(ws))


def quant_sparse_attend(Q, Kq, Vq, scales, idx, scale: float, O, ws=None):
    """Attention over listed rows idx [B, Hkv, k] int32 (-1: none) of a quantised cache: O [B, Hq, d] f32."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = Kq.shape
    k = idx.shape[-1]
    code = _want_cache(Kq, Vq, scales, (B, Hkv, Ncap, d), quantised=True)
    _need(idx, torch.int32, (B, Hkv, k), "idx")
    _need(O, torch.float32, (B, Hq, d), "O")
    i = Q.get_device()
    ws = _ws_arg(ws, OP_QUANT_SPARSE_ATTEND, Q, B, Hq, Hkv, Ncap, k, d, 0, 0, k)
    pq, pk, pv, ps, pi, po, pw = _addresses(i, Q, Kq, Vq, scales, idx, O, ws)
    _run(i, "quant_sparse_attend", pq, _dtype_code(Q), pk, pv, code, ps, pi, B, Hq, Hkv, Ncap, d, k, scale, po, pw, _ws_bytes(ws))


def socket_decode_quant(Q, Kq, Vq, scales, R, ids, norms, N: int, L: int, P: int, tau: float, k: int, scale: float, O,
                        idx_out=None, ws=None):
    """socket_decode over a quantised K/V cache (the hashed-key cache as there): O [B, Hq, d] f32."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = Kq.shape
    code = _want_cache(Kq, Vq, scales, (B, Hkv, Ncap, d), quantised=True)
    _need(R, torch.bfloat16, (L * P, d), "R")
    _need(ids, torch.uint8, (B, Hkv, Ncap, ids_bytes_per_key(L)), "ids")
    _need(norms, torch.float16, (B, Hkv, Ncap), "norms")
    _need(O, torch.float32, (B, Hq, d), "O")
    if idx_out is not None:
        _need(idx_out, torch.int32, (B, Hkv, k), "idx_out")
    i = Q.get_device()
    ws = _ws_arg(ws, OP_SOCKET_DECODE_QUANT, Q, B, Hq, Hkv, Ncap, N, d, L, P, k)
    pq, pk, pv, ps, pr, p_ids, pn, po, pi, pw = _addresses(i, Q, Kq, Vq, scales, R, ids, norms, O, idx_out, ws)
    _run(i, "socket_decode_quant", pq, _dtype_code(Q), pk, pv, code, ps, pr, p_ids, pn, B, Hq, Hkv, Ncap, N, d, L, P, tau, k, scale,
         po, pi, pw, _ws_bytes(ws))


def block_summarize(K, block: int, bsum, n_begin: int = 0, n_count: int | None = None, scales=None, starts=None, lens=None):
    """Summaries (per-channel minima and maxima) of the blocks that hold rows [n_begin, n_begin + n_count) of each pair."""
    B, Hkv, Ncap, d = K.shape
    n_count = Ncap - n_begin if n_count is None else n_count
    code = _want_cache(K, None, scales, (B, Hkv, Ncap, d))
    _need(bsum, torch.bfloat16, (B, Hkv, -(-Ncap // block) if block > 0 else 0, 2, d), "bsum")
    _want_lens(starts, B, "starts")
    _want_lens(lens, B)
    i = K.get_device()
    pk, ps, p_starts, p_lens, pb = _addresses(i, K, scales, starts, lens, bsum)
    _run(i, "block_summarize", pk, code, ps, p_starts, p_lens, B, Hkv, Ncap, n_begin, n_count, d, block, pb)


def _block_shapes(Q, bsum, Ncap, block):
    B, Hq, d = Q.shape
    Hkv = bsum.shape[1]
    _need(bsum, torch.bfloat16, (B, Hkv, -(-Ncap // block) if block > 0 else 0, 2, d), "bsum")
    return B, Hq, Hkv, d


def block_select(Q, bsum, Ncap: int, N: int, block: int, n_first: int, n_last: int, idx, lens=None, ws=None):
    """The idx.shape[-1] blocks of each pair with the largest bounds: idx [B, Hkv, k] int32, ascending, then -1."""
    B, Hq, Hkv, d = _block_shapes(Q, bsum, Ncap, block)
    k = idx.shape[-1]
    _need(idx, torch.int32, (B, Hkv, k), "idx")
    _want_lens(lens, B)
    i = Q.get_device()
    ws = _ws_arg(ws, OP_BLOCK_SELECT, Q, B, Hq, Hkv, Ncap, N, d, block, 0, k)
    pq, pb, pl, pi, pw = _addresses(i, Q, bsum, lens, idx, ws)
    _run(i, "block_select", pq, _dtype_code(Q), pb, pl, B, Hq, Hkv, Ncap, N, d, block, k, n_first, n_last, pi, pw, _ws_bytes(ws))


def block_attend(Q, K, V, N: int, block: int, idx, scale: float, O, scales=None, lens=None, ws=None):
    """Attention over the keys of the listed blocks idx [B, Hkv, k] int32 (-1: none): O [B, Hq, d] f32."""
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    k = idx.shape[-1]
    code = _want_cache(K, V, scales, (B, Hkv, Ncap, d))
    _need(idx, torch.int32, (B, Hkv, k), "idx")
    _need(O, torch.float32, (B, Hq, d), "O")
    _want_lens(lens, B)
    i = Q.get_device()
    ws = _ws_arg(ws, OP_BLOCK_ATTEND, Q, B, Hq, Hkv, Ncap, N, d, block, 0, k)
    pq, pk, pv, ps, pl, pi, po, pw = _addresses(i, Q, K, V, scales, lens, idx, O, ws)
    _run(i, "block_attend", pq, _dtype_code(Q), pk, pv, code, ps, pl, pi, B, Hq, Hkv, Ncap, N, d, block, k, scale, po, pw,
         _ws_bytes(ws))


def block_decode(Q, K, V, bsum, N: int, block: int, k: int, n_first: int, n_last: int, scale: float, O, scales=None, lens=None,
                 idx_out=None, ws=None):
    """block_select, then block_attend over its choice: O [B, Hq, d] f32; idx_out [B, Hkv, k] int32 if given."""
    Ncap = K.shape[2]
    B, Hq, Hkv, d = _block_shapes(Q, bsum, Ncap, block)
    code = _want_cache(K, V, scales, (B, Hkv, Ncap, d))
    _need(O, torch.float32, (B, Hq, d), "O")
    if idx_out is not None:
        _need(idx_out, torch.int32, (B, Hkv, k), "idx_out")
    _want_lens(lens, B)
    i = Q.get_device()
    ws = _ws_arg(ws, OP_BLOCK_DECODE, Q, B, Hq, Hkv, Ncap, N, d, block, 0, k)
    pq, pk, pv, ps, pb, pl, po, pi, pw = _addresses(i, Q, K, V, scales, bsum, lens, O, idx_out, ws)
    _run(i, "block_decode", pq, _dtype_code(Q), pk, pv, code, ps, pb, pl, B, Hq, Hkv, Ncap, N, d, block, k, n_first, n_last, scale,
         po, pi, pw, _ws_bytes(ws))


def tree_decode(Q, K, V, N: int, scale: float, O, mask=None, scales=None, lens=None, ws=None):
    """Attention of T drafted tokens Q [B, T, Hq, d] over each sequence's cached keys and, under mask (tree_mask; None: a
    chain), its drafted keys behind them: O [B, T, Hq, d] f32 or bf16 (see the C header)."""
    B, T, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    code = _want_cache(K, V, scales, (B, Hkv, Ncap, d))
    _need(O, O.dtype, (B, T, Hq, d), "O")
    if mask is not None:
        _need(mask, torch.int32, (B, T, -(-T // 32)), "mask")
    _want_lens(lens, B)
    i = Q.get_device()
    ws = _ws_arg(ws, OP_TREE_DECODE, Q, B, Hq, Hkv, Ncap, N, d, 0, 0, T)
    pq, pk, pv, ps, pl, pm, po, pw = _addresses(i, Q, K, V, scales, lens, mask, O, ws)
    _run(i, "tree_decode", pq, _dtype_code(Q), pk, pv, code, ps, pl, pm, B, T, Hq, Hkv, Ncap, N, d, scale, po, _dtype_code(O), pw,
         _ws_bytes(ws))
