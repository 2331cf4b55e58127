"""memory_efficient_exact_mea_b200 -- memory-efficient exact attention on B200.

A thin ctypes binding of ``libmea.so`` (C ABI in ``include/mea.h``).  This module
only marshals arguments: every step of the computation runs in the library's
sm_100a kernels.  PyTorch supplies device memory and the current stream.  There
is no fallback: importing this package fails loudly if ``libmea.so`` is missing.

Operations (sources cited in ``include/mea.h``):
  mea_fwd     softmax(Q K^T * scale + bias) V and the per-row log-sum-exp, with
              no / causal / block-diagonal (causal) masks, GQA and ALiBi.
  mea_fwd_block_sparse  mea_fwd with whole 128x128 score blocks left out by a mask.
  mea_prefill_chunk  a chunk of new queries against a KV cache, appending its keys/values.
  mea_bwd     dq, dk, dv by recomputing the weights from the forward's lse.
  mea_decode  one query per sequence against a packed, ragged KV cache.
  mea_kv4_append, mea_kv4_read, mea_decode_kv4  a KV cache held in 4 bits: rows put
              into it, rows read back in 16 bits, one decode step against it.
  mea_key_weights  the attention weight each key gathered, from q, k and the lse.
  mea_cache_evict  a cache cut down to its newest and heaviest rows.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

__all__ = ["mea_fwd", "mea_fwd_block_sparse", "mea_prefill_chunk", "mea_bwd", "mea_decode",
           "mea_decode_workspace_size", "mea_decode_chunk", "Kv4Cache", "mea_kv4_alloc",
           "mea_kv4_append", "mea_kv4_read", "mea_decode_kv4", "mea_decode_kv4_workspace_size",
           "mea_key_weights", "mea_cache_evict", "read_device_status", "status_string",
           "MeaError", "PreparedCall", "BIAS", "BWD_PREP", "BWD_MAIN", "BWD_DQ", "LIB_PATH", "lib"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmea.so")

BIAS = {"none": 0, "causal": 1, "blockdiag": 2, "blockdiag_causal": 3}
BWD_PREP, BWD_MAIN, BWD_DQ = 1, 2, 4  # stages of the backward (mea_bwd_stages)
_DTYPE = {torch.float16: 0, torch.bfloat16: 1}
_i64x3 = ctypes.c_int64 * 3


class _Plane(ctypes.Structure):  # mea_plane_t
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("src_strides", _i64x3),
                ("dst_strides", _i64x3), ("row_bytes", ctypes.c_int32)]


class MeaError(RuntimeError):
    """A libmea entry point returned an error status."""

    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {status_string(code)} ({code})")
        self.code = code


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python memory_efficient_exact_mea_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.mea_fwd.restype = i
    L.mea_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, vp, vp, i, i, vp, vp,
                          i, i, i, i, f, vp]
    L.mea_decode_workspace_size.restype = sz
    L.mea_decode_workspace_size.argtypes = [i, i, i, i, i]
    L.mea_decode.restype = i
    L.mea_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp, sz, vp]
    L.mea_fwd_block_sparse.restype = i
    L.mea_fwd_block_sparse.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, vp, vp, i, i,
                                       vp, vp, i, f, vp]
    L.mea_prefill_chunk.restype = i
    L.mea_prefill_chunk.argtypes = [vp] * 9 + [i] * 6 + [vp] * 6 + [i, i, i, f, vp]
    L.mea_sparse_block_size.restype = i
    L.mea_sparse_block_size.argtypes = []
    L.mea_bwd_workspace_size.restype = sz
    L.mea_bwd_workspace_size.argtypes = [i, i, i, i]
    L.mea_bwd.restype = i
    L.mea_bwd.argtypes = [vp] * 9 + [i] * 8 + [vp, vp, i, i, i, i, f, vp, sz, vp]
    L.mea_bwd_stages.restype = i
    L.mea_bwd_stages.argtypes = [vp] * 9 + [i] * 8 + [vp, vp, i, i, i, i, f, vp, sz, i, vp]
    L.mea_kv4_append.restype = i
    L.mea_kv4_append.argtypes = [vp] * 8 + [i] * 5 + [vp, vp, i, vp]
    L.mea_kv4_read.restype = i
    L.mea_kv4_read.argtypes = [vp] * 8 + [i] * 5 + [vp, vp, i, vp]
    L.mea_decode_kv4_workspace_size.restype = sz
    L.mea_decode_kv4_workspace_size.argtypes = [i] * 6
    L.mea_decode_kv4.restype = i
    L.mea_decode_kv4.argtypes = [vp] * 10 + [i] * 8 + [f, vp, sz, vp]
    L.mea_key_weights.restype = i
    L.mea_key_weights.argtypes = [vp] * 7 + [i] * 6 + [vp, vp, i, i, i, f, vp]
    L.mea_cache_evict.restype = i
    L.mea_cache_evict.argtypes = [ctypes.POINTER(_Plane), i] + [vp] * 5 + [i] * 6 + [vp]
    L.mea_decode_chunk.restype = i
    L.mea_decode_chunk.argtypes = []
    L.mea_status_string.restype = ctypes.c_char_p
    L.mea_status_string.argtypes = [i]
    L.mea_read_device_status.restype = i
    L.mea_read_device_status.argtypes = [vp, i]
    L.mea_version.restype = i
    L.mea_version.argtypes = []
    return L


lib = _load()


def status_string(code: int) -> str:
    return lib.mea_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None):
    """The CUDA stream handle to launch on: `stream`, else the current stream of
    `device` (a torch.device, default the current device)."""
    if stream is None:
        if _raw_stream is not None and device is not None and device.index is not None:
            return ctypes.c_void_p(_raw_stream(device.index))
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise MeaError(fn, rc)


_STRIDES: dict = {}  # (sb, sm, sh) -> ctypes int64[3], reused across calls (read-only)



def _bmhk_strides(t: torch.Tensor, name: str):
    st = t.stride()
    if len(st) != 4:
        raise ValueError(f"{name} must be [B, rows, heads, K]")
    if st[3] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    key = st[:3]
    arr = _STRIDES.get(key)
    if arr is None:
        if len(_STRIDES) > 4096:
            _STRIDES.clear()
        arr = _STRIDES[key] = _i64x3(*key)
    return arr


def _grouped_views(q, k, v, out):
    """The 5-D grouped-query layout as 4-D views (no copy): q [B,M,G,H,K] ->
    [B,M,G*H,K] (query head g*H + r); k, v [B,N,G,1,K], or [B,N,G,H,K] expanded
    along H with stride 0, -> [B,N,G,K] (key/value head g, shared by the H query
    heads of group g); k, v with a real H axis -> [B,N,G*H,K]."""
    B, M, G, H, K = q.shape
    if k.dim() != 5 or v.dim() != 5 or k.shape[:3] != v.shape[:3] or k.shape[2] != G:
        raise ValueError("5-D q [B,M,G,H,K] needs k, v [B,N,G,1|H,K]")

    def flat(t, name):
        if t.shape[3] != 1 and t.stride(2) != t.shape[3] * t.stride(3):
            raise ValueError(f"{name}: the group and head axes must merge into one (a view)")
        return t.flatten(2, 3)

    def kv4(t, name):
        if t.shape[3] == 1 or t.stride(3) == 0:
            return t[:, :, :, 0]
        return flat(t, name)

    q4 = flat(q, "q")
    o4 = None if out is None else flat(out, "out")
    return q4, kv4(k, "k"), kv4(v, "v"), o4


class PreparedCall:
    """One C-ABI call with every argument marshalled once, for launching the same
    computation again and again (a serving or training loop whose buffers stay
    put): calling it only runs the C entry point, on the stream chosen when it
    was prepared.  It keeps the tensors it points into alive.  `outputs` holds
    what the call writes."""

    __slots__ = ("_fn", "_args", "_name", "_keep", "outputs")

    def __init__(self, fn, args, name, keep, outputs):
        self._fn, self._args, self._name, self._keep, self.outputs = fn, args, name, keep, outputs

    def __call__(self):
        rc = self._fn(*self._args)
        if rc != 0:
            raise MeaError(self._name, rc)
        return self.outputs


def mea_fwd(q, k, v, bias: str = "none", scale: float | None = None, alibi: bool = False,
            seqstart_q=None, seqstart_k=None, max_seqlen_q: int | None = None,
            max_seqlen_k: int | None = None, out=None, lse=None, return_lse: bool = True,
            stream=None, prepare: bool = False):
    """Attention forward.  q [B,M,Hq,K], k/v [B,N,Hkv,K] (fp16/bf16, CUDA) ->
    (out [B,M,Hq,K], lse [B,Hq,M] fp32 or None).

    bias: "none" | "causal" | "blockdiag" | "blockdiag_causal".  The block-diagonal
    kinds take B == 1 and int32 CUDA offsets ``seqstart_q`` (and ``seqstart_k``);
    ``max_seqlen_q`` is the longest query sequence (read from the offsets, with a
    device-to-host copy, when not given).

    Grouped-query 5-D layout: q [B,M,G,H,K] with k, v [B,N,G,1,K] (or expanded to
    [B,N,G,H,K] with stride 0) is the same call with Hq = G*H query heads and
    Hkv = G key/value heads, query head g*H + r reading key/value head g; out is
    returned as [B,M,G,H,K] and lse as [B,G*H,M].

    prepare=True launches nothing and returns a PreparedCall instead: each call
    of it runs this forward again on the same buffers (its outputs are
    (out, lse)), with no Python-side argument handling.
    """
    if q.dim() == 5:
        if prepare:
            raise ValueError("prepare=True takes the 4-D layout")
        shape5 = tuple(q.shape)
        q, k, v, out4 = _grouped_views(q, k, v, out)
        o, l = mea_fwd(q, k, v, bias, scale, alibi, seqstart_q, seqstart_k, max_seqlen_q,
                       max_seqlen_k, out4, lse, return_lse, stream)
        return o.view(shape5) if out is None else out, l
    B, M, Hq, K = q.shape
    N, Hkv = k.shape[1], k.shape[2]
    if q.dtype not in _DTYPE or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share dtype float16 or bfloat16")
    if tuple(k.shape) != (B, N, Hkv, K) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, N, Hkv, K]")
    scale = K ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, M, Hq, K), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, M), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [B, Hq, M] tensor")
    kind = BIAS[bias]
    ns = 0
    if kind >= 2:
        if seqstart_q is None:
            raise ValueError("block-diagonal bias needs seqstart_q")
        for s in (seqstart_q, seqstart_k):
            if s is not None and (s.dtype != torch.int32 or not s.is_cuda):
                raise ValueError("seqstart offsets must be int32 CUDA tensors")
        ns = seqstart_q.numel() - 1
        if max_seqlen_q is None:
            max_seqlen_q = int(torch.diff(seqstart_q).max().item()) if ns > 0 else 0
        if max_seqlen_k is None:
            sk = seqstart_q if seqstart_k is None else seqstart_k
            max_seqlen_k = int(torch.diff(sk).max().item()) if ns > 0 else 0
    else:
        seqstart_q = seqstart_k = None
        max_seqlen_q = max_seqlen_k = 0
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, M, N, Hq, Hkv, K,
            _bmhk_strides(q, "q"), _bmhk_strides(k, "k"), _bmhk_strides(v, "v"),
            _bmhk_strides(out, "out"), _DTYPE[q.dtype], kind, _ptr(seqstart_q), _ptr(seqstart_k),
            ns, int(max_seqlen_q), int(max_seqlen_k), int(bool(alibi)), scale,
            _stream(stream, q.device))
    if prepare:
        return PreparedCall(lib.mea_fwd, args, "mea_fwd",
                            (q, k, v, out, lse, seqstart_q, seqstart_k), (out, lse))
    _check("mea_fwd", lib.mea_fwd(*args))
    return out, lse


def mea_fwd_block_sparse(q, k, v, block_mask, bias: str = "none", scale: float | None = None,
                         alibi: bool = False, out=None, lse=None, return_lse: bool = True,
                         stream=None):
    """Block-sparse attention forward.  As ``mea_fwd`` (bias "none" or "causal"),
    plus ``block_mask``: a uint8 CUDA tensor [B, Hq, ceil(M/128), ceil(N/128)]
    (size-1 or stride-0 batch/head dimensions broadcast; the last two dimensions
    contiguous); a zero entry leaves that 128x128 block of scores out."""
    B, M, Hq, K = q.shape
    N, Hkv = k.shape[1], k.shape[2]
    if q.dtype not in _DTYPE or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share dtype float16 or bfloat16")
    if tuple(k.shape) != (B, N, Hkv, K) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, N, Hkv, K]")
    blk = int(lib.mea_sparse_block_size())
    mb, nb = -(-M // blk), -(-N // blk)
    if (block_mask.dtype != torch.uint8 or block_mask.dim() != 4 or not block_mask.is_cuda
            or tuple(block_mask.shape[2:]) != (mb, nb)
            or block_mask.shape[0] not in (1, B) or block_mask.shape[1] not in (1, Hq)):
        raise ValueError(f"block_mask must be a uint8 CUDA tensor [B|1, Hq|1, {mb}, {nb}]")
    if block_mask.stride(3) != 1 or block_mask.stride(2) != nb:
        raise ValueError("block_mask: the last two dimensions must be contiguous")
    mst = (ctypes.c_int64 * 2)(block_mask.stride(0) if block_mask.shape[0] > 1 else 0,
                               block_mask.stride(1) if block_mask.shape[1] > 1 else 0)
    scale = K ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, M, Hq, K), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, M), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [B, Hq, M] tensor")
    rc = lib.mea_fwd_block_sparse(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, M, N, Hq,
                                  Hkv, K, _bmhk_strides(q, "q"), _bmhk_strides(k, "k"),
                                  _bmhk_strides(v, "v"), _bmhk_strides(out, "out"),
                                  _DTYPE[q.dtype], BIAS[bias], _ptr(block_mask), mst,
                                  int(bool(alibi)), scale, _stream(stream, q.device))
    _check("mea_fwd_block_sparse", rc)
    return out, lse


def mea_prefill_chunk(q, k_new, v_new, k_cache, v_cache, cache_seqlens, q_seqlens=None,
                      causal: bool = True, scale: float | None = None, alibi: bool = False,
                      out=None, lse=None, return_lse: bool = True, stream=None):
    """One prefill chunk against a KV cache, with the append fused in.

    q [B,M,Hq,K], k_new/v_new [B,M,Hkv,K], k_cache/v_cache [B,cap,Hkv,K] (updated
    in place: rows cache_seqlens[b] .. + q_seqlens[b] receive the chunk's keys and
    values), cache_seqlens / q_seqlens int32 CUDA [B] (q_seqlens None: every
    sequence has M new rows).  Returns (out [B,M,Hq,K], lse [B,Hq,M] or None);
    rows past q_seqlens[b] are not written.  The caller advances cache_seqlens."""
    B, M, Hq, K = q.shape
    cap, Hkv = k_cache.shape[1], k_cache.shape[2]
    ts = (q, k_new, v_new, k_cache, v_cache)
    if q.dtype not in _DTYPE or any(t.dtype != q.dtype for t in ts):
        raise ValueError("q, k_new, v_new, k_cache, v_cache must share dtype float16 or bfloat16")
    if tuple(k_new.shape) != (B, M, Hkv, K) or tuple(v_new.shape) != (B, M, Hkv, K):
        raise ValueError("k_new and v_new must be [B, M, Hkv, K]")
    if tuple(k_cache.shape) != (B, cap, Hkv, K) or tuple(v_cache.shape) != (B, cap, Hkv, K):
        raise ValueError("k_cache and v_cache must be [B, cap, Hkv, K]")
    for name, t in (("cache_seqlens", cache_seqlens), ("q_seqlens", q_seqlens)):
        if t is not None and (t.dtype != torch.int32 or not t.is_cuda or t.numel() != B):
            raise ValueError(f"{name} must be an int32 CUDA tensor of B entries")
    scale = K ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, M, Hq, K), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, M), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [B, Hq, M] tensor")
    rc = lib.mea_prefill_chunk(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                               _ptr(cache_seqlens), _ptr(q_seqlens), _ptr(out), _ptr(lse), B, M,
                               cap, Hq, Hkv, K, _bmhk_strides(q, "q"),
                               _bmhk_strides(k_new, "k_new"), _bmhk_strides(v_new, "v_new"),
                               _bmhk_strides(k_cache, "k_cache"),
                               _bmhk_strides(v_cache, "v_cache"), _bmhk_strides(out, "out"),
                               _DTYPE[q.dtype], int(bool(causal)), int(bool(alibi)), scale,
                               _stream(stream, q.device))
    _check("mea_prefill_chunk", rc)
    return out, lse


def mea_bwd(q, k, v, out, dout, lse, bias: str = "none", scale: float | None = None,
            alibi: bool = False, seqstart_q=None, seqstart_k=None,
            max_seqlen_q: int | None = None, max_seqlen_k: int | None = None,
            dq=None, dk=None, dv=None, workspace=None, stages: int = 7, stream=None):
    """Attention backward.  Contiguous q/out/dout [B,M,Hq,K], k/v [B,N,Hkv,K] and the
    forward's lse [B,Hq,M] -> (dq, dk, dv) shaped like q, k, v.

    ``stages`` (bitwise OR of BWD_PREP, BWD_MAIN, BWD_DQ; default all) runs only
    those launches of the backward (mea_bwd_stages); running them one at a time
    with the same arguments and workspace equals one full call."""
    B, M, Hq, K = q.shape
    N, Hkv = k.shape[1], k.shape[2]
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout), ("lse", lse)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if q.dtype not in _DTYPE or any(t.dtype != q.dtype for t in (k, v, out, dout)):
        raise ValueError("q, k, v, out, dout must share dtype float16 or bfloat16")
    scale = K ** -0.5 if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = int(lib.mea_bwd_workspace_size(B, M, Hq, K))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    kind = BIAS[bias]
    ns = 0
    if kind >= 2:
        ns = seqstart_q.numel() - 1
        if max_seqlen_q is None:
            max_seqlen_q = int(torch.diff(seqstart_q).max().item()) if ns > 0 else 0
        if max_seqlen_k is None:
            sk = seqstart_q if seqstart_k is None else seqstart_k
            max_seqlen_k = int(torch.diff(sk).max().item()) if ns > 0 else 0
    else:
        seqstart_q = seqstart_k = None
        max_seqlen_q = max_seqlen_k = 0
    rc = lib.mea_bwd_stages(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
                            _ptr(dq), _ptr(dk), _ptr(dv), B, M, N, Hq, Hkv, K, _DTYPE[q.dtype],
                            kind, _ptr(seqstart_q), _ptr(seqstart_k), ns, int(max_seqlen_q),
                            int(max_seqlen_k), int(bool(alibi)), scale, _ptr(workspace), ws_bytes,
                            int(stages), _stream(stream, q.device))
    _check("mea_bwd", rc)
    return dq, dk, dv


def mea_decode_workspace_size(B: int, Hq: int, Hkv: int, K: int, max_kv_len: int) -> int:
    return int(lib.mea_decode_workspace_size(B, Hq, Hkv, K, max_kv_len))


def mea_decode_chunk() -> int:
    return int(lib.mea_decode_chunk())


def mea_decode(q, k_cache, v_cache, kv_seqstart, max_kv_len: int, scale: float | None = None,
               alibi: bool = False, out=None, lse=None, workspace=None, return_lse: bool = True,
               stream=None):
    """One decode step.  q [B,Hq,K] or [B,1,Hq,K]; caches [T,Hkv,K]; kv_seqstart int32
    CUDA [B+1] -> (out shaped like q, lse [B,Hq] fp32 or None)."""
    qshape = tuple(q.shape)
    q3 = q.reshape(q.shape[0], q.shape[-2], q.shape[-1])
    B, Hq, K = q3.shape
    T, Hkv = k_cache.shape[0], k_cache.shape[1]
    for name, t in (("q", q3), ("k_cache", k_cache), ("v_cache", v_cache)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if tuple(v_cache.shape) != tuple(k_cache.shape) or k_cache.shape[2] != K:
        raise ValueError("caches must be [T, Hkv, K]")
    if q.dtype not in _DTYPE or k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise ValueError("q and caches must share dtype float16 or bfloat16")
    if kv_seqstart.dtype != torch.int32 or not kv_seqstart.is_cuda:
        raise ValueError("kv_seqstart must be an int32 CUDA tensor")
    scale = K ** -0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty(qshape, dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = mea_decode_workspace_size(B, Hq, Hkv, K, max_kv_len)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.mea_decode(_ptr(q3), _ptr(k_cache), _ptr(v_cache), _ptr(kv_seqstart), _ptr(out),
                        _ptr(lse), B, Hq, Hkv, K, T, int(max_kv_len), _DTYPE[q.dtype],
                        int(bool(alibi)), scale, _ptr(workspace), ws_bytes, _stream(stream, q.device))
    _check("mea_decode", rc)
    return out, lse


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(name, fn, index, stream, args):
    """Runs fn(*args, stream) with CUDA device `index` current."""
    if stream is None:
        raw = _raw_stream(index) if _raw_stream is not None else \
            torch.cuda.current_stream(index).cuda_stream
    else:
        raw = stream.cuda_stream
    if index == _current_device():
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != 0:
        raise MeaError(name, rc)


def _on_stream(index, stream):
    """stream, if given, belongs to CUDA device `index`."""
    if stream is not None and stream.device_index != index:
        raise ValueError(f"stream must be a stream of cuda:{index}")


def _empty(shape, dtype, device, stream, returned=True):
    """An uninitialised tensor for a call that runs on `stream` (None: the current one).  It
    is allocated on that stream: memory freed on the current stream may still be in use by
    work queued there, which nothing orders before the call.  If the caller gets it, its
    current stream counts as a user of the memory too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned and current != stream:
        t.record_stream(current)
    return t


def _addr(t):
    return None if t is None else t.data_ptr()


def _cuda_index(t, name):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _elsewhere(name, index):
    return ValueError(f"{name} must be a CUDA tensor on cuda:{index}")


def _on(index, t, name):
    """t, if given, lies on CUDA device `index`."""
    if t is not None and t.get_device() != index:
        raise _elsewhere(name, index)


_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


def _lens(B, index, t, name):
    """t, if given, is one int32 a sequence on CUDA device `index`."""
    if t is not None and (t.dtype is not _I32 or t.get_device() != index or t.dim() != 1
                          or t.numel() != B or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of B entries on cuda:{index}")


def _f32(t, shape, index, name):
    """t, if given, is a contiguous float32 tensor of `shape` on CUDA device `index`."""
    if t is not None and (t.dtype is not _F32 or t.shape != shape or t.get_device() != index
                          or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 {list(shape)} tensor on "
                         f"cuda:{index}")


class Kv4Cache(NamedTuple):
    """The planes of a 4-bit KV cache (see mea_kv4_append in ``include/mea.h``):
    codes uint8 [B, Hkv, rows, K/2] and params [B, Hkv, rows, K/64, 2] (step and zero,
    float16 or bfloat16) of the keys and of the values, all contiguous."""

    k_codes: torch.Tensor
    k_params: torch.Tensor
    v_codes: torch.Tensor
    v_params: torch.Tensor


def mea_kv4_alloc(B: int, cache_rows: int, Hkv: int, K: int, dtype=torch.bfloat16,
                  device="cuda") -> Kv4Cache:
    """An uninitialised 4-bit cache for rows of `dtype` (float16 or bfloat16)."""
    if dtype not in _DTYPE:
        raise ValueError("dtype must be float16 or bfloat16")
    if K not in (64, 128):
        raise ValueError("K must be 64 or 128")
    planes = []
    for _ in range(2):
        planes.append(torch.empty((B, Hkv, cache_rows, K // 2), dtype=torch.uint8, device=device))
        planes.append(torch.empty((B, Hkv, cache_rows, K // 64, 2), dtype=dtype, device=device))
    return Kv4Cache(*planes)


def _kv4_dims(cache: Kv4Cache, what="cache"):
    """(B, Hkv, rows, K, dtype, device index) of a 4-bit cache, checked."""
    kc, kp, vc, vp = cache
    shape = kc.shape
    if len(shape) != 4 or kc.dtype is not _U8:
        raise ValueError(f"{what}: codes must be uint8 [B, Hkv, rows, K/2]")
    B, Hkv, rows, half = shape
    dtype = kp.dtype
    if dtype not in _DTYPE or vp.dtype != dtype:
        raise ValueError(f"{what}: params must share dtype float16 or bfloat16")
    if vc.dtype is not _U8 or vc.shape != shape:
        raise ValueError(f"{what}: k_codes and v_codes must be alike")
    want = (B, Hkv, rows, half // 32, 2)
    if half % 32 or kp.shape != want or vp.shape != want:
        raise ValueError(f"{what}: params must be [B, Hkv, rows, K/64, 2]")
    if not (kc.is_contiguous() and kp.is_contiguous() and vc.is_contiguous()
            and vp.is_contiguous()):
        raise ValueError(f"{what}: the planes must be contiguous")
    index = _cuda_index(kc, what)
    if kp.get_device() != index or vc.get_device() != index or vp.get_device() != index:
        raise ValueError(f"{what}: the planes must lie on one device")
    return B, Hkv, rows, 2 * half, dtype, index


def mea_kv4_append(k_new, v_new, cache: Kv4Cache, cache_seqlens, q_seqlens=None, stream=None):
    """Puts new rows into a 4-bit cache.  k_new/v_new [B,M,Hkv,K] (any (b, m, h) strides),
    cache_seqlens / q_seqlens int32 CUDA [B] (rows already there, and rows of the chunk, M
    if None): rows cache_seqlens[b] .. + q_seqlens[b] of the cache are written.  The caller
    advances cache_seqlens.  Returns the cache."""
    B, Hkv, rows, K, dtype, index = _kv4_dims(cache)
    shape = k_new.shape
    M = shape[1] if len(shape) == 4 else 0
    if shape != (B, M, Hkv, K) or v_new.shape != shape:
        raise ValueError("k_new and v_new must be [B, M, Hkv, K]")
    if k_new.dtype != dtype or v_new.dtype != dtype:
        raise ValueError("k_new and v_new must have the dtype of the cache's params")
    _on(index, k_new, "k_new")
    _on(index, v_new, "v_new")
    _lens(B, index, cache_seqlens, "cache_seqlens")
    _lens(B, index, q_seqlens, "q_seqlens")
    _on_stream(index, stream)
    kc, kp, vc, vp = cache
    _launch("mea_kv4_append", lib.mea_kv4_append, index, stream,
            (k_new.data_ptr(), v_new.data_ptr(), kc.data_ptr(), kp.data_ptr(), vc.data_ptr(),
             vp.data_ptr(), cache_seqlens.data_ptr(), _addr(q_seqlens), B, M, rows, Hkv, K,
             _bmhk_strides(k_new, "k_new"), _bmhk_strides(v_new, "v_new"), _DTYPE[dtype]))
    return cache


def mea_kv4_read(cache: Kv4Cache, rows, first_rows=None, k_out=None, v_out=None,
                 out_rows: int | None = None, stream=None):
    """Rows first_rows[b] .. + rows[b] (from row 0 if None) of a 4-bit cache in 16 bits:
    (k, v), each [B, out_rows, Hkv, K] (out_rows defaults to the cache's rows, or to that of
    k_out); rows past rows[b] are not written."""
    B, Hkv, cap, K, dtype, index = _kv4_dims(cache)
    if out_rows is None:
        ref = k_out if k_out is not None else v_out
        out_rows = cap if ref is None else ref.shape[1]
    _on_stream(index, stream)
    shape = (B, int(out_rows), Hkv, K)
    if k_out is None:
        k_out = _empty(shape, dtype, cache.k_codes.device, stream)
    if v_out is None:
        v_out = _empty(shape, dtype, cache.k_codes.device, stream)
    if k_out.shape != shape or v_out.shape != shape or k_out.dtype != dtype \
            or v_out.dtype != dtype:
        raise ValueError(f"k_out and v_out must be {list(shape)} of the params' dtype")
    _on(index, k_out, "k_out")
    _on(index, v_out, "v_out")
    _lens(B, index, rows, "rows")
    _lens(B, index, first_rows, "first_rows")
    kc, kp, vc, vp = cache
    _launch("mea_kv4_read", lib.mea_kv4_read, index, stream,
            (kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), rows.data_ptr(),
             _addr(first_rows), k_out.data_ptr(), v_out.data_ptr(), B, cap, shape[1], Hkv, K,
             _bmhk_strides(k_out, "k_out"), _bmhk_strides(v_out, "v_out"), _DTYPE[dtype]))
    return k_out, v_out


def mea_decode_kv4_workspace_size(B: int, Hq: int, Hkv: int, K: int, max_kv_len: int,
                                  weights: bool = False) -> int:
    return int(lib.mea_decode_kv4_workspace_size(B, Hq, Hkv, K, max_kv_len, int(bool(weights))))


def mea_decode_kv4(q, cache: Kv4Cache, kv_seqlens, max_kv_len: int, scale: float | None = None,
                   alibi: bool = False, weights=None, weights_out=None,
                   return_weights: bool = False, out=None, lse=None, workspace=None,
                   return_lse: bool = True, stream=None):
    """One decode step against a 4-bit cache.  q [B,Hq,K] or [B,1,Hq,K]; kv_seqlens int32
    CUDA [B], the rows of each sequence (its new token included) -> (out shaped like q, lse
    [B,Hq] fp32 or None).

    With ``return_weights`` (or ``weights_out``) a third result: weights_out [B,Hkv,rows]
    fp32 = ``weights`` (zeros if None) + the softmax weight each row got in this step, summed
    over the query heads of its kv head; 0 for rows past kv_seqlens[b].  weights_out may be
    weights itself."""
    B, Hkv, cap, K, dtype, index = _kv4_dims(cache)
    shape = q.shape
    if len(shape) not in (3, 4) or (len(shape) == 4 and shape[1] != 1) or shape[0] != B \
            or shape[-1] != K:
        raise ValueError("q must be [B, Hq, K] or [B, 1, Hq, K]")
    Hq = shape[-2]
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if q.dtype != dtype:
        raise ValueError("q must have the dtype of the cache's params")
    scale = K ** -0.5 if scale is None else float(scale)
    max_kv_len = int(max_kv_len)
    _on(index, q, "q")
    _on_stream(index, stream)
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty(shape, dtype, q.device, stream)
    elif out.shape != shape or out.dtype != dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous and shaped and typed like q")
    if lse is not None:
        _f32(lse, (B, Hq), index, "lse")
    elif return_lse:
        lse = _empty((B, Hq), _F32, q.device, stream)
    want = return_weights or weights_out is not None
    if weights is not None and not want:
        raise ValueError("weights needs return_weights or weights_out")
    if want:
        if weights_out is None:
            weights_out = _empty((B, Hkv, cap), _F32, q.device, stream)
        _f32(weights, (B, Hkv, cap), index, "weights")
        _f32(weights_out, (B, Hkv, cap), index, "weights_out")
    _on(index, out, "out")
    _on(index, workspace, "workspace")
    _lens(B, index, kv_seqlens, "kv_seqlens")
    ws_bytes = 0
    if workspace is None:
        need = mea_decode_kv4_workspace_size(B, Hq, Hkv, K, max_kv_len, want)
        if need > 0:
            workspace = _empty(need, _U8, q.device, stream, returned=False)
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws_bytes = workspace.numel() * workspace.element_size()
    kc, kp, vc, vp = cache
    _launch("mea_decode_kv4", lib.mea_decode_kv4, index, stream,
            (q.data_ptr(), kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(),
             kv_seqlens.data_ptr(), out.data_ptr(), _addr(lse), _addr(weights),
             _addr(weights_out), B, Hq, Hkv, K, cap, max_kv_len, _DTYPE[dtype],
             1 if alibi else 0, scale, _addr(workspace), ws_bytes))
    return (out, lse, weights_out) if want else (out, lse)


def mea_key_weights(q, k, lse, cache_seqlens=None, q_seqlens=None, causal: bool = True,
                    scale: float | None = None, alibi: bool = False, weights=None, out=None,
                    stream=None):
    """The attention weight every key gathered from the queries q [B,M,Hq,K], summed over
    the rows and over the query heads of its kv head: out [B,Hkv,N] fp32 = ``weights`` (zeros
    if None) + sum exp(scale q.k + bias - lse).  k [B,N,Hkv,K] is the keys of mea_fwd or, with
    ``cache_seqlens`` (and ``q_seqlens``) as given to mea_prefill_chunk, the cache; lse
    [B,Hq,M] is what that attention returned.  Rows past the sequence get 0.  out may be
    weights itself."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, M, Hq, K] and k [B, N, Hkv, K]")
    B, M, Hq, K = q.shape
    _, N, Hkv, _ = k.shape
    if k.shape != (B, N, Hkv, K):
        raise ValueError("k must be [B, N, Hkv, K]")
    if q.dtype not in _DTYPE or k.dtype != q.dtype:
        raise ValueError("q and k must share dtype float16 or bfloat16")
    if q_seqlens is not None and cache_seqlens is None:
        raise ValueError("q_seqlens needs cache_seqlens")
    if lse is None:
        raise ValueError("lse must be what the attention of these queries returned")
    scale = K ** -0.5 if scale is None else float(scale)
    index = _cuda_index(q, "q")
    _on_stream(index, stream)
    if out is None:
        out = _empty((B, Hkv, N), _F32, q.device, stream)
    _f32(lse, (B, Hq, M), index, "lse")
    _f32(weights, (B, Hkv, N), index, "weights")
    _f32(out, (B, Hkv, N), index, "out")
    _on(index, k, "k")
    _lens(B, index, cache_seqlens, "cache_seqlens")
    _lens(B, index, q_seqlens, "q_seqlens")
    _launch("mea_key_weights", lib.mea_key_weights, index, stream,
            (q.data_ptr(), k.data_ptr(), lse.data_ptr(), _addr(cache_seqlens), _addr(q_seqlens),
             _addr(weights), out.data_ptr(), B, M, N, Hq, Hkv, K, _bmhk_strides(q, "q"),
             _bmhk_strides(k, "k"), _DTYPE[q.dtype], 1 if causal else 0, 1 if alibi else 0,
             scale))
    return out


def _byte_strides(st, size, r, h):
    """ctypes int64[3] of a tensor's (b, row, head) strides in bytes."""
    return _i64x3(st[0] * size, st[r] * size, st[h] * size)


def _planes_of(cache, what):
    """A cache as ([(tensor, (row axis, head axis))], B, Hkv, rows, device): a Kv4Cache, or a
    (k_cache, v_cache) pair of [B, rows, Hkv, K] tensors with contiguous K."""
    if isinstance(cache, Kv4Cache):
        B, Hkv, rows, _, _, index = _kv4_dims(cache, what)
        return [(t, (2, 1)) for t in cache], B, Hkv, rows, index
    k, v = cache
    for name, t in (("k", k), ("v", v)):
        if t.dim() != 4 or t.stride(3) != 1:
            raise ValueError(f"{what}: {name} must be [B, rows, Hkv, K] with contiguous K")
        if t.dtype not in _DTYPE:
            raise ValueError(f"{what}: {name} must be float16 or bfloat16")
    if k.shape[:3] != v.shape[:3]:
        raise ValueError(f"{what}: k and v must have the same rows and heads")
    index = _cuda_index(k, what)
    _on(index, v, f"{what}: v")
    return [(k, (1, 2)), (v, (1, 2))], k.shape[0], k.shape[2], k.shape[1], index


def mea_cache_evict(cache, weights, cache_seqlens, budget: int, recent: int, out=None,
                    weights_out=None, new_seqlens=None, kept=None, stream=None):
    """Cuts each sequence of a cache down to ``budget`` rows, per kv head: the newest
    ``recent`` and the heaviest others by ``weights`` [B,Hkv,rows] fp32 (equal weights: the
    lowest row), moved to the front in their old order together with their weights.

    cache: a Kv4Cache or a (k_cache, v_cache) pair of [B,rows,Hkv,K] tensors.  out: another
    cache of the same kind with at least ``budget`` rows, or None to work in place (then
    weights are cut in place too).  Returns (new_seqlens int32 [B], kept int32 [B,Hkv,budget]
    -- the old row of every kept row, -1 after the last --, weights_out [B,Hkv,out rows], 0
    past the kept rows)."""
    src, B, Hkv, rows, index = _planes_of(cache, "cache")
    if out is None:
        dst, out_rows = src, rows
        if weights_out is not None and weights_out.data_ptr() != weights.data_ptr():
            raise ValueError("in place, weights are cut in place too")
        weights_out = weights
    else:
        dst, Bo, Ho, out_rows, out_index = _planes_of(out, "out")
        if isinstance(cache, Kv4Cache) != isinstance(out, Kv4Cache) or (Bo, Ho) != (B, Hkv):
            raise ValueError("out must be a cache of the same kind, batch and heads")
        if out_index != index:
            raise ValueError(f"out must lie on cuda:{index}")
    budget, recent = int(budget), int(recent)
    dev = src[0][0].device
    _on_stream(index, stream)
    if weights_out is None:
        weights_out = _empty((B, Hkv, out_rows), _F32, dev, stream)
    if new_seqlens is None:
        new_seqlens = _empty((B,), _I32, dev, stream)
    if kept is None:
        kept = _empty((B, Hkv, max(budget, 0)), _I32, dev, stream)
    _f32(weights, (B, Hkv, rows), index, "weights")
    _f32(weights_out, (B, Hkv, out_rows), index, "weights_out")
    if kept.dtype is not _I32 or kept.shape != (B, Hkv, budget) or not kept.is_contiguous():
        raise ValueError("kept must be a contiguous int32 [B, Hkv, budget] tensor")
    _on(index, kept, "kept")
    _lens(B, index, cache_seqlens, "cache_seqlens")
    _lens(B, index, new_seqlens, "new_seqlens")
    planes = (_Plane * len(src))()
    for plane, (s, (r, h)), (d, _) in zip(planes, src, dst):
        if s.dtype is not d.dtype or s.shape[3:] != d.shape[3:]:
            raise ValueError("out must have the rows of the cache")
        size = s.element_size()
        plane.src, plane.dst = s.data_ptr(), d.data_ptr()
        plane.src_strides = _byte_strides(s.stride(), size, r, h)
        plane.dst_strides = plane.src_strides if d is s else _byte_strides(d.stride(), size, r, h)
        plane.row_bytes = s.shape[3:].numel() * size
    _launch("mea_cache_evict", lib.mea_cache_evict, index, stream,
            (planes, len(src), weights.data_ptr(), weights_out.data_ptr(),
             cache_seqlens.data_ptr(), new_seqlens.data_ptr(), kept.data_ptr(), B, Hkv, rows,
             out_rows, budget, recent))
    return new_seqlens, kept, weights_out


def read_device_status(clear: bool = True, stream=None) -> int:
    """Synchronise and return the first error a kernel recorded on this device (0 = none)."""
    return int(lib.mea_read_device_status(_stream(stream), int(bool(clear))))
