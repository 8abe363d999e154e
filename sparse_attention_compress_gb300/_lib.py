"""ctypes binding of libnsa.so: argument marshalling only.

Every function here has the name of the C entry point it calls (see include/nsa.h)
and does nothing but shape bookkeeping, output allocation through PyTorch and the
call itself; all arithmetic of the path runs in the CUDA kernels.  There is no
fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# NSA_LIBRARY may point at another build of the same library (e.g. with other tuning flags)
LIB_PATH = os.environ.get("NSA_LIBRARY") or os.path.join(_PKG, "libnsa.so")

NSA_F32, NSA_BF16 = 0, 1
_c_int, _c_i64, _c_p, _c_f, _c_sz = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t


class NsaShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int64), ("h", ctypes.c_int32),
                ("h_kv", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int)]


class NsaLayerSaved(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_cmp", "v_cmp", "o_cmp", "o_slc", "o_swa", "lse_cmp", "lse_slc",
                                                "lse_swa", "idx")]


class NsaPagedCache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("cache_lens", ctypes.c_void_p), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("page_stride", ctypes.c_int64)]


class NsaRope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p)]


class NsaPagedCacheQ8(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("cache_lens", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("page_stride", ctypes.c_int64)]


_SIGS = {
    "nsa_version": ([], ctypes.c_char_p),
    "nsa_last_error": ([], ctypes.c_char_p),
    "nsa_device_status": ([_c_p, _c_int], _c_int),
    "nsa_set_wait_limit_ns": ([ctypes.c_uint64], _c_int),
    "nsa_compress_k": ([_c_p, _c_p, _c_p, _c_int, _c_int, _c_p], _c_int),
    "nsa_cmp_scores_pool": ([_c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_f, _c_p, _c_p, _c_int, _c_p], _c_int),
    "nsa_topk_select": ([_c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p], _c_int),
    "nsa_cis_block_scores": ([_c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p], _c_int),
    "nsa_topk_two_stage": ([_c_p, _c_p, _c_int, _c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p], _c_int),
    "nsa_sparse_cis_fwd": ([_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p], _c_int),
    "nsa_select_workspace_size": ([_c_p, _c_int], _c_sz),
    "nsa_block_sparse_workspace_size": ([_c_p], _c_sz),
    "nsa_block_sparse_fwd": ([_c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p, _c_sz, _c_p],
                             _c_int),
    "nsa_select": ([_c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_f, _c_int, _c_int, _c_int, _c_p, _c_p, _c_sz,
                    _c_p], _c_int),
    "nsa_sparse_fwd": ([_c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p], _c_int),
    "nsa_sparse_bwd_workspace_size": ([_c_p, _c_int, _c_int], _c_sz),
    "nsa_cmp_attn_bwd_workspace_size": ([_c_p, _c_int, _c_int], _c_sz),
    "nsa_cmp_attn_bwd": ([_c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                          _c_sz, _c_p], _c_int),
    "nsa_compress_bwd": ([_c_p, _c_p, _c_int, _c_int, _c_p, _c_p], _c_int),
    "nsa_swa_bwd_workspace_size": ([_c_p, _c_int], _c_sz),
    "nsa_swa_bwd": ([_c_p, _c_p, _c_p, _c_p, _c_int, _c_f, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p],
                    _c_int),
    "nsa_gate_combine_bwd": ([_c_i64, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p],
                             _c_int),
    "nsa_sparse_bwd": ([_c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                        _c_sz, _c_p], _c_int),
    "nsa_cmp_attn_fwd_workspace_size": ([_c_p, _c_int, _c_int], _c_sz),
    "nsa_cmp_attn_fwd": ([_c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "nsa_swa_fwd_workspace_size": ([_c_p], _c_sz),
    "nsa_swa_fwd": ([_c_p, _c_p, _c_p, _c_p, _c_int, _c_f, _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "nsa_gate_combine": ([_c_i64, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p], _c_int),
    "nsa_sparse_decode_workspace_size": ([_c_int] * 9, _c_sz),
    "nsa_sparse_decode": ([_c_int, _c_p, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int,
                           _c_int, _c_int, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "nsa_sparse_decode_cis": ([_c_int, _c_p, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                               _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p,
                               _c_sz, _c_p], _c_int),
    "nsa_sparse_decode_noalloc_max_bytes": ([], _c_sz),
    "nsa_sparse_decode_noalloc": ([_c_int, _c_p, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_int,
                                   _c_int, _c_int, _c_int, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p], _c_int),
    "nsa_layer_fwd_workspace_size": ([_c_p, _c_int, _c_int, _c_int, _c_int], _c_sz),
    "nsa_layer_fwd_train": ([_c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                             _c_f, _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "nsa_layer_bwd_workspace_size": ([_c_p, _c_int, _c_int, _c_int, _c_int, _c_int], _c_sz),
    "nsa_layer_bwd": ([_c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p,
                       _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "nsa_layer_fwd": ([_c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_f,
                       _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "nsa_paged_append": ([_c_p, _c_p, _c_p, _c_p, _c_p], _c_int),
    "nsa_paged_append_rope": ([_c_p, _c_p, _c_p, _c_p, _c_p, _c_p], _c_int),
    "nsa_paged_q8_append": ([_c_p, _c_p, _c_p, _c_p, _c_p, _c_p], _c_int),
    "nsa_paged_q8_attn_fwd_workspace_size": ([_c_p, _c_p, _c_i64, _c_int, _c_int], _c_sz),
    "nsa_paged_q8_attn_fwd": ([_c_p, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "nsa_paged_attn_fwd_workspace_size": ([_c_p, _c_i64, _c_int, _c_int], _c_sz),
    "nsa_paged_attn_fwd": ([_c_p, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "nsa_paged_attn_weights": ([_c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_f, _c_f, _c_p, _c_p], _c_int),
    "nsa_paged_evict": ([_c_int, _c_int, _c_int, _c_p, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p, _c_p, _c_p],
                        _c_int),
    "nsa_swa_sink_fwd_workspace_size": ([_c_p, _c_int, _c_int], _c_sz),
    "nsa_swa_sink_fwd": ([_c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p, _c_sz, _c_p], _c_int),
    "nsa_swa_sink_bwd_workspace_size": ([_c_p, _c_int, _c_int], _c_sz),
    "nsa_swa_sink_bwd": ([_c_p, _c_p, _c_p, _c_p, _c_int, _c_int, _c_f, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                          _c_sz, _c_p], _c_int),
}

_lib = None


def load() -> ctypes.CDLL:
    """Load libnsa.so (built by __graft_entry__.build() / build.py); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build the CUDA library first "
                              "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


class NsaError(RuntimeError):
    pass


def _check(rc: int, fn: str) -> None:
    if rc != 0:
        msg = load().nsa_last_error().decode()
        raise NsaError(f"{fn} failed (status {rc}): {msg}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return NSA_BF16
    if t.dtype == torch.float32:
        return NSA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def make_shape(tokens: int, h: int, h_kv: int, d: int, dtype: int, *, cu_seqlens=None, max_seqlen=None,
               batch=None, seqlen=None) -> NsaShape:
    """Dense layout (batch, seqlen) or packed varlen (cu_seqlens device int32, max_seqlen)."""
    s = NsaShape()
    s.h, s.h_kv, s.d, s.dtype = h, h_kv, d, dtype
    if cu_seqlens is not None:
        if max_seqlen is None:
            raise ValueError("varlen needs max_seqlen")
        s.cu_seqlens = cu_seqlens.data_ptr()
        s.n_seqs = cu_seqlens.numel() - 1
        s.total_tokens = tokens
        s.seqlen = int(max_seqlen)
    else:
        if batch is None:
            batch, seqlen = 1, tokens
        s.batch, s.seqlen = int(batch), int(seqlen)
        if batch * seqlen != tokens:
            raise ValueError("batch * seqlen must equal the token count")
        s.cu_seqlens = None
        s.total_tokens = tokens
    return s


def _flat(t: torch.Tensor):
    """[B, T, H, d] -> ([B*T, H, d], B, T); [N, H, d] -> (t, None, None)."""
    if t.dim() == 4:
        B, T = t.shape[0], t.shape[1]
        return t.reshape(B * T, t.shape[2], t.shape[3]), B, T
    if t.dim() == 3:
        return t, None, None
    raise ValueError("expected [B, T, H, d] or [tokens, H, d]")


def _shape_for(q, h_kv, cu_seqlens, max_seqlen):
    qf, B, T = _flat(q)
    if cu_seqlens is None and B is None:
        B, T = 1, qf.shape[0]
    return qf, make_shape(qf.shape[0], qf.shape[1], h_kv, qf.shape[2], _dtype(qf), cu_seqlens=cu_seqlens,
                          max_seqlen=max_seqlen, batch=B, seqlen=T)


def num_cmp(L: int, kernel: int = 32, stride: int = 16) -> int:
    return (L - kernel) // stride + 1 if L >= kernel else 0


# ----------------------------------------------------------------------------- entry points
def nsa_compress_k(k, kernel=32, stride=16, *, cu_seqlens=None, max_seqlen=None, n_cmp=None, out=None,
                   stream=None):
    """S1.  k [B,T,Hkv,d] or packed [tokens,Hkv,d] -> packed compressed rows [n_cmp, Hkv, d]."""
    kf, shp = _shape_for(k, k.shape[-2], cu_seqlens, max_seqlen)
    if out is None:
        if n_cmp is None:
            if cu_seqlens is not None:
                lens = (cu_seqlens[1:] - cu_seqlens[:-1]).tolist()
                n_cmp = sum(num_cmp(int(L), kernel, stride) for L in lens)
            else:
                n_cmp = shp.batch * num_cmp(shp.seqlen, kernel, stride)
        out = torch.empty((n_cmp, kf.shape[1], kf.shape[2]), dtype=kf.dtype, device=kf.device)
    _check(load().nsa_compress_k(ctypes.byref(shp), _ptr(kf), _ptr(out), kernel, stride, _stream(stream)),
           "nsa_compress_k")
    return out


def nsa_cmp_scores_pool(q, k_cmp, h_kv, kernel=32, stride=16, block_size=64, scale=0.0, *, lse_in=None,
                        cu_seqlens=None, max_seqlen=None, nb_stride=None, out=None, stream=None):
    """S2+S3.  Returns block scores [tokens, Hkv, nb_stride] fp32."""
    qf, shp = _shape_for(q, h_kv, cu_seqlens, max_seqlen)
    if nb_stride is None:
        nb_stride = -(-shp.seqlen // block_size)
    if out is None:
        out = torch.empty((qf.shape[0], h_kv, nb_stride), dtype=torch.float32, device=qf.device)
    _check(load().nsa_cmp_scores_pool(ctypes.byref(shp), _ptr(qf), _ptr(k_cmp), kernel, stride, block_size,
                                      float(scale), _ptr(lse_in), _ptr(out), nb_stride, _stream(stream)),
           "nsa_cmp_scores_pool")
    return out


def nsa_block_sparse_workspace_size(shape: NsaShape) -> int:
    return int(load().nsa_block_sparse_workspace_size(ctypes.byref(shape)))


def nsa_select_workspace_size(shape: NsaShape, block_size=64) -> int:
    return int(load().nsa_select_workspace_size(ctypes.byref(shape), block_size))


def nsa_block_sparse_fwd(q, k, v, block_mask, causal=True, block_size=64, scale=0.0, *, workspace=None, out=None,
                         lse=None, stream=None):
    """Block-mask sparse attention; q/k/v [B, T, H, d] bf16, block_mask uint8 [B, H, T/64, T/64]."""
    qf, shp = _shape_for(q, k.shape[-2], None, None)
    if workspace is None:
        ws = int(load().nsa_block_sparse_workspace_size(ctypes.byref(shp)))
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=qf.device)
    if out is None:
        out = torch.empty_like(qf)
    _check(load().nsa_block_sparse_fwd(ctypes.byref(shp), _ptr(qf), _ptr(k), _ptr(v), _ptr(block_mask), block_size,
                                       int(bool(causal)), float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                       workspace.numel(), _stream(stream)), "nsa_block_sparse_fwd")
    return out


def nsa_select(q, k_cmp, h_kv, k=16, kernel=32, stride=16, block_size=64, n_init=1, n_local=2, scale=0.0, *,
               cu_seqlens=None, max_seqlen=None, workspace=None, out=None, stream=None):
    """S2-S4 in one call: block indices [tokens, Hkv, k] int32 from q and the compressed keys."""
    qf, shp = _shape_for(q, h_kv, cu_seqlens, max_seqlen)
    if workspace is None:
        ws = int(load().nsa_select_workspace_size(ctypes.byref(shp), block_size))
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=qf.device)
    if out is None:
        out = torch.empty((qf.shape[0], h_kv, k), dtype=torch.int32, device=qf.device)
    _check(load().nsa_select(ctypes.byref(shp), _ptr(qf), _ptr(k_cmp), kernel, stride, block_size, float(scale),
                             n_init, n_local, k, _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "nsa_select")
    return out


def nsa_topk_select(block_scores, k, block_size=64, n_init=1, n_local=2, *, cu_seqlens=None, max_seqlen=None,
                    batch=None, seqlen=None, out=None, stream=None):
    """S4.  block_scores [tokens, Hkv, nb_stride] fp32 -> indices [tokens, Hkv, k] int32."""
    tokens, h_kv, nb_stride = block_scores.shape
    if cu_seqlens is None and batch is None:
        batch, seqlen = 1, tokens
    shp = make_shape(tokens, h_kv, h_kv, 1, NSA_F32, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen, batch=batch,
                     seqlen=seqlen)
    if out is None:
        out = torch.empty((tokens, h_kv, k), dtype=torch.int32, device=block_scores.device)
    _check(load().nsa_topk_select(ctypes.byref(shp), _ptr(block_scores), nb_stride, block_size, n_init, n_local, k,
                                  _ptr(out), _stream(stream)), "nsa_topk_select")
    return out


def nsa_cis_block_scores(cis, kernel=32, stride=16, block_size=64, *, cu_seqlens=None, max_seqlen=None, batch=None,
                         seqlen=None, nb_stride=None, out=None, stream=None):
    """NOSA stage 2.  cis [tokens, Hkv] fp32 -> block CIS scores [n_seqs, Hkv, nb_stride] fp32."""
    tokens, h_kv = cis.shape
    if cu_seqlens is None and batch is None:
        batch, seqlen = 1, tokens
    shp = make_shape(tokens, h_kv, h_kv, 1, NSA_F32, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen, batch=batch,
                     seqlen=seqlen)
    n_seqs = shp.n_seqs if cu_seqlens is not None else shp.batch
    if nb_stride is None:
        nb_stride = max(1, -(-shp.seqlen // block_size))
    if out is None:
        out = torch.empty((n_seqs, h_kv, nb_stride), dtype=torch.float32, device=cis.device)
    _check(load().nsa_cis_block_scores(ctypes.byref(shp), _ptr(cis), kernel, stride, block_size, nb_stride,
                                       _ptr(out), _stream(stream)), "nsa_cis_block_scores")
    return out


def nsa_topk_two_stage(block_scores, cis_block_scores, qk_select, k, block_size=64, n_init=1, n_local=2, *,
                       cu_seqlens=None, max_seqlen=None, batch=None, seqlen=None, out=None, stream=None):
    """NOSA two-stage selection: block_scores [tokens, Hkv, nb_stride], cis_block_scores
    [n_seqs, Hkv, nb_stride] -> indices [tokens, Hkv, k] int32."""
    tokens, h_kv, nb_stride = block_scores.shape
    if cu_seqlens is None and batch is None:
        batch, seqlen = 1, tokens
    shp = make_shape(tokens, h_kv, h_kv, 1, NSA_F32, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen, batch=batch,
                     seqlen=seqlen)
    if out is None:
        out = torch.empty((tokens, h_kv, k), dtype=torch.int32, device=block_scores.device)
    _check(load().nsa_topk_two_stage(ctypes.byref(shp), _ptr(block_scores), nb_stride, _ptr(cis_block_scores),
                                     block_size, n_init, n_local, qk_select, k, _ptr(out), _stream(stream)),
           "nsa_topk_two_stage")
    return out


def nsa_sparse_cis_fwd(q, k, v, cis, block_indices, block_size=64, scale=0.0, *, cu_seqlens=None, max_seqlen=None,
                       out=None, lse=None, stream=None):
    """NOSA sparse_forward: selected attention with weights p * cis (normalised); cis [tokens, Hkv] fp32."""
    qf, shp = _shape_for(q, k.shape[-2], cu_seqlens, max_seqlen)
    S = block_indices.shape[-1]
    if out is None:
        out = torch.empty_like(qf)
    _check(load().nsa_sparse_cis_fwd(ctypes.byref(shp), _ptr(qf), _ptr(k), _ptr(v), _ptr(cis), _ptr(block_indices),
                                     S, block_size, float(scale), _ptr(out), _ptr(lse), _stream(stream)),
           "nsa_sparse_cis_fwd")
    return out.view(q.shape) if q.dim() == 4 else out


def nsa_sparse_fwd(q, k, v, block_indices, block_size=64, scale=0.0, *, cu_seqlens=None, max_seqlen=None,
                   out=None, lse=None, stream=None):
    """S5.  q [B,T,H,d] / [tokens,H,d]; k, v with Hkv heads; block_indices [..., Hkv, S] int32."""
    qf, shp = _shape_for(q, k.shape[-2], cu_seqlens, max_seqlen)
    S = block_indices.shape[-1]
    if out is None:
        out = torch.empty_like(qf)
    _check(load().nsa_sparse_fwd(ctypes.byref(shp), _ptr(qf), _ptr(k), _ptr(v), _ptr(block_indices), S, block_size,
                                 float(scale), _ptr(out), _ptr(lse), _stream(stream)), "nsa_sparse_fwd")
    return out.view(q.shape) if q.dim() == 4 else out


def nsa_sparse_bwd_workspace_size(shape: NsaShape, S: int, block_size: int = 64) -> int:
    return int(load().nsa_sparse_bwd_workspace_size(ctypes.byref(shape), S, block_size))


def nsa_sparse_bwd(q, k, v, block_indices, o, lse, d_o, block_size=64, scale=0.0, *, cu_seqlens=None,
                   max_seqlen=None, workspace=None, dq=None, dk=None, dv=None, stream=None):
    """Backward of S5: returns (dq, dk, dv) shaped like q, k, v.  o and lse come from
    nsa_sparse_fwd on the same inputs; d_o is the upstream gradient (like q)."""
    qf, shp = _shape_for(q, k.shape[-2], cu_seqlens, max_seqlen)
    S = block_indices.shape[-1]
    if workspace is None:
        ws = nsa_sparse_bwd_workspace_size(shp, S, block_size)
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(load().nsa_sparse_bwd(ctypes.byref(shp), _ptr(qf), _ptr(k), _ptr(v), _ptr(block_indices), S, block_size,
                                 float(scale), _ptr(o), _ptr(lse), _ptr(d_o), _ptr(dq), _ptr(dk), _ptr(dv),
                                 _ptr(workspace), workspace.numel(), _stream(stream)), "nsa_sparse_bwd")
    return dq, dk, dv


def nsa_cmp_attn_bwd_workspace_size(shape: NsaShape, kernel: int = 32, stride: int = 16) -> int:
    return int(load().nsa_cmp_attn_bwd_workspace_size(ctypes.byref(shape), kernel, stride))


def nsa_cmp_attn_bwd(q, k_cmp, v_cmp, o, lse, d_o, h_kv, kernel=32, stride=16, scale=0.0, *, cu_seqlens=None,
                     max_seqlen=None, workspace=None, dq=None, dk_cmp=None, dv_cmp=None, stream=None):
    """Backward of S7: (dq like q, dk_cmp and dv_cmp like k_cmp) from the forward's o, lse."""
    qf, shp = _shape_for(q, h_kv, cu_seqlens, max_seqlen)
    if workspace is None:
        ws = nsa_cmp_attn_bwd_workspace_size(shp, kernel, stride)
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk_cmp = torch.empty_like(k_cmp) if dk_cmp is None else dk_cmp
    dv_cmp = torch.empty_like(v_cmp) if dv_cmp is None else dv_cmp
    _check(load().nsa_cmp_attn_bwd(ctypes.byref(shp), _ptr(qf), _ptr(k_cmp), _ptr(v_cmp), kernel, stride,
                                   float(scale), _ptr(o), _ptr(lse), _ptr(d_o), _ptr(dq), _ptr(dk_cmp), _ptr(dv_cmp),
                                   _ptr(workspace), workspace.numel(), _stream(stream)), "nsa_cmp_attn_bwd")
    return dq, dk_cmp, dv_cmp


def nsa_compress_bwd(dk_cmp, tokens, kernel=32, stride=16, *, cu_seqlens=None, max_seqlen=None, batch=None,
                     seqlen=None, out=None, stream=None):
    """Backward of S1: token-row gradient [tokens, Hkv, d] from the window gradient dk_cmp."""
    _, h_kv, d = dk_cmp.shape
    if cu_seqlens is None and batch is None:
        batch, seqlen = 1, tokens
    shp = make_shape(tokens, h_kv, h_kv, d, NSA_BF16, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen, batch=batch,
                     seqlen=seqlen)
    if out is None:
        out = torch.empty((tokens, h_kv, d), dtype=dk_cmp.dtype, device=dk_cmp.device)
    _check(load().nsa_compress_bwd(ctypes.byref(shp), _ptr(dk_cmp), kernel, stride, _ptr(out), _stream(stream)),
           "nsa_compress_bwd")
    return out


def nsa_swa_bwd_workspace_size(shape: NsaShape, window: int = 512) -> int:
    return int(load().nsa_swa_bwd_workspace_size(ctypes.byref(shape), window))


def nsa_swa_bwd(q, k, v, o, lse, d_o, window=512, scale=0.0, *, cu_seqlens=None, max_seqlen=None, workspace=None,
                dq=None, dk=None, dv=None, stream=None):
    """Backward of S8: (dq, dk, dv) shaped like q, k, v from the forward's o and lse."""
    qf, shp = _shape_for(q, k.shape[-2], cu_seqlens, max_seqlen)
    if workspace is None:
        ws = nsa_swa_bwd_workspace_size(shp, window)
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(load().nsa_swa_bwd(ctypes.byref(shp), _ptr(qf), _ptr(k), _ptr(v), window, float(scale), _ptr(o),
                              _ptr(lse), _ptr(d_o), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                              workspace.numel(), _stream(stream)), "nsa_swa_bwd")
    return dq, dk, dv


def nsa_gate_combine_bwd(d_o, o_cmp, o_slc, o_swa, gate_logits, *, stream=None):
    """Backward of S9: (d o_cmp, d o_slc, d o_swa, d gate_logits)."""
    tokens, h, d = d_o.shape
    outs = [torch.empty_like(d_o) for _ in range(3)]
    dg = torch.empty_like(gate_logits)
    _check(load().nsa_gate_combine_bwd(tokens, h, d, _ptr(d_o), _ptr(o_cmp), _ptr(o_slc), _ptr(o_swa),
                                       _ptr(gate_logits), _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(dg),
                                       _stream(stream)), "nsa_gate_combine_bwd")
    return outs[0], outs[1], outs[2], dg


def _workspace(nbytes, device, workspace=None):
    """Caller's workspace, or a fresh one of nbytes (None when nothing is needed)."""
    if workspace is not None or nbytes == 0:
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def nsa_cmp_attn_fwd(q, k_cmp, v_cmp, h_kv, kernel=32, stride=16, scale=0.0, *, cu_seqlens=None,
                     max_seqlen=None, out=None, lse=None, workspace=None, stream=None):
    """S7.  Compressed branch over packed compressed keys / values."""
    qf, shp = _shape_for(q, h_kv, cu_seqlens, max_seqlen)
    if out is None:
        out = torch.empty_like(qf)
    ws = _workspace(int(load().nsa_cmp_attn_fwd_workspace_size(ctypes.byref(shp), kernel, stride)), qf.device,
                    workspace)
    _check(load().nsa_cmp_attn_fwd(ctypes.byref(shp), _ptr(qf), _ptr(k_cmp), _ptr(v_cmp), kernel, stride,
                                   float(scale), _ptr(out), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(),
                                   _stream(stream)), "nsa_cmp_attn_fwd")
    return out


def nsa_swa_fwd(q, k, v, window=512, scale=0.0, *, cu_seqlens=None, max_seqlen=None, out=None, lse=None,
                workspace=None, stream=None):
    """S8.  Sliding-window branch."""
    qf, shp = _shape_for(q, k.shape[-2], cu_seqlens, max_seqlen)
    if out is None:
        out = torch.empty_like(qf)
    ws = _workspace(int(load().nsa_swa_fwd_workspace_size(ctypes.byref(shp))), qf.device, workspace)
    _check(load().nsa_swa_fwd(ctypes.byref(shp), _ptr(qf), _ptr(k), _ptr(v), window, float(scale), _ptr(out),
                              _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)), "nsa_swa_fwd")
    return out


def nsa_gate_combine(o_cmp, o_slc, o_swa, gate_logits, *, out=None, stream=None):
    """S9.  out = sigmoid(g0) o_cmp + sigmoid(g1) o_slc + sigmoid(g2) o_swa."""
    tokens, h, d = o_cmp.shape
    if out is None:
        out = torch.empty_like(o_cmp)
    _check(load().nsa_gate_combine(tokens, h, d, _ptr(o_cmp), _ptr(o_slc), _ptr(o_swa), _ptr(gate_logits),
                                   _ptr(out), _stream(stream)), "nsa_gate_combine")
    return out


def nsa_sparse_decode_workspace_size(batch, max_len, h, h_kv, d, kernel=32, stride=16, block_size=64, k=64):
    return int(load().nsa_sparse_decode_workspace_size(batch, max_len, h, h_kv, d, kernel, stride, block_size, k))


def nsa_sparse_decode(q, k_cache, v_cache, k_cmp_cache, seqlens, k=64, kernel=32, stride=16, block_size=64,
                      n_init=1, n_local=2, scale=0.0, *, workspace=None, idx_out=None, out=None, stream=None):
    """S6.  q [B,H,d]; caches [B,L,Hkv,d]; k_cmp_cache [B,n_c(L),Hkv,d]; seqlens device int32 [B]."""
    B, h, d = q.shape
    max_len, h_kv = k_cache.shape[1], k_cache.shape[2]
    if workspace is None:
        ws = nsa_sparse_decode_workspace_size(B, max_len, h, h_kv, d, kernel, stride, block_size, k)
        workspace = torch.empty(ws, dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    _check(load().nsa_sparse_decode(B, _ptr(seqlens), max_len, h, h_kv, d, _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(k_cmp_cache), kernel, stride, block_size, n_init, n_local, k, float(scale),
                                    _ptr(idx_out), _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "nsa_sparse_decode")
    return out


def nsa_sparse_decode_cis(q, k_cache, v_cache, k_cmp_cache, cis_cache, seqlens, cis_block_scores=None, qk_select=0,
                          k=64, kernel=32, stride=16, block_size=64, n_init=1, n_local=2, scale=0.0, *,
                          workspace=None, idx_out=None, out=None, stream=None):
    """NOSA decode step: CIS-weighted attention, two-stage selection when cis_block_scores
    [B, Hkv, nb_stride] is given.  cis_cache [B, max_len, Hkv] fp32."""
    B, h, d = q.shape
    max_len, h_kv = k_cache.shape[1], k_cache.shape[2]
    if workspace is None:
        ws = nsa_sparse_decode_workspace_size(B, max_len, h, h_kv, d, kernel, stride, block_size, k)
        workspace = torch.empty(ws, dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    nb_stride = 0 if cis_block_scores is None else cis_block_scores.shape[-1]
    _check(load().nsa_sparse_decode_cis(B, _ptr(seqlens), max_len, h, h_kv, d, _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(k_cmp_cache), _ptr(cis_cache), _ptr(cis_block_scores), nb_stride,
                                        qk_select, kernel, stride, block_size, n_init, n_local, k, float(scale),
                                        _ptr(idx_out), _ptr(out), _ptr(workspace), workspace.numel(),
                                        _stream(stream)), "nsa_sparse_decode_cis")
    return out


def nsa_sparse_decode_noalloc(q, k_cache, v_cache, k_cmp_cache, seqlens, k=64, kernel=32, stride=16,
                              block_size=64, n_init=1, n_local=2, scale=0.0, *, idx_out=None, out=None, stream=None):
    """S6 without a workspace: the scratch is the library's fixed device array (see nsa.h)."""
    B, h, d = q.shape
    max_len, h_kv = k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty_like(q)
    _check(load().nsa_sparse_decode_noalloc(B, _ptr(seqlens), max_len, h, h_kv, d, _ptr(q), _ptr(k_cache),
                                            _ptr(v_cache), _ptr(k_cmp_cache), kernel, stride, block_size, n_init,
                                            n_local, k, float(scale), _ptr(idx_out), _ptr(out), _stream(stream)),
           "nsa_sparse_decode_noalloc")
    return out


def nsa_device_status(reset: bool = False) -> int:
    """Device status word (0 or NSA_ERR_TIMEOUT = 4); synchronises the device."""
    st = ctypes.c_int32(0)
    _check(load().nsa_device_status(ctypes.byref(st), int(bool(reset))), "nsa_device_status")
    return int(st.value)


def nsa_set_wait_limit_ns(ns: int = 0) -> None:
    """Limit of the kernels' first-level bounded waits in ns (0: the default second)."""
    _check(load().nsa_set_wait_limit_ns(int(ns)), "nsa_set_wait_limit_ns")


def nsa_layer_fwd_workspace_size(shape: NsaShape, kernel=32, stride=16, block_size=64, S=16) -> int:
    return int(load().nsa_layer_fwd_workspace_size(ctypes.byref(shape), kernel, stride, block_size, S))


def nsa_layer_fwd(q, k, v, gate_logits, kernel=32, stride=16, block_size=64, S=16, n_init=1, n_local=2,
                  window=512, scale=0.0, *, cu_seqlens=None, max_seqlen=None, workspace=None, idx_out=None,
                  out=None, stream=None):
    """Full three-branch layer forward."""
    qf, shp = _shape_for(q, k.shape[-2], cu_seqlens, max_seqlen)
    if workspace is None:
        ws = nsa_layer_fwd_workspace_size(shp, kernel, stride, block_size, S)
        workspace = torch.empty(ws, dtype=torch.uint8, device=qf.device)
    if out is None:
        out = torch.empty_like(qf)
    _check(load().nsa_layer_fwd(ctypes.byref(shp), _ptr(qf), _ptr(k), _ptr(v), _ptr(gate_logits), kernel, stride,
                                block_size, S, n_init, n_local, window, float(scale), _ptr(out), _ptr(idx_out),
                                _ptr(workspace), workspace.numel(), _stream(stream)), "nsa_layer_fwd")
    return out


def nsa_layer_saved_buffers(tokens, n_cmp, h, h_kv, d, S, device):
    """Allocate the tensors a training forward keeps for the backward (a dict of tensors)."""
    bf = torch.bfloat16
    return {"k_cmp": torch.empty((n_cmp, h_kv, d), dtype=bf, device=device),
            "v_cmp": torch.empty((n_cmp, h_kv, d), dtype=bf, device=device),
            "o_cmp": torch.empty((tokens, h, d), dtype=bf, device=device),
            "o_slc": torch.empty((tokens, h, d), dtype=bf, device=device),
            "o_swa": torch.empty((tokens, h, d), dtype=bf, device=device),
            "lse_cmp": torch.empty((tokens, h), dtype=torch.float32, device=device),
            "lse_slc": torch.empty((tokens, h), dtype=torch.float32, device=device),
            "lse_swa": torch.empty((tokens, h), dtype=torch.float32, device=device),
            "idx": torch.empty((tokens, h_kv, S), dtype=torch.int32, device=device)}


def _saved_struct(saved):
    st = NsaLayerSaved()
    for name, _ in NsaLayerSaved._fields_:
        setattr(st, name, saved[name].data_ptr())
    return st


def nsa_layer_fwd_train(q, k, v, gate_logits, saved, kernel=32, stride=16, block_size=64, S=16, n_init=1,
                        n_local=2, window=512, scale=0.0, *, cu_seqlens=None, max_seqlen=None, workspace=None,
                        out=None, stream=None):
    """Layer forward that also fills `saved` (nsa_layer_saved_buffers) for nsa_layer_bwd."""
    qf, shp = _shape_for(q, k.shape[-2], cu_seqlens, max_seqlen)
    if workspace is None:
        ws = int(load().nsa_layer_fwd_workspace_size(ctypes.byref(shp), kernel, stride, block_size, S))
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=q.device)
    out = torch.empty_like(qf) if out is None else out
    st = _saved_struct(saved)
    _check(load().nsa_layer_fwd_train(ctypes.byref(shp), _ptr(qf), _ptr(k), _ptr(v), _ptr(gate_logits), kernel,
                                      stride, block_size, S, n_init, n_local, window, float(scale), _ptr(out),
                                      ctypes.byref(st), _ptr(workspace), workspace.numel(), _stream(stream)),
           "nsa_layer_fwd_train")
    return out


def nsa_layer_bwd(q, k, v, gate_logits, saved, d_o, kernel=32, stride=16, block_size=64, S=16, window=512,
                  scale=0.0, *, cu_seqlens=None, max_seqlen=None, workspace=None, stream=None):
    """Layer backward: returns (dq, dk, dv, d_gate_logits)."""
    qf, shp = _shape_for(q, k.shape[-2], cu_seqlens, max_seqlen)
    if workspace is None:
        ws = int(load().nsa_layer_bwd_workspace_size(ctypes.byref(shp), kernel, stride, block_size, S, window))
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty_like(gate_logits)
    st = _saved_struct(saved)
    _check(load().nsa_layer_bwd(ctypes.byref(shp), _ptr(qf), _ptr(k), _ptr(v), _ptr(gate_logits), kernel, stride,
                                block_size, S, window, float(scale), ctypes.byref(st), _ptr(d_o), _ptr(dq), _ptr(dk),
                                _ptr(dv), _ptr(dg), _ptr(workspace), workspace.numel(), _stream(stream)),
           "nsa_layer_bwd")
    return dq, dk, dv, dg


# ----------------------------------------------------------------------------- paged cache
# These calls check what the C entry points cannot see: that every tensor lies on one GPU,
# dense and of its type.  Tensors they allocate belong to the stream the call runs on.  A
# decode step is a few microseconds of GPU time, so the checks come in two forms: a quick
# test, and the search for what is wrong when it fails.
_BF16, _F32, _I32, _U8, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn
_HERE = contextlib.nullcontext()


def _fits(t, dtype, shape, index) -> bool:
    """A dense tensor of this type and shape on GPU `index` (or none given)."""
    return t is None or (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                         and t.get_device() == index and t.is_contiguous())


def _expect(fn, device, **tensors):
    """Raise for the first of the named (tensor, dtype, shape) that does not fit.  Entries of a
    shape that are None may be anything."""
    for name, (t, dtype, shape) in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{fn}: {name} must be a tensor")
        if t.dtype != dtype:
            raise TypeError(f"{fn}: {name} must be {dtype}, not {t.dtype}")
        if t.device != device:
            raise ValueError(f"{fn}: {name} is on {t.device}, not on {device}")
        if len(t.shape) != len(shape) or any(b is not None and a != b for a, b in zip(t.shape, shape)):
            raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be dense (contiguous)")


def _int32(fn, **values):
    """ctypes would pass the low 32 bits of a larger number without a word.  (Called where a number
    has a bit past the 31st: small negative ones are the C entry points' to refuse.)"""
    for name, x in values.items():
        if not -0x80000000 <= x <= 0x7fffffff:
            raise ValueError(f"{fn}: {name} = {x} does not fit 32 bits")


def _on(device, stream):
    """(context that makes the call's device and stream current, raw stream, the caller's stream
    where it is another one)."""
    if device.type != "cuda":
        raise ValueError(f"expected tensors on a GPU, got {device}")
    if stream is None:
        here = torch.cuda.current_device() == device.index
        return _HERE if here else torch.cuda.device(device), torch._C._cuda_getCurrentRawStream(device.index), None
    if stream.device != device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")
    now = torch.cuda.current_stream(device)
    return torch.cuda.stream(stream), stream.cuda_stream, (None if now == stream else now)


def _new(shape, dtype, device, share):
    """A tensor of the call's stream; `share`: the caller's stream, which may use it too."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if share is not None:
        t.record_stream(share)
    return t


def _addr(t):
    return None if t is None else t.data_ptr()


def _page_stride(fn, name, t, dtype=_BF16):
    """Pages may lie apart (a pool that interleaves K and V); a page itself is dense."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{fn}: {name} must be [n_pages, page_size, h_kv, d]")
    if t.dtype is not dtype:
        raise TypeError(f"{fn}: {name} must be {dtype}, not {t.dtype}")
    n, p, h, d = t.shape
    s = t.stride()
    if s[3] != 1 or (h > 1 and s[2] != d) or (p > 1 and s[1] != h * d):
        raise ValueError(f"{fn}: the rows of a page of {name} must be dense")
    return s[0] if n > 1 else p * h * d


def _paged_cache(fn, k_pages, v_pages, block_table, cache_lens, n_seqs, weights=None):
    """(struct, page_size, h_kv, d) of a paged cache."""
    stride = _page_stride(fn, "k_pages", k_pages)
    shape = k_pages.shape
    n_pages, page, h_kv, d = shape
    if v_pages is not None and v_pages is not k_pages:
        if _page_stride(fn, "v_pages", v_pages) != stride or v_pages.shape != shape:
            raise ValueError(f"{fn}: v_pages must have the shape and strides of k_pages")
        if v_pages.device != k_pages.device:
            raise ValueError(f"{fn}: v_pages is on {v_pages.device}, k_pages on {k_pages.device}")
    index = k_pages.get_device()
    width = block_table.shape[1] if isinstance(block_table, torch.Tensor) and block_table.dim() == 2 else 0
    if (block_table is None or cache_lens is None or not _fits(block_table, _I32, (n_seqs, width), index)
            or not _fits(cache_lens, _I32, (n_seqs,), index)
            or not _fits(weights, _F32, (n_pages, h_kv, page), index)):
        if block_table is None or cache_lens is None:
            raise TypeError(f"{fn}: block_table and cache_lens must be tensors")
        _expect(fn, k_pages.device, block_table=(block_table, _I32, (n_seqs, None)),
                cache_lens=(cache_lens, _I32, (n_seqs,)), weights=(weights, _F32, (n_pages, h_kv, page)))
    return (NsaPagedCache(k_pages.data_ptr(), _addr(v_pages), _addr(weights), block_table.data_ptr(),
                          cache_lens.data_ptr(), n_pages, page, width, stride), page, h_kv, d)


def _span_shape(fn, q, h_kv, d, device, cu_seqlens, max_seqlen):
    """(tokens, shape struct, number of sequences) of new tokens [B, T, H, d] or packed
    [tokens, H, d]."""
    dims = q.shape if isinstance(q, torch.Tensor) else ()
    if len(dims) not in (3, 4) or dims[-1] != d or h_kv < 1 or dims[-2] % h_kv:
        raise ValueError(f"{fn}: expected [..., heads, {d}] with heads a multiple of {h_kv}, got {tuple(dims)}")
    index = device.index if device.type == "cuda" else -1
    if not _fits(q, _BF16, dims, index):
        _expect(fn, device, tokens=(q, _BF16, dims))
    if cu_seqlens is None:
        B, T = (dims[0], dims[1]) if len(dims) == 4 else (1, dims[0])
        return B * T, NsaShape(B, T, None, 0, B * T, dims[-2], h_kv, d, NSA_BF16), B
    if len(dims) == 4:
        raise ValueError(f"{fn}: with cu_seqlens the tokens are packed [tokens, heads, d]")
    n = cu_seqlens.numel() - 1 if isinstance(cu_seqlens, torch.Tensor) else 0
    if n < 1 or not _fits(cu_seqlens, _I32, (n + 1,), index):
        _expect(fn, device, cu_seqlens=(cu_seqlens, _I32, (None,)))
        raise ValueError(f"{fn}: cu_seqlens needs at least two entries")
    if max_seqlen is None:
        raise ValueError(f"{fn}: cu_seqlens needs max_seqlen")
    longest = int(max_seqlen)
    if longest >> 31:
        _int32(fn, max_seqlen=longest)
    return dims[0], NsaShape(0, longest, cu_seqlens.data_ptr(), n, dims[0], dims[1], h_kv, d, NSA_BF16), n


def nsa_paged_append(k_new, v_new, k_pages, v_pages, block_table, cache_lens, *, weights=None, cu_seqlens=None,
                     max_seqlen=None, stream=None):
    """New tokens' keys and values [B, T, Hkv, d] or packed [tokens, Hkv, d] into the cache, at the
    last positions of cache_lens; the weights of the written positions become 0."""
    fn = "nsa_paged_append"
    dev = k_pages.device
    ctx, raw, _ = _on(dev, stream)
    _, shp, n = _span_shape(fn, k_new, k_pages.shape[-2], k_pages.shape[-1], dev, cu_seqlens, max_seqlen)
    c = _paged_cache(fn, k_pages, v_pages, block_table, cache_lens, n, weights)[0]
    if v_new is None or k_new.shape[-2] != k_pages.shape[-2] or not _fits(v_new, _BF16, k_new.shape, dev.index):
        want = (*k_new.shape[:-2], *k_pages.shape[-2:])
        _expect(fn, dev, k_new=(k_new, _BF16, want), v_new=(v_new, _BF16, want))
        raise TypeError(f"{fn}: v_new must be a tensor")
    with ctx:
        rc = load().nsa_paged_append(ctypes.byref(shp), k_new.data_ptr(), v_new.data_ptr(), ctypes.byref(c), raw)
    if rc:
        _check(rc, fn)


def nsa_paged_attn_fwd_workspace_size(shape: NsaShape, max_cache_len: int = 0, window: int = 0, n_sink: int = 0) -> int:
    _int32("nsa_paged_attn_fwd_workspace_size", window=window, n_sink=n_sink)
    return int(load().nsa_paged_attn_fwd_workspace_size(ctypes.byref(shape), max_cache_len, window, n_sink))


def _scratch(fn, workspace, need, dev, index):
    """(tensor to keep alive, its address, its bytes) of a call's workspace."""
    if workspace is None:
        workspace = torch.empty(need, dtype=_U8, device=dev) if need else None
    elif not _fits(workspace, _U8, workspace.shape if workspace.dim() == 1 else (0,), index):
        _expect(fn, dev, workspace=(workspace, _U8, (None,)))
    return workspace, _addr(workspace), 0 if workspace is None else workspace.numel()


def nsa_paged_attn_fwd(q, k_pages, v_pages, block_table, cache_lens, window=0, n_sink=0, scale=0.0, *, cu_seqlens=None,
                       max_seqlen=None, max_cache_len=None, workspace=None, out=None, lse=None, stream=None):
    """Attention of new tokens q [B, T, H, d] or packed [tokens, H, d] over the paged cache (which
    already holds their keys), causal, with an optional window and n_sink tokens that stay
    visible beside it.  Returns out, shaped like q; fills lse [tokens, H] fp32 if given."""
    fn = "nsa_paged_attn_fwd"
    if (window | n_sink) >> 31:
        _int32(fn, window=window, n_sink=n_sink)
    dev = k_pages.device
    ctx, raw, share = _on(dev, stream)
    tokens, shp, n = _span_shape(fn, q, k_pages.shape[-2], k_pages.shape[-1], dev, cu_seqlens, max_seqlen)
    c, page, _, _ = _paged_cache(fn, k_pages, v_pages, block_table, cache_lens, n)
    rows = (tokens, q.shape[-2])
    if not _fits(out, _BF16, q.shape, dev.index) or not _fits(lse, _F32, rows, dev.index):
        _expect(fn, dev, out=(out, _BF16, q.shape), lse=(lse, _F32, rows))
    if max_cache_len is None:
        max_cache_len = c.max_pages * page
    lib, sp = load(), ctypes.byref(shp)
    with ctx:
        if out is None:
            out = torch.empty_like(q) if share is None else _new(q.shape, _BF16, dev, share)
        need = 0 if workspace is not None else lib.nsa_paged_attn_fwd_workspace_size(sp, max_cache_len, window, n_sink)
        ws, at, size = _scratch(fn, workspace, need, dev, dev.index)
        rc = lib.nsa_paged_attn_fwd(sp, q.data_ptr(), ctypes.byref(c), max_cache_len, window, n_sink, scale,
                                    out.data_ptr(), _addr(lse), at, size, raw)
    if rc:
        _check(rc, fn)
    return out


def nsa_paged_attn_weights(q, k_pages, lse, block_table, cache_lens, window=0, n_sink=0, scale=0.0, *, weights=None,
                           decay=1.0, cu_seqlens=None, max_seqlen=None, out=None, stream=None):
    """out[page, kv-head, row] = decay * weights + the attention probabilities that the queries of a
    nsa_paged_attn_fwd call (same masks, its lse) gave to the key, over the heads of its group.
    Without weights the sum alone; out may be weights (the default when weights are given).  Cells
    of no cached position are left as they were (in a new tensor they hold anything)."""
    fn = "nsa_paged_attn_weights"
    if (window | n_sink) >> 31:
        _int32(fn, window=window, n_sink=n_sink)
    dev = k_pages.device
    ctx, raw, share = _on(dev, stream)
    tokens, shp, n = _span_shape(fn, q, k_pages.shape[-2], k_pages.shape[-1], dev, cu_seqlens, max_seqlen)
    c, page, h_kv, _ = _paged_cache(fn, k_pages, None, block_table, cache_lens, n, weights)
    rows, cells = (tokens, q.shape[-2]), (k_pages.shape[0], h_kv, page)
    if lse is None or not _fits(lse, _F32, rows, dev.index) or not _fits(out, _F32, cells, dev.index):
        _expect(fn, dev, lse=(lse, _F32, rows), out=(out, _F32, cells))
        raise TypeError(f"{fn}: lse must be a tensor")
    with ctx:
        if out is None:
            out = weights if weights is not None else _new(cells, _F32, dev, share)
        rc = load().nsa_paged_attn_weights(ctypes.byref(shp), q.data_ptr(), ctypes.byref(c), lse.data_ptr(), window,
                                           n_sink, scale, decay, out.data_ptr(), raw)
    if rc:
        _check(rc, fn)
    return out


def nsa_paged_evict(k_pages, v_pages, weights, block_table, cache_lens, new_table, budget, n_sink=0, n_recent=0, *,
                    keep=None, new_lens=None, stream=None):
    """Cut every cache to at most `budget` keys per kv-head: the first n_sink, the last n_recent and
    the heaviest others, copied in order to new_table's pages (none of them in block_table, none
    listed twice).  Returns (keep [n_seqs, Hkv,
    budget] int32, -1 padded, and new_lens [n_seqs] int32)."""
    fn = "nsa_paged_evict"
    if (budget | n_sink | n_recent) >> 31:
        _int32(fn, budget=budget, n_sink=n_sink, n_recent=n_recent)
    dev = k_pages.device
    ctx, raw, share = _on(dev, stream)
    if weights is None:
        raise ValueError(f"{fn}: the cache has no weights")
    if not isinstance(cache_lens, torch.Tensor) or cache_lens.dim() != 1:
        raise ValueError(f"{fn}: cache_lens must be [n_seqs]")
    n = cache_lens.shape[0]
    c, _, h_kv, d = _paged_cache(fn, k_pages, v_pages, block_table, cache_lens, n, weights)
    width = new_table.shape[1] if isinstance(new_table, torch.Tensor) and new_table.dim() == 2 else 0
    kept = (n, h_kv, budget)
    if (new_table is None or not _fits(new_table, _I32, (n, width), dev.index)
            or not _fits(keep, _I32, kept, dev.index) or not _fits(new_lens, _I32, (n,), dev.index)):
        _expect(fn, dev, new_table=(new_table, _I32, (n, None)), keep=(keep, _I32, kept), new_lens=(new_lens, _I32, (n,)))
        raise TypeError(f"{fn}: new_table must be a tensor")
    with ctx:
        if keep is None:
            keep = _new((n, h_kv, max(0, budget)), _I32, dev, share)
        if new_lens is None:
            new_lens = _new((n,), _I32, dev, share)
        rc = load().nsa_paged_evict(n, h_kv, d, ctypes.byref(c), budget, n_sink, n_recent, new_table.data_ptr(), width,
                                    keep.data_ptr(), new_lens.data_ptr(), raw)
    if rc:
        _check(rc, fn)
    return keep, new_lens


# ----------------------------------------------------------------------------- rotation, 8-bit cache
def _rope(fn, dev, tokens, dims, h_kv, d, q, inv_freq, positions, interleaved, q_out, share):
    """(struct, q_out) of a rotation; q is shaped like the new tokens but for its heads."""
    if inv_freq is None or not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError(f"{fn}: inv_freq must be [rot_dim / 2]")
    index, pairs = dev.index, inv_freq.shape[0]
    if not _fits(inv_freq, _F32, (pairs,), index) or not _fits(positions, _I32, (tokens,), index):
        _expect(fn, dev, inv_freq=(inv_freq, _F32, (pairs,)), positions=(positions, _I32, (tokens,)))
    if q is None:
        if q_out is not None:
            raise ValueError(f"{fn}: q_out needs q")
        return NsaRope(inv_freq.data_ptr(), _addr(positions), 2 * pairs, int(bool(interleaved)), None, None), None
    heads = q.shape[-2] if isinstance(q, torch.Tensor) and q.dim() == len(dims) else 0
    if heads < 1 or heads % h_kv:
        raise ValueError(f"{fn}: q must be shaped like k_new, with heads a multiple of {h_kv}")
    shape = (*dims[:-2], heads, d)
    if not _fits(q, _BF16, shape, index) or not _fits(q_out, _BF16, shape, index):
        _expect(fn, dev, q=(q, _BF16, shape), q_out=(q_out, _BF16, shape))
    if q_out is None:
        q_out = _new(shape, _BF16, dev, share)
    return NsaRope(inv_freq.data_ptr(), _addr(positions), 2 * pairs, int(bool(interleaved)), q.data_ptr(),
                   q_out.data_ptr()), q_out


def nsa_paged_append_rope(k_new, v_new, k_pages, v_pages, block_table, cache_lens, inv_freq, *, q=None, positions=None,
                          interleaved=False, q_out=None, weights=None, cu_seqlens=None, max_seqlen=None, stream=None):
    """nsa_paged_append of keys that are rotated by their position on the way: pair i of the first
    2 * len(inv_freq) dimensions by position * inv_freq[i].  positions (int32 [tokens]) where the
    place in the cache is not the position.  With q (the same tokens' queries) returns them
    rotated too, in q_out (which may be q, and otherwise overlaps no input)."""
    fn = "nsa_paged_append_rope"
    dev = k_pages.device
    ctx, raw, share = _on(dev, stream)
    h_kv, d = k_pages.shape[-2:]
    tokens, shp, n = _span_shape(fn, k_new, h_kv, d, dev, cu_seqlens, max_seqlen)
    c = _paged_cache(fn, k_pages, v_pages, block_table, cache_lens, n, weights)[0]
    if v_new is None or k_new.shape[-2] != h_kv or not _fits(v_new, _BF16, k_new.shape, dev.index):
        want = (*k_new.shape[:-2], h_kv, d)
        _expect(fn, dev, k_new=(k_new, _BF16, want), v_new=(v_new, _BF16, want))
        raise TypeError(f"{fn}: v_new must be a tensor")
    with ctx:
        r, q_out = _rope(fn, dev, tokens, k_new.shape, h_kv, d, q, inv_freq, positions, interleaved, q_out, share)
        if q is not None:
            shp.h = q.shape[-2]
        rc = load().nsa_paged_append_rope(ctypes.byref(shp), k_new.data_ptr(), v_new.data_ptr(), ctypes.byref(r),
                                          ctypes.byref(c), raw)
    if rc:
        _check(rc, fn)
    return q_out


def _paged_cache_q8(fn, k_pages, v_pages, k_scales, v_scales, block_table, cache_lens, n_seqs):
    """(struct, page_size) of a cache held in 8 bits."""
    stride = _page_stride(fn, "k_pages", k_pages, _E4M3)
    shape = k_pages.shape
    n_pages, page, h_kv, _ = shape
    index = k_pages.get_device()
    if not (isinstance(v_pages, torch.Tensor) and v_pages.dtype is _E4M3 and v_pages.shape == shape
            and v_pages.stride() == k_pages.stride() and v_pages.get_device() == index):
        if _page_stride(fn, "v_pages", v_pages, _E4M3) != stride or v_pages.shape != shape:
            raise ValueError(f"{fn}: v_pages must have the shape and strides of k_pages")
        if v_pages.device != k_pages.device:
            raise ValueError(f"{fn}: v_pages is on {v_pages.device}, k_pages on {k_pages.device}")
    blocks = k_scales.shape[2] if isinstance(k_scales, torch.Tensor) and k_scales.dim() == 3 else 0
    if blocks < 1 or page % blocks:
        raise ValueError(f"{fn}: k_scales must be [n_pages, h_kv, page_size / block_size]")
    width = block_table.shape[1] if isinstance(block_table, torch.Tensor) and block_table.dim() == 2 else 0
    cells = (n_pages, h_kv, blocks)
    if (v_scales is None or block_table is None or cache_lens is None or not _fits(k_scales, _F32, cells, index)
            or not _fits(v_scales, _F32, cells, index) or not _fits(block_table, _I32, (n_seqs, width), index)
            or not _fits(cache_lens, _I32, (n_seqs,), index)):
        _expect(fn, k_pages.device, k_scales=(k_scales, _F32, cells), v_scales=(v_scales, _F32, cells),
                block_table=(block_table, _I32, (n_seqs, None)), cache_lens=(cache_lens, _I32, (n_seqs,)))
        raise TypeError(f"{fn}: v_scales, block_table and cache_lens must be tensors")
    return NsaPagedCacheQ8(k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                           block_table.data_ptr(), cache_lens.data_ptr(), n_pages, page, width, page // blocks,
                           stride), page


def nsa_paged_q8_append(k_new, v_new, k_pages, v_pages, k_scales, v_scales, block_table, cache_lens, *, q=None,
                        inv_freq=None, positions=None, interleaved=False, q_out=None, cu_seqlens=None, max_seqlen=None,
                        stream=None):
    """New tokens' keys and values into a cache held in 8 bits: pages float8_e4m3fn [n_pages,
    page_size, Hkv, d], scales fp32 [n_pages, Hkv, page_size / block_size], powers of two.  A block's
    scale grows with its largest value (its earlier codes are then rounded again).  With inv_freq
    the keys (and q, returned) are rotated on the way as by nsa_paged_append_rope."""
    fn = "nsa_paged_q8_append"
    dev = k_pages.device
    ctx, raw, share = _on(dev, stream)
    h_kv, d = k_pages.shape[-2:]
    tokens, shp, n = _span_shape(fn, k_new, h_kv, d, dev, cu_seqlens, max_seqlen)
    c, _ = _paged_cache_q8(fn, k_pages, v_pages, k_scales, v_scales, block_table, cache_lens, n)
    if v_new is None or k_new.shape[-2] != h_kv or not _fits(v_new, _BF16, k_new.shape, dev.index):
        want = (*k_new.shape[:-2], h_kv, d)
        _expect(fn, dev, k_new=(k_new, _BF16, want), v_new=(v_new, _BF16, want))
        raise TypeError(f"{fn}: v_new must be a tensor")
    if inv_freq is None and not (q is None and positions is None and q_out is None):
        raise ValueError(f"{fn}: q, positions and q_out need inv_freq")
    with ctx:
        r = None
        if inv_freq is not None:
            r, q_out = _rope(fn, dev, tokens, k_new.shape, h_kv, d, q, inv_freq, positions, interleaved, q_out, share)
            if q is not None:
                shp.h = q.shape[-2]
        rc = load().nsa_paged_q8_append(ctypes.byref(shp), k_new.data_ptr(), v_new.data_ptr(),
                                        None if r is None else ctypes.byref(r), ctypes.byref(c), raw)
    if rc:
        _check(rc, fn)
    return q_out


def nsa_paged_q8_attn_fwd_workspace_size(shape: NsaShape, cache: NsaPagedCacheQ8, max_cache_len: int = 0,
                                         window: int = 0, n_sink: int = 0) -> int:
    _int32("nsa_paged_q8_attn_fwd_workspace_size", window=window, n_sink=n_sink)
    return int(load().nsa_paged_q8_attn_fwd_workspace_size(ctypes.byref(shape), ctypes.byref(cache), max_cache_len,
                                                           window, n_sink))


def nsa_paged_q8_attn_fwd(q, k_pages, v_pages, k_scales, v_scales, block_table, cache_lens, window=0, n_sink=0,
                          scale=0.0, *, cu_seqlens=None, max_seqlen=None, max_cache_len=None, workspace=None, out=None,
                          lse=None, stream=None):
    """nsa_paged_attn_fwd over a cache held in 8 bits (as nsa_paged_q8_append writes it): k = code *
    k_scale, v = code * v_scale.  Calls of more than 256 rows (tokens x heads of a group) expand the keys that they see
    to bf16 in the workspace first, which max_cache_len sizes: give it where tables are much wider than caches.
    There it has to bound cache_lens: the queries of a longer cache see no key (out = 0, lse = -inf, no error).
    None is always right."""
    fn = "nsa_paged_q8_attn_fwd"
    if (window | n_sink) >> 31:
        _int32(fn, window=window, n_sink=n_sink)
    dev = k_pages.device
    ctx, raw, share = _on(dev, stream)
    tokens, shp, n = _span_shape(fn, q, k_pages.shape[-2], k_pages.shape[-1], dev, cu_seqlens, max_seqlen)
    c, page = _paged_cache_q8(fn, k_pages, v_pages, k_scales, v_scales, block_table, cache_lens, n)
    rows = (tokens, q.shape[-2])
    if not _fits(out, _BF16, q.shape, dev.index) or not _fits(lse, _F32, rows, dev.index):
        _expect(fn, dev, out=(out, _BF16, q.shape), lse=(lse, _F32, rows))
    if max_cache_len is None:
        max_cache_len = c.max_pages * page
    lib, sp = load(), ctypes.byref(shp)
    with ctx:
        if out is None:
            out = torch.empty_like(q) if share is None else _new(q.shape, _BF16, dev, share)
        need = 0 if workspace is not None else lib.nsa_paged_q8_attn_fwd_workspace_size(sp, ctypes.byref(c), max_cache_len, window, n_sink)
        ws, at, size = _scratch(fn, workspace, need, dev, dev.index)
        rc = lib.nsa_paged_q8_attn_fwd(sp, q.data_ptr(), ctypes.byref(c), max_cache_len, window, n_sink, scale,
                                       out.data_ptr(), _addr(lse), at, size, raw)
    if rc:
        _check(rc, fn)
    return out


# ----------------------------------------------------------------------------- window with sinks
def nsa_swa_sink_fwd_workspace_size(shape: NsaShape, window: int = 512, n_sink: int = 4) -> int:
    _int32("nsa_swa_sink_fwd_workspace_size", window=window, n_sink=n_sink)
    return int(load().nsa_swa_sink_fwd_workspace_size(ctypes.byref(shape), window, n_sink))


def _packed_kv(fn, q, k, v, cu_seqlens, max_seqlen):
    """_span_shape of q, with k and v checked against it."""
    if not isinstance(k, torch.Tensor) or k.dim() != q.dim() or q.dim() not in (3, 4) or k.shape[-2] == 0:
        raise ValueError(f"{fn}: q and k must both be [B, T, heads, d] or packed [tokens, heads, d]")
    r = _span_shape(fn, q, k.shape[-2], q.shape[-1], q.device, cu_seqlens, max_seqlen)
    kv = (*q.shape[:-2], k.shape[-2], q.shape[-1])
    index = q.get_device()
    if v is None or not _fits(k, _BF16, kv, index) or not _fits(v, _BF16, kv, index):
        _expect(fn, q.device, k=(k, _BF16, kv), v=(v, _BF16, kv))
        raise TypeError(f"{fn}: v must be a tensor")
    return r


def nsa_swa_sink_fwd(q, k, v, window=512, n_sink=4, scale=0.0, *, cu_seqlens=None, max_seqlen=None, workspace=None,
                     out=None, lse=None, stream=None):
    """Sliding window beside which the first n_sink tokens of each sequence stay visible.  Returns
    out, shaped like q; fills lse [tokens, H] fp32 if given."""
    fn = "nsa_swa_sink_fwd"
    if (window | n_sink) >> 31:
        _int32(fn, window=window, n_sink=n_sink)
    dev = q.device
    ctx, raw, share = _on(dev, stream)
    tokens, shp, _ = _packed_kv(fn, q, k, v, cu_seqlens, max_seqlen)
    rows = (tokens, q.shape[-2])
    if not _fits(out, _BF16, q.shape, dev.index) or not _fits(lse, _F32, rows, dev.index):
        _expect(fn, dev, out=(out, _BF16, q.shape), lse=(lse, _F32, rows))
    lib, sp = load(), ctypes.byref(shp)
    with ctx:
        if out is None:
            out = torch.empty_like(q) if share is None else _new(q.shape, _BF16, dev, share)
        need = 0 if workspace is not None else lib.nsa_swa_sink_fwd_workspace_size(sp, window, n_sink)
        ws, at, size = _scratch(fn, workspace, need, dev, dev.index)
        rc = lib.nsa_swa_sink_fwd(sp, q.data_ptr(), k.data_ptr(), v.data_ptr(), window, n_sink, scale, out.data_ptr(),
                                  _addr(lse), at, size, raw)
    if rc:
        _check(rc, fn)
    return out


def nsa_swa_sink_bwd_workspace_size(shape: NsaShape, window: int = 512, n_sink: int = 4) -> int:
    _int32("nsa_swa_sink_bwd_workspace_size", window=window, n_sink=n_sink)
    return int(load().nsa_swa_sink_bwd_workspace_size(ctypes.byref(shape), window, n_sink))


def nsa_swa_sink_bwd(q, k, v, o, lse, d_o, window=512, n_sink=4, scale=0.0, *, cu_seqlens=None, max_seqlen=None,
                     workspace=None, dq=None, dk=None, dv=None, stream=None):
    """Backward of nsa_swa_sink_fwd: (dq, dk, dv) shaped like q, k, v from its o and lse."""
    fn = "nsa_swa_sink_bwd"
    if (window | n_sink) >> 31:
        _int32(fn, window=window, n_sink=n_sink)
    dev = q.device
    ctx, raw, share = _on(dev, stream)
    tokens, shp, _ = _packed_kv(fn, q, k, v, cu_seqlens, max_seqlen)
    rows = (tokens, q.shape[-2])
    like_q, like_k = q.shape, k.shape
    if (o is None or d_o is None or lse is None
            or not all(_fits(t, _BF16, like_q, dev.index) for t in (o, d_o, dq))
            or not all(_fits(t, _BF16, like_k, dev.index) for t in (dk, dv)) or not _fits(lse, _F32, rows, dev.index)):
        _expect(fn, dev, o=(o, _BF16, like_q), d_o=(d_o, _BF16, like_q), lse=(lse, _F32, rows), dq=(dq, _BF16, like_q),
                dk=(dk, _BF16, like_k), dv=(dv, _BF16, like_k))
        raise TypeError(f"{fn}: o, lse and d_o must be tensors")
    lib, sp = load(), ctypes.byref(shp)
    with ctx:
        dq = _new(like_q, _BF16, dev, share) if dq is None else dq
        dk = _new(like_k, _BF16, dev, share) if dk is None else dk
        dv = _new(like_k, _BF16, dev, share) if dv is None else dv
        need = 0 if workspace is not None else lib.nsa_swa_sink_bwd_workspace_size(sp, window, n_sink)
        ws, at, size = _scratch(fn, workspace, need, dev, dev.index)
        rc = lib.nsa_swa_sink_bwd(sp, q.data_ptr(), k.data_ptr(), v.data_ptr(), window, n_sink, scale, o.data_ptr(),
                                  lse.data_ptr(), d_o.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), at, size,
                                  raw)
    if rc:
        _check(rc, fn)
    return dq, dk, dv
