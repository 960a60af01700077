"""block_sparse_flash_gb300 -- Python binding of libsplash.so, the sm_103a
block-sparse (Splash) masked attention forward library.

This module only marshals arguments, through ctypes and for the serving calls
through a compiled module (csrc/binding.cpp): torch tensors become device
pointers, the current torch stream becomes the cudaStream_t.  Every step of the
computation runs in the library's CUDA kernels (rope_table, a constant laid
out once, is the exception); there is no CPU or PyTorch fallback.  If the
library has not been built, importing works but every call raises
SplashLibraryMissing; so do the serving calls without the compiled module.

    spec = MaskSpec(causal=True, window_left=4095)
    mi = build_mask_info(spec, L, L, 128, 128)
    out, lse = attention_fwd(q, k, v, mi, scale=1 / 128 ** 0.5, softcap=30.0)

Serving, with positions rotated: rope_fwd / rope_bwd around the attention,
paged_append for the keys and values of new tokens, paged_decode for their
attention over the pages.  rope_axes_fwd / rope_axes_bwd / paged_append_axes
take several position axes, paged_tree_decode a tree of drafted tokens,
paged_compact, paged_remap and paged_copy keep the pages in order.

C ABI: include/splash.h.
"""
import ctypes
import functools
import importlib.util
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libsplash.so")

SPLASH_OK = 0
_STATUS = {
    0: "SPLASH_OK", 1: "SPLASH_ERR_INVALID_ARG", 2: "SPLASH_ERR_SHAPE", 3: "SPLASH_ERR_UNSUPPORTED",
    4: "SPLASH_ERR_CUDA", 5: "SPLASH_ERR_DEVICE_TIMEOUT", 6: "SPLASH_ERR_OOM", 7: "SPLASH_ERR_DEVICE_CHECK",
}


class SplashLibraryMissing(RuntimeError):
    pass


class SplashError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {_status_string(status)}")


class _Spec(ctypes.Structure):
    _fields_ = [
        ("causal", ctypes.c_int32),
        ("window_left", ctypes.c_int64),
        ("window_right", ctypes.c_int64),
        ("q_segment_ids", ctypes.c_void_p),
        ("kv_segment_ids", ctypes.c_void_p),
        ("batch", ctypes.c_int32),
    ]


_lib = None


def lib():
    """The loaded libsplash.so (ctypes.CDLL); raises SplashLibraryMissing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise SplashLibraryMissing(
            f"{LIB_PATH} is missing: build it with block_sparse_flash_gb300.build.build() "
            "(there is no fallback implementation)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    P = ctypes.POINTER
    L.splash_build_mask_info.argtypes = [P(_Spec), i64, i64, i32, i32, vp, P(vp)]
    L.splash_mask_info_rebuild.argtypes = [vp, P(_Spec), i64, i64, i32, i32, vp]
    L.splash_mask_info_shape.argtypes = [vp, P(i32), P(i64), P(i64), P(i32), P(i32)]
    L.splash_mask_info_counts.argtypes = [vp, P(i64), P(i64), P(i64), P(i64)]
    L.splash_mask_info_to_host.argtypes = [vp] + [vp] * 8
    L.splash_mask_info_destroy.argtypes = [vp]
    L.splash_mask_info_destroy.restype = None
    L.splash_attention_fwd.argtypes = [vp, vp, vp, i32, i32, i32, i64, i64, i32, i32, vp, vp, vp, f32, f32,
                                       vp, vp, vp]
    L.splash_attention_fwd_split.argtypes = [vp, vp, vp, i32, i32, i32, i64, i64, i32, i32, vp, vp, vp, f32, f32,
                                             i32, vp, vp, vp]
    L.splash_attention_fwd_mle.argtypes = [vp, vp, vp, i32, i32, i32, i64, i64, i32, i32, vp, vp, vp, f32, f32,
                                           f32, vp, vp, vp]
    L.splash_attention_bwd_workspace_size.argtypes = [i32, i32, i64, i32, P(ctypes.c_size_t)]
    L.splash_attention_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i64, i64, i32, i32, vp, vp, vp,
                                       f32, f32, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.splash_mask_info_set_pattern_source.argtypes = [vp, i32]
    L.splash_attention_fwd_host.argtypes = [vp, vp, vp, i32, i32, i32, i64, i64, i32, i32, vp, vp, vp, f32, f32,
                                            vp, vp, vp, vp, vp, vp, vp, vp]
    L.splash_paged_decode_workspace_size.argtypes = [i32] * 9 + [i64, P(ctypes.c_size_t)]
    L.splash_paged_decode_workspace_size.restype = ctypes.c_int
    L.splash_paged_tree_decode_workspace_size.argtypes = [i32] * 9 + [i64, P(ctypes.c_size_t)]
    L.splash_paged_tree_decode_workspace_size.restype = ctypes.c_int
    L.splash_paged_remap_workspace_size.argtypes = [i64, i32, P(ctypes.c_size_t)]
    L.splash_paged_remap_workspace_size.restype = ctypes.c_int
    L.splash_attention_merge.argtypes = [vp, vp, i32, i64, i32, vp, vp, vp]
    L.splash_last_device_error.argtypes = [vp]
    L.splash_debug_wait_selftest.argtypes = [ctypes.c_uint64, vp]
    L.splash_status_string.argtypes = [ctypes.c_int]
    L.splash_status_string.restype = ctypes.c_char_p
    L.splash_version.argtypes = []
    L.splash_version.restype = ctypes.c_char_p
    L.splash_shard_items.argtypes = [i32, i32, i32, i32, P(i64), P(i64)]
    L.splash_kernel_launches.argtypes = []
    L.splash_kernel_launches.restype = ctypes.c_uint64
    for f in (L.splash_build_mask_info, L.splash_mask_info_rebuild, L.splash_mask_info_shape,
              L.splash_mask_info_counts, L.splash_mask_info_to_host, L.splash_attention_fwd,
              L.splash_attention_fwd_split, L.splash_attention_merge,
              L.splash_last_device_error, L.splash_debug_wait_selftest, L.splash_shard_items):
        f.restype = ctypes.c_int
    _lib = L
    return L


def _status_string(s):
    try:
        return lib().splash_status_string(int(s)).decode()
    except SplashLibraryMissing:
        return _STATUS.get(int(s), f"status {s}")


def _check(status, what):
    if status != SPLASH_OK:
        raise SplashError(status, what)


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


@dataclass
class MaskSpec:
    """Joint mask = causal AND window AND segment equality (splash_mask_spec).

    window_left / window_right: inclusive distances, -1 = unbounded.
    q_segment_ids / kv_segment_ids: int32 CUDA tensors [batch, L] (or [L]) or None.
    """
    causal: bool = False
    window_left: int = -1
    window_right: int = -1
    q_segment_ids: Optional[torch.Tensor] = None
    kv_segment_ids: Optional[torch.Tensor] = None

    def _c(self):
        qs, kvs, batch = self.q_segment_ids, self.kv_segment_ids, 0
        for t in (qs, kvs):
            if t is not None and (t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous()):
                raise ValueError("segment ids must be contiguous int32 CUDA tensors")
        if qs is not None:
            batch = 1 if qs.dim() == 1 else qs.shape[0]
        return _Spec(int(bool(self.causal)), int(self.window_left), int(self.window_right),
                     qs.data_ptr() if qs is not None else None,
                     kvs.data_ptr() if kvs is not None else None, batch)


class MaskInfo:
    """Owner of a splash_mask_info handle (device memory freed on close)."""

    def __init__(self, handle):
        self._h = ctypes.c_void_p(handle)

    @property
    def handle(self):
        if not self._h:
            raise ValueError("MaskInfo is closed")
        return self._h

    def close(self):
        if self._h:
            lib().splash_mask_info_destroy(self._h)
            self._h = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def rebuild(self, spec: MaskSpec, Lq, Lk, bq, bk, stream=None):
        s = spec._c()
        _check(lib().splash_mask_info_rebuild(self.handle, ctypes.byref(s), Lq, Lk, bq, bk, _stream(stream)),
               "splash_mask_info_rebuild")
        return self

    def shape(self):
        bm, bq, bk = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        nq, nk = ctypes.c_int64(), ctypes.c_int64()
        _check(lib().splash_mask_info_shape(self.handle, ctypes.byref(bm), ctypes.byref(nq), ctypes.byref(nk),
                                            ctypes.byref(bq), ctypes.byref(bk)), "splash_mask_info_shape")
        return dict(batch_rows=bm.value, nq=nq.value, nk=nk.value, bq=bq.value, bk=bk.value)

    def set_pattern_source(self, source: str):
        """'stored' (default) or 'positions': the forward computes partial
        blocks' masks from positions, and for a table built with segment IDs
        from the segment arrays, which every forward call must then pass."""
        code = {"stored": 0, "positions": 1}[source]
        _check(lib().splash_mask_info_set_pattern_source(self.handle, code), "splash_mask_info_set_pattern_source")

    def counts(self):
        a, p, n, u = (ctypes.c_int64() for _ in range(4))
        _check(lib().splash_mask_info_counts(self.handle, ctypes.byref(a), ctypes.byref(p), ctypes.byref(n),
                                             ctypes.byref(u)), "splash_mask_info_counts")
        return dict(num_active=a.value, num_partial=p.value, num_patterns=n.value, allowed_pairs=u.value)

    def to_host(self):
        """All table arrays as numpy arrays (synchronous copy)."""
        sh, c = self.shape(), self.counts()
        R, A, P = sh["batch_rows"] * sh["nq"], c["num_active"], c["num_patterns"]
        out = dict(
            block_mask=np.zeros((sh["batch_rows"], sh["nq"], sh["nk"]), dtype=np.int8),
            row_ptr=np.zeros(R + 1, dtype=np.int32),
            active_rows=np.zeros(max(A, 1), dtype=np.int32),
            active_cols=np.zeros(max(A, 1), dtype=np.int32),
            mask_next=np.zeros(max(A, 1), dtype=np.int32),
            bounds_start=np.zeros(max(A, 1), dtype=np.uint8),
            bounds_end=np.zeros(max(A, 1), dtype=np.uint8),
            partial_mask_blocks=np.zeros((max(P, 1), sh["bq"], sh["bk"]), dtype=np.uint8),
        )
        order = ["block_mask", "row_ptr", "active_rows", "active_cols", "mask_next", "bounds_start",
                 "bounds_end", "partial_mask_blocks"]
        _check(lib().splash_mask_info_to_host(self.handle, *[out[k].ctypes.data for k in order]),
               "splash_mask_info_to_host")
        for k in ("active_rows", "active_cols", "mask_next", "bounds_start", "bounds_end"):
            out[k] = out[k][:A]
        out["partial_mask_blocks"] = out["partial_mask_blocks"][:P]
        out.update(c)
        out.update(sh)
        return out


def build_mask_info(spec: MaskSpec, Lq: int, Lk: int, bq: int, bk: int, stream=None) -> MaskInfo:
    """The sparse execution table of `spec` on a (Lq, Lk) grid of bq x bk
    blocks (splash_build_mask_info): bk in {64, 128}, bq in {64, 128, 256}.
    The forward takes bq == bk, or bq = 256 with bk = 128 (each 256-row
    q-block computed as two 128-row tiles of one head sharing every K/V tile,
    the faster choice for MHA); the backward takes 128 x 128."""
    h = ctypes.c_void_p()
    s = spec._c()
    _check(lib().splash_build_mask_info(ctypes.byref(s), Lq, Lk, bq, bk, _stream(stream), ctypes.byref(h)),
           "splash_build_mask_info")
    return MaskInfo(h.value)


def _qkv_shapes(q, k, v):
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q, k, v must be contiguous 4-D bf16 CUDA tensors")
    B, Hq, Lq, dqk = q.shape
    return B, Hq, Lq, dqk, k.shape[1], k.shape[2], v.shape[3]


def attention_fwd(q, k, v, mask_info: MaskInfo, scale: float, softcap: float = 0.0, q_segment_ids=None,
                  kv_segment_ids=None, out=None, lse=None, stream=None, num_splits: int = 1,
                  max_logit=None):
    """out [B, Hq, Lq, dv] bf16 and lse [B, Hq, Lq] fp32 (allocated if not given).

    num_splits > 1 runs the split-KV forward into fp32 workspace allocated
    here, then the LSE merge (same result).  max_logit = c runs the Max Logit
    Estimate variant (the softmax reference fixed at c; same result while c
    is in the safe range, e.g. c = softcap)."""
    B, Hq, Lq, dqk, Hkv, Lk, dv = _qkv_shapes(q, k, v)
    if out is None:
        out = torch.empty((B, Hq, Lq, dv), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    if max_logit is not None:
        if num_splits > 1:
            raise ValueError("max_logit is supported by the one-pass forward only (num_splits == 1)")
        _check(lib().splash_attention_fwd_mle(_ptr(q), _ptr(k), _ptr(v), B, Hq, Hkv, Lq, Lk, dqk, dv,
                                              _ptr(q_segment_ids), _ptr(kv_segment_ids), mask_info.handle,
                                              float(scale), float(softcap), float(max_logit), _ptr(out),
                                              _ptr(lse), _stream(stream)),
               "splash_attention_fwd_mle")
        return out, lse
    if num_splits > 1:
        o_part, lse_part = attention_fwd_split(q, k, v, mask_info, scale, softcap, num_splits, q_segment_ids,
                                               kv_segment_ids, stream=stream)
        return attention_merge(o_part, lse_part, out=out, lse=lse, stream=stream)
    _check(lib().splash_attention_fwd(_ptr(q), _ptr(k), _ptr(v), B, Hq, Hkv, Lq, Lk, dqk, dv,
                                      _ptr(q_segment_ids), _ptr(kv_segment_ids), mask_info.handle,
                                      float(scale), float(softcap), _ptr(out), _ptr(lse), _stream(stream)),
           "splash_attention_fwd")
    return out, lse


def attention_fwd_host(q_host, k_host, v_host, mask_info: MaskInfo, scale: float, softcap: float = 0.0,
                       out_host=None, lse_host=None, q=None, k=None, v=None, out=None, lse=None,
                       q_segment_ids=None, kv_segment_ids=None, stream=None):
    """attention_fwd for CPU tensors (pinned for overlap): copies in, computes
    and copies out, pipelined in chunks.  Device buffers q, k, v, out, lse are
    allocated on the current device when not given.  Returns (out_host,
    lse_host); they are complete once the stream has reached this point."""
    for t in (q_host, k_host, v_host):
        if t.dtype != torch.bfloat16 or t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q_host, k_host, v_host must be contiguous 4-D bf16 CPU tensors")
    B, Hq, Lq, dqk = q_host.shape
    Hkv, Lk, dv = k_host.shape[1], k_host.shape[2], v_host.shape[3]
    dev = torch.device("cuda", torch.cuda.current_device())
    if out_host is None:
        out_host = torch.empty((B, Hq, Lq, dv), dtype=torch.bfloat16).pin_memory()
    if lse_host is None:
        lse_host = torch.empty((B, Hq, Lq), dtype=torch.float32).pin_memory()
    q = torch.empty_like(q_host, device=dev) if q is None else q
    k = torch.empty_like(k_host, device=dev) if k is None else k
    v = torch.empty_like(v_host, device=dev) if v is None else v
    out = torch.empty((B, Hq, Lq, dv), dtype=torch.bfloat16, device=dev) if out is None else out
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=dev) if lse is None else lse
    _check(lib().splash_attention_fwd_host(_ptr(q_host), _ptr(k_host), _ptr(v_host), B, Hq, Hkv, Lq, Lk, dqk, dv,
                                           _ptr(q_segment_ids), _ptr(kv_segment_ids), mask_info.handle,
                                           float(scale), float(softcap), _ptr(out_host), _ptr(lse_host), _ptr(q),
                                           _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _stream(stream)),
           "splash_attention_fwd_host")
    return out_host, lse_host


def attention_fwd_split(q, k, v, mask_info: MaskInfo, scale: float, softcap: float, num_splits: int,
                        q_segment_ids=None, kv_segment_ids=None, o_part=None, lse_part=None, stream=None):
    """Split-KV partials: o_part [S, B, Hq, Lq, dv] fp32 and lse_part [S, B, Hq, Lq] fp32."""
    B, Hq, Lq, dqk, Hkv, Lk, dv = _qkv_shapes(q, k, v)
    if o_part is None:
        o_part = torch.empty((num_splits, B, Hq, Lq, dv), dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty((num_splits, B, Hq, Lq), dtype=torch.float32, device=q.device)
    _check(lib().splash_attention_fwd_split(_ptr(q), _ptr(k), _ptr(v), B, Hq, Hkv, Lq, Lk, dqk, dv,
                                            _ptr(q_segment_ids), _ptr(kv_segment_ids), mask_info.handle,
                                            float(scale), float(softcap), int(num_splits), _ptr(o_part),
                                            _ptr(lse_part), _stream(stream)),
           "splash_attention_fwd_split")
    return o_part, lse_part


def attention_merge(o_part, lse_part, out=None, lse=None, stream=None):
    """Merges split-KV partials [S, ..., dv] / [S, ...] into bf16 out [..., dv] and fp32 lse [...]."""
    if o_part.dtype != torch.float32 or lse_part.dtype != torch.float32 or not o_part.is_contiguous() \
            or not lse_part.is_contiguous():
        raise ValueError("o_part and lse_part must be contiguous fp32 tensors")
    S, dv = o_part.shape[0], o_part.shape[-1]
    rows = lse_part[0].numel()
    if out is None:
        out = torch.empty(o_part.shape[1:], dtype=torch.bfloat16, device=o_part.device)
    if lse is None:
        lse = torch.empty(lse_part.shape[1:], dtype=torch.float32, device=o_part.device)
    _check(lib().splash_attention_merge(_ptr(o_part), _ptr(lse_part), int(S), int(rows), int(dv), _ptr(out),
                                        _ptr(lse), _stream(stream)), "splash_attention_merge")
    return out, lse


def attention_bwd(q, k, v, out, lse, dout, mask_info: MaskInfo, scale: float, softcap: float = 0.0,
                  q_segment_ids=None, kv_segment_ids=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of attention_fwd for the upstream gradient dout,
    from the forward's out and lse (bf16 tensors shaped like q, k, v; allocated
    if not given).  workspace: optional uint8 device tensor of at least
    attention_bwd_workspace_size(...) bytes."""
    B, Hq, Lq, dqk, Hkv, Lk, dvd = _qkv_shapes(q, k, v)
    for name, t, shape, dt in (("out", out, (B, Hq, Lq, dvd), torch.bfloat16),
                               ("dout", dout, (B, Hq, Lq, dvd), torch.bfloat16),
                               ("lse", lse, (B, Hq, Lq), torch.float32)):
        if tuple(t.shape) != shape or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {shape}")
    if dq is None:
        dq = torch.empty_like(q)
    if dk is None:
        dk = torch.empty_like(k)
    if dv is None:
        dv = torch.empty_like(v)
    need = attention_bwd_workspace_size(B, Hq, Lq, dqk)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(lib().splash_attention_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), B, Hq, Hkv,
                                      Lq, Lk, dqk, dvd, _ptr(q_segment_ids), _ptr(kv_segment_ids),
                                      mask_info.handle, float(scale), float(softcap), _ptr(dq), _ptr(dk), _ptr(dv),
                                      _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                                      _stream(stream)),
           "splash_attention_bwd")
    return dq, dk, dv


def attention_bwd_workspace_size(B: int, Hq: int, Lq: int, dqk: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().splash_attention_bwd_workspace_size(int(B), int(Hq), int(Lq), int(dqk), ctypes.byref(n)),
           "splash_attention_bwd_workspace_size")
    return int(n.value)


def shard_items(B: int, Hkv: int, world: int, rank: int):
    """This rank's half-open range [begin, end) of the B * Hkv (batch, KV
    head) groups when a workload is split across `world` GPUs
    (splash_shard_items)."""
    b, e = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().splash_shard_items(int(B), int(Hkv), int(world), int(rank), ctypes.byref(b), ctypes.byref(e)),
           "splash_shard_items")
    return b.value, e.value


def shard_views(q, k, v, begin: int, end: int, out=None, lse=None, segment_ids=None):
    """Sub-tensors of groups [begin, end) as a problem of (end - begin) batch
    rows, Hq / Hkv query heads and one KV head: views of q [B, Hq, L, dqk],
    k, v, out and lse (no copy), and with segment IDs [B, L] a per-group copy
    of the rows they read (row g // Hkv for group g).  Returns a dict with
    the same keys."""
    B, Hq, Lq, dqk = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    r = dict(q=q.view(B * Hkv, G, Lq, dqk)[begin:end],
             k=k.view(B * Hkv, 1, k.shape[2], k.shape[3])[begin:end],
             v=v.view(B * Hkv, 1, v.shape[2], v.shape[3])[begin:end])
    if out is not None:
        r["out"] = out.view(B * Hkv, G, Lq, out.shape[3])[begin:end]
    if lse is not None:
        r["lse"] = lse.view(B * Hkv, G, Lq)[begin:end]
    if segment_ids is not None:
        idx = torch.arange(begin, end, device=segment_ids.device) // Hkv
        r["segment_ids"] = segment_ids.index_select(0, idx).contiguous()
    return r


# ---- serving: rotary positions, paged append, paged decode

_CACHE_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}
_binding = None


def _native():
    """The compiled part of the binding (csrc/binding.cpp): the serving calls,
    whose kernels take a few microseconds, as long as reading their tensors'
    attributes from Python would.  Raises SplashLibraryMissing."""
    global _binding
    if _binding is None:
        from .build import binding_path
        lib()
        path = binding_path()
        if not os.path.exists(path):
            raise SplashLibraryMissing(
                f"{path} is missing: build it with block_sparse_flash_gb300.build.build() "
                "(there is no fallback implementation)")
        spec = importlib.util.spec_from_file_location("_binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.set_error(SplashError)
        _binding = module
    return _binding


def _handle(stream):
    """The handle of a call's stream; None: torch's current one."""
    if not isinstance(stream, torch.cuda.Stream):
        return None if stream is None else int(stream)
    if stream.device_index != torch.cuda.current_device():
        raise ValueError(f"the stream must be on the current CUDA device (got one of cuda:{stream.device_index})")
    return stream.cuda_stream


def rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """The rotations of positions 0 .. max_positions - 1 for rope_fwd and
    paged_append: fp32 [max_positions, rot_dim], cosines then sines of
    position * base^(-2i / rot_dim), from 64-bit angles (far positions would
    lose their angle in 32 bits).  Any other table of that layout will do."""
    f = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def _rope(inverse, q, k, positions, table, rot_offset, interleaved, q_out, k_out, stream):
    return (_binding or _native()).rope(q, k, positions, table, rot_offset, interleaved, inverse, q_out, k_out,
                                        _handle(stream))


def rope_fwd(q, k, positions, table, rot_offset: int = 0, interleaved: bool = False, q_out=None, k_out=None,
             stream=None):
    """q [B, Hq, L, d] and k [B, Hkv, L, d] (bf16, any strides with d
    contiguous; k may be None) rotated by positions (int32 [B, L] or [L];
    negative: not rotated).  table: fp32 [positions, rot_dim] (rope_table); the
    rotated dimensions start at rot_offset, pairs are half a rotation apart or
    adjacent (interleaved).  Returns (q_out, k_out), dense unless given;
    q_out=q rotates in place (splash_rope)."""
    return _rope(0, q, k, positions, table, rot_offset, interleaved, q_out, k_out, stream)


def rope_bwd(dq, dk, positions, table, rot_offset: int = 0, interleaved: bool = False, dq_out=None, dk_out=None,
             stream=None):
    """The gradients of rope_fwd's inputs from those of its outputs (the
    transposed rotation); arguments as rope_fwd."""
    return _rope(1, dq, dk, positions, table, rot_offset, interleaved, dq_out, dk_out, stream)


def paged_append(k, v, k_cache, v_cache, block_table, positions, q=None, table=None, rot_offset: int = 0,
                 interleaved: bool = False, seq_ids=None, k_scale=None, v_scale=None, q_out=None, k_out=None,
                 stream=None):
    """Writes k [B, Hkv, L, dqk] and v [B, Hkv, L, dv] of new tokens into the
    pages of their sequences, rotating k (and q) on the way when a table is
    given (splash_paged_append).  Returns (q_out, k_out).

    k_cache, v_cache: [pages, Hkv, page_size, d], bf16 or float8_e4m3fn (then
    with k_scale, v_scale fp32 [Hkv]); pages stored token by token are passed
    as cache.transpose(1, 2).  block_table: int32 [sequences, max_pages].
    positions, seq_ids: int32 [B, L] or [L]; a negative position is padding
    (nothing is stored); seq_ids is the row of block_table (default: b).
    q [B, Hq, L, dqk] is rotated into q_out (allocated if not given); k_out
    receives the rotated keys when given (for attention_fwd of a prompt)."""
    return (_binding or _native()).paged_append(k, v, k_cache, v_cache, block_table, positions, q, table, rot_offset,
                                                interleaved, seq_ids, k_scale, v_scale, q_out, k_out, _handle(stream))


def paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale: float, softcap: float = 0.0,
                 window_left: int = -1, k_scale=None, v_scale=None, out=None, lse=None, workspace=None, stream=None):
    """out [B, Hq, Lq, dv] bf16 and lse [B, Hq, Lq] fp32 of the newest Lq
    (1 .. 16) tokens of each sequence over its pages (splash_paged_decode).

    q [B, Hq, Lq, dqk]: bf16, any strides with dqk contiguous.  seq_lens: int32
    [B], cached tokens, the Lq new ones among them.  Caches, scales and
    block_table [B, max_pages] as for paged_append.  workspace: optional uint8
    device tensor of at least paged_decode_workspace_size(...) bytes, not
    shared by calls that may overlap."""
    return (_binding or _native()).paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale, softcap,
                                                window_left, k_scale, v_scale, out, lse, workspace, _handle(stream))


@functools.lru_cache(maxsize=256)
def _decode_workspace_size(name, *sizes):
    n = ctypes.c_size_t(0)
    _check(getattr(lib(), name)(*sizes, ctypes.byref(n)), name)
    return int(n.value)


def _workspace_of(name, q, k_cache, v_cache, block_table, window_left):
    if q.dim() != 4 or k_cache.dim() != 4 or v_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q, k_cache and v_cache must be 4-D and block_table 2-D")
    if k_cache.dtype not in _CACHE_TYPES:
        raise ValueError("k_cache and v_cache must be bf16 or float8_e4m3fn tensors")
    return _decode_workspace_size(name, q.shape[0], q.shape[1], k_cache.shape[1], q.shape[2], q.shape[3],
                                  v_cache.shape[3], block_table.shape[1], k_cache.shape[2],
                                  _CACHE_TYPES[k_cache.dtype], int(window_left))


def paged_decode_workspace_size(q, k_cache, v_cache, block_table, window_left: int = -1) -> int:
    """Bytes of paged_decode's workspace for tensors of these shapes and types
    (0 where it needs none)."""
    return _workspace_of("splash_paged_decode_workspace_size", q, k_cache, v_cache, block_table, window_left)


# ---- several position axes, trees of drafted tokens, upkeep of the paged cache


def rope_axis_map(sections, cycled: bool = False) -> bytes:
    """The `axes` argument of rope_axes_fwd and paged_append_axes: which axis
    each rotated pair turns by.  sections: pairs of each axis, e.g. (16, 24, 24)
    for time, height and width; in a row, or (cycled) taking turns from pair to
    pair until each is used up.  Laid out once."""
    left = [int(n) for n in sections]
    if not left or min(left) < 0 or len(left) > 255:
        raise ValueError("sections must be a pair count for each axis")
    if not cycled:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    return bytes(a for i in range(max(left)) for a, n in enumerate(left) if i < n)


def _rope_axes(inverse, q, k, positions, table, axes, rot_offset, interleaved, q_out, k_out, stream):
    return (_binding or _native()).rope_axes(q, k, positions, table, axes, rot_offset, interleaved, inverse, q_out, k_out,
                                             _handle(stream))


def rope_axes_fwd(q, k, positions, table, axes, rot_offset: int = 0, interleaved: bool = False, q_out=None, k_out=None,
                  stream=None):
    """rope_fwd with several position axes (time, height, width of images and
    video; splash_rope_axes): pair i turns by positions[axes[i]].  positions:
    int32 [axes, B, L], up to 4 axes; axes: bytes, one for each pair
    (rope_axis_map); the others as rope_fwd."""
    return _rope_axes(0, q, k, positions, table, axes, rot_offset, interleaved, q_out, k_out, stream)


def rope_axes_bwd(dq, dk, positions, table, axes, rot_offset: int = 0, interleaved: bool = False, dq_out=None,
                  dk_out=None, stream=None):
    """The gradients of rope_axes_fwd's inputs from those of its outputs (the
    transposed rotation); arguments as rope_axes_fwd."""
    return _rope_axes(1, dq, dk, positions, table, axes, rot_offset, interleaved, dq_out, dk_out, stream)


def paged_append_axes(k, v, k_cache, v_cache, block_table, positions, rot_positions, table, axes, q=None,
                      rot_offset: int = 0, interleaved: bool = False, seq_ids=None, k_scale=None, v_scale=None,
                      q_out=None, k_out=None, stream=None):
    """paged_append where a token's slot and its rotation are apart
    (splash_paged_append_axes): it is stored at positions [B, L] and turned by
    rot_positions (int32 [axes, B, L]) as in rope_axes_fwd.  With one axis
    (axes = rope_axis_map([rot_dim // 2])) this stores a tree of drafts: slots
    in a row, rotations by depth.  The others as paged_append."""
    return (_binding or _native()).paged_append_axes(k, v, k_cache, v_cache, block_table, positions, q, table, rot_offset,
                                                     interleaved, seq_ids, k_scale, v_scale, q_out, k_out,
                                                     _handle(stream), rot_positions, axes)


def paged_tree_decode(q, k_cache, v_cache, block_table, seq_lens, parents, scale: float, softcap: float = 0.0,
                      window_left: int = -1, k_scale=None, v_scale=None, out=None, lse=None, workspace=None, stream=None):
    """out [B, Hq, T, dv] bf16 and lse [B, Hq, T] fp32 of a tree of T (1 .. 64)
    drafted tokens of each sequence, whose keys and values are its newest T
    cached tokens (splash_paged_tree_decode).

    parents: int32 [B, T] or [T]: the earlier token of the tree that each
    continues, -1 for the context, below -1 for padding.  A token sees the
    context, its ancestors and itself.  q [B, Hq, T, dqk]; the others as
    paged_decode; the workspace is of paged_tree_decode_workspace_size(...)
    bytes."""
    return (_binding or _native()).paged_tree_decode(q, k_cache, v_cache, block_table, seq_lens, scale, softcap,
                                                     window_left, k_scale, v_scale, out, lse, workspace,
                                                     _handle(stream), parents)


def paged_tree_decode_workspace_size(q, k_cache, v_cache, block_table, window_left: int = -1) -> int:
    """Bytes of paged_tree_decode's workspace for tensors of these shapes and
    types (0 where it needs none)."""
    return _workspace_of("splash_paged_tree_decode_workspace_size", q, k_cache, v_cache, block_table, window_left)


def paged_compact(k_cache, v_cache, block_table, src, start, stream=None):
    """Moves tokens inside their sequences (splash_paged_compact): the one at
    position src[b, m] becomes the one at start[b] + m.  src: int32 [B, moves],
    ascending, src[b, m] >= start[b] + m, a negative entry ends a row's list;
    start: int32 [B].  Keeps the accepted branch of a tree of drafts (start =
    the context's length), or what an eviction leaves.  Caches and block_table
    as for paged_append (e4m3 without scales: values move as they are)."""
    (_binding or _native()).paged_compact(k_cache, v_cache, block_table, src, start, _handle(stream))


def paged_remap(block_table, parents, keep, room, refs, page_size: int, new_table=None, refs_out=None, copies=None,
                short=None, workspace=None, stream=None):
    """(new_table, refs_out, copies, short): forks, extends, truncates, frees
    and admits sequences (splash_paged_remap).

    Row i of the new table takes over the first keep[i] tokens of row
    parents[i] of block_table (int32 [rows, max_pages], unused entries -1;
    negative parent: none) and has pages for max(keep[i], room[i]) tokens.
    refs: int32 [pages], uses of each page (0: free).  Whole pages are shared;
    a page kept in part is copied unless the row alone has it.  copies: int32
    [new rows, 3], to be given to paged_copy for every layer's cache.  short:
    int32 [1], pages that were missing (then use none of the results)."""
    return (_binding or _native()).paged_remap(block_table, parents, keep, room, refs, page_size, new_table, refs_out,
                                               copies, short, workspace, _handle(stream))


def paged_remap_workspace_size(num_pages: int, new_rows: int) -> int:
    """Bytes of paged_remap's workspace."""
    n = ctypes.c_size_t(0)
    _check(lib().splash_paged_remap_workspace_size(int(num_pages), int(new_rows), ctypes.byref(n)),
           "splash_paged_remap_workspace_size")
    return int(n.value)


def paged_copy(k_cache, v_cache, copies, stream=None):
    """Copies rows between pages (splash_paged_copy): for each (source page,
    destination page, n) of copies, int32 [count, 3], the first n rows of every
    head.  Entries of -1 are skipped."""
    (_binding or _native()).paged_copy(k_cache, v_cache, copies, _handle(stream))


def last_device_error(stream=None) -> int:
    """Synchronises and returns (and clears) the device error status code."""
    return lib().splash_last_device_error(_stream(stream))


def check_device_error(stream=None):
    _check(last_device_error(stream), "device")


def debug_wait_selftest(timeout_ns: int, stream=None) -> int:
    return lib().splash_debug_wait_selftest(int(timeout_ns), _stream(stream))


def kernel_launches() -> int:
    """Kernels launched by the library in this process so far."""
    return int(lib().splash_kernel_launches())


def version() -> str:
    return lib().splash_version().decode()
