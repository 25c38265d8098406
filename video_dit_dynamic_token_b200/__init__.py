"""Dynamic block-sparse, low-precision self-attention for video DiTs on B200.

Thin Python binding over the C-ABI library ``liblx_sparse_attn.so`` (see
``include/lx_sparse_attn.h``).  Functions carry the C names; they only marshal
arguments: torch allocates device memory and supplies the current stream, and
every step of the computation runs in the library's CUDA kernels.  There is no
CPU fallback -- a missing library raises.

Entry points: the planner (lx_pool_means, lx_score_topk, lx_sparse_attn_plan),
the quantisers (lx_quantize_qk, lx_pool_quantize_qk, lx_quantize_v), the
attention (lx_attn_bf16, lx_attn_int8fp8, lx_sparse_attn_fwd), plan and
forward in one call (lx_sparse_attn), the fused Q/K prologue (lx_rope3d_table,
lx_qk_prologue), K smoothing (lx_k_channel_mean, lx_quantize_qk_smooth,
lx_pool_quantize_qk_smooth), NVFP4 (lx_nvfp4_quantize, lx_nvfp4_gemm, and
lx_nvfp4_gemv for few bf16 rows), dense attention over packed sequences
(lx_attn_packed: prompts, cross-attention, single tokens over a cache) and
behind a shared prefix (lx_attn_prefix); the host-to-host pipeline is in
``pipeline`` and the Light-Ulysses exchange in ``ulysses``.
"""
from __future__ import annotations

import ctypes
import math
import struct
from dataclasses import dataclass
from functools import lru_cache

import torch

from . import _abi
from ._abi import LX_BLOCK, LX_MODE_BF16, LX_MODE_INT8FP8, LxBhld, LxPack, LxPlan  # noqa: F401

MODES = {"bf16": LX_MODE_BF16, "int8fp8": LX_MODE_INT8FP8}


class LxError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _abi.load()
        super().__init__(f"{where}: {lib.lx_status_string(status).decode()} (status {status})")
        self.status = status


def _check(status: int, where: str):
    if status != 0:
        raise LxError(status, where)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


_pack_bhld = struct.Struct("P7q").pack


def bhld(t: torch.Tensor) -> LxBhld:
    """View of a bf16 [B,H,L,D] CUDA tensor whose last dim is contiguous."""
    strides = t.stride()
    if t.dtype is not torch.bfloat16 or len(strides) != 4 or strides[3] != 1:
        raise ValueError("expected a bf16 [B,H,L,D] tensor with contiguous D")
    # packed in one go, which takes half the time of eight ctypes fields
    return LxBhld.from_buffer_copy(_pack_bhld(t.data_ptr(), *t.shape, *strides[:3]))


@dataclass
class Plan:
    """Kept-block plan: idx int32 [B,H,nB,k] ascending, mask uint32-bits [B,H,nB,W]."""
    idx: torch.Tensor
    mask: torch.Tensor | None
    B: int
    H: int
    L: int
    nB: int
    k: int

    def c(self) -> LxPlan:
        return LxPlan(self.idx.data_ptr(), self.mask.data_ptr() if self.mask is not None else None,
                      self.B, self.H, self.L, self.nB, self.k, LX_BLOCK)


def lx_plan_size(B, H, L, D, keep):
    lib = _abi.load()
    k = ctypes.c_int64()
    ib, mb, wb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.lx_plan_size(B, H, L, D, float(keep), ctypes.byref(k), ctypes.byref(ib), ctypes.byref(mb),
                            ctypes.byref(wb)), "lx_plan_size")
    return k.value, ib.value, mb.value, wb.value


def empty_plan(B, H, L, D, keep, device, with_mask=True) -> Plan:
    k, _, _, _ = lx_plan_size(B, H, L, D, keep)
    nB = (L + LX_BLOCK - 1) // LX_BLOCK
    idx = torch.empty((B, H, nB, k), dtype=torch.int32, device=device)
    mask = torch.empty((B, H, nB, (nB + 31) // 32), dtype=torch.int32, device=device) if with_mask else None
    return Plan(idx, mask, B, H, L, nB, k)


def lx_pool_means(Q, K, out=None, stream=None):
    lib = _abi.load()
    B, H, L, D = Q.shape
    nB = (L + LX_BLOCK - 1) // LX_BLOCK
    if out is None:
        out = (torch.empty((B, H, nB, D), dtype=torch.float32, device=Q.device),
               torch.empty((B, H, nB, D), dtype=torch.float32, device=Q.device))
    q, k = bhld(Q), bhld(K)
    _check(lib.lx_pool_means(ctypes.byref(q), ctypes.byref(k), _ptr(out[0]), _ptr(out[1]), _stream(stream)),
           "lx_pool_means")
    return out


def score_ws_bytes(B, H, nB) -> int:
    """Scratch of lx_score_topk: the fp32 [B,H,nB,ldS] score matrix (ldS = nB
    rounded up to 32), 256-byte rounded."""
    ldS = (nB + 31) // 32 * 32
    return (4 * B * H * nB * ldS + 255) // 256 * 256


def lx_score_topk(mq, mk, L, keep, plan: Plan | None = None, ws=None, stream=None) -> Plan:
    lib = _abi.load()
    B, H, nB, D = mq.shape
    if plan is None:
        plan = empty_plan(B, H, L, D, keep, mq.device)
    if ws is None:
        ws = torch.empty(score_ws_bytes(B, H, nB), dtype=torch.uint8, device=mq.device)
    cp = plan.c()
    _check(lib.lx_score_topk(_ptr(mq), _ptr(mk), B, H, L, D, float(keep), ctypes.byref(cp), _ptr(ws), ws.numel(),
                             _stream(stream)), "lx_score_topk")
    return plan


def lx_sparse_attn_plan(Q, K, keep, plan: Plan | None = None, ws=None, stream=None, with_mask=True) -> Plan:
    lib = _abi.load()
    B, H, L, D = Q.shape
    _, _, _, wb = lx_plan_size(B, H, L, D, keep)
    if plan is None:
        plan = empty_plan(B, H, L, D, keep, Q.device, with_mask)
    if ws is None:
        ws = torch.empty(wb, dtype=torch.uint8, device=Q.device)
    q, k, cp = bhld(Q), bhld(K), plan.c()
    _check(lib.lx_sparse_attn_plan(ctypes.byref(q), ctypes.byref(k), float(keep), ctypes.byref(cp), _ptr(ws),
                                   ws.numel(), _stream(stream)), "lx_sparse_attn_plan")
    return plan


def lx_quantize_qk(Q, K, out=None, stream=None):
    lib = _abi.load()
    B, H, L, D = Q.shape
    nB = (L + LX_BLOCK - 1) // LX_BLOCK
    if out is None:
        dev = Q.device
        out = (torch.empty((B, H, L, D), dtype=torch.int8, device=dev),
               torch.empty((B, H, nB), dtype=torch.float32, device=dev),
               torch.empty((B, H, L, D), dtype=torch.int8, device=dev),
               torch.empty((B, H, nB), dtype=torch.float32, device=dev))
    qc, qs, kc, ks = out
    q, k = bhld(Q), bhld(K)
    _check(lib.lx_quantize_qk(ctypes.byref(q), ctypes.byref(k), _ptr(qc), _ptr(qs), _ptr(kc), _ptr(ks),
                              _stream(stream)), "lx_quantize_qk")
    return out


def lx_pool_quantize_qk(Q, K, out=None, stream=None):
    """Block means and INT8 codes of Q and K in one pass: (mq, mk, qc, qs, kc, ks)."""
    lib = _abi.load()
    B, H, L, D = Q.shape
    nB = (L + LX_BLOCK - 1) // LX_BLOCK
    if out is None:
        dev = Q.device
        out = (torch.empty((B, H, nB, D), dtype=torch.float32, device=dev),
               torch.empty((B, H, nB, D), dtype=torch.float32, device=dev),
               torch.empty((B, H, L, D), dtype=torch.int8, device=dev),
               torch.empty((B, H, nB), dtype=torch.float32, device=dev),
               torch.empty((B, H, L, D), dtype=torch.int8, device=dev),
               torch.empty((B, H, nB), dtype=torch.float32, device=dev))
    mq, mk, qc, qs, kc, ks = out
    q, k = bhld(Q), bhld(K)
    _check(lib.lx_pool_quantize_qk(ctypes.byref(q), ctypes.byref(k), _ptr(mq), _ptr(mk), _ptr(qc), _ptr(qs), _ptr(kc),
                                   _ptr(ks), _stream(stream)), "lx_pool_quantize_qk")
    return out


def rope3d_default_split(D):
    """The default (t, h, w) channel split of a head dimension D."""
    q = D // 6
    return D - 4 * q, 2 * q, 2 * q


def _rope(grid, D, theta, split):
    dt, dh, dw = rope3d_default_split(D) if split is None else split
    T, Hh, W = grid
    return _abi.LxRope3d(T, Hh, W, dt, dh, dw, float(theta))


def lx_rope3d_table(grid, D, theta=10000.0, split=None, device="cuda", stream=None):
    """The (cos, sin) table of the 3D RoPE of a (T, Hh, W) grid, fp32 on the device."""
    lib = _abi.load()
    r = _rope(grid, D, theta, split)
    n = ctypes.c_size_t()
    _check(lib.lx_rope3d_table_size(ctypes.byref(r), D, ctypes.byref(n)), "lx_rope3d_table_size")
    table = torch.empty(max(n.value // 4, 4), dtype=torch.float32, device=device)
    _check(lib.lx_rope3d_table(ctypes.byref(r), D, _ptr(table), _stream(stream)), "lx_rope3d_table")
    return table


def lx_qk_prologue(Q, K, wq, wk, eps, grid, theta=10000.0, split=None, table=None, with_y=True, with_codes=True,
                   stream=None):
    """Per-head RMSNorm + 3D RoPE of Q and K, with the block means and INT8 codes
    of the bf16 result, in one pass: dict(Yq, Yk, mq, mk, qc, qs, kc, ks)."""
    B, H, L, D = Q.shape
    nB = (L + LX_BLOCK - 1) // LX_BLOCK
    dev = Q.device
    if table is None:
        table = lx_rope3d_table(grid, D, theta, split, dev, stream)
    out = {"mq": torch.empty((B, H, nB, D), dtype=torch.float32, device=dev),
           "mk": torch.empty((B, H, nB, D), dtype=torch.float32, device=dev)}
    if with_y:
        out["Yq"] = torch.empty((B, H, L, D), dtype=torch.bfloat16, device=dev)
        out["Yk"] = torch.empty((B, H, L, D), dtype=torch.bfloat16, device=dev)
    if with_codes:
        out["qc"] = torch.empty((B, H, L, D), dtype=torch.int8, device=dev)
        out["qs"] = torch.empty((B, H, nB), dtype=torch.float32, device=dev)
        out["kc"] = torch.empty((B, H, L, D), dtype=torch.int8, device=dev)
        out["ks"] = torch.empty((B, H, nB), dtype=torch.float32, device=dev)
    lx_qk_prologue_into(Q, K, wq, wk, eps, grid, table, out["mq"], out["mk"], out.get("qc"), out.get("qs"),
                        out.get("kc"), out.get("ks"), out.get("Yq"), out.get("Yk"), theta, split, stream)
    return out


def lx_qk_prologue_into(Q, K, wq, wk, eps, grid, table, mq, mk, qc=None, qs=None, kc=None, ks=None, Yq=None, Yk=None,
                        theta=10000.0, split=None, stream=None):
    """lx_qk_prologue into caller buffers (no allocation): means, optional codes
    and optional bf16 outputs."""
    lib = _abi.load()
    D = Q.shape[-1]
    r = _rope(grid, D, theta, split)
    q, k = bhld(Q), bhld(K)
    yq = bhld(Yq) if Yq is not None else None
    yk = bhld(Yk) if Yk is not None else None
    _check(lib.lx_qk_prologue(ctypes.byref(q), ctypes.byref(k), _ptr(wq), _ptr(wk), float(eps), ctypes.byref(r),
                              _ptr(table), ctypes.byref(yq) if yq is not None else None,
                              ctypes.byref(yk) if yk is not None else None, _ptr(mq), _ptr(mk), _ptr(qc), _ptr(qs),
                              _ptr(kc), _ptr(ks), _stream(stream)), "lx_qk_prologue")


def lx_k_channel_mean(K, out=None, ws=None, stream=None):
    """Per-(b, h, channel) mean of K over all tokens (fp64 sums, fp32 result) [B,H,D]."""
    lib = _abi.load()
    B, H, L, D = K.shape
    k = bhld(K)
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.float32, device=K.device)
    if ws is None:
        n = ctypes.c_size_t()
        _check(lib.lx_k_channel_mean_ws_size(ctypes.byref(k), ctypes.byref(n)), "lx_k_channel_mean_ws_size")
        ws = torch.empty(max(n.value, 16), dtype=torch.uint8, device=K.device)
    _check(lib.lx_k_channel_mean(ctypes.byref(k), _ptr(ws), ws.numel(), _ptr(out), _stream(stream)),
           "lx_k_channel_mean")
    return out


def lx_quantize_qk_smooth(Q, K, km=None, out=None, stream=None):
    """INT8 codes of Q and of K minus its channel means: (qc, qs, kc, ks, km)."""
    lib = _abi.load()
    B, H, L, D = Q.shape
    nB = (L + LX_BLOCK - 1) // LX_BLOCK
    if km is None:
        km = lx_k_channel_mean(K, stream=stream)
    if out is None:
        dev = Q.device
        out = (torch.empty((B, H, L, D), dtype=torch.int8, device=dev),
               torch.empty((B, H, nB), dtype=torch.float32, device=dev),
               torch.empty((B, H, L, D), dtype=torch.int8, device=dev),
               torch.empty((B, H, nB), dtype=torch.float32, device=dev))
    qc, qs, kc, ks = out
    q, k = bhld(Q), bhld(K)
    _check(lib.lx_quantize_qk_smooth(ctypes.byref(q), ctypes.byref(k), _ptr(km), _ptr(qc), _ptr(qs), _ptr(kc),
                                     _ptr(ks), _stream(stream)), "lx_quantize_qk_smooth")
    return qc, qs, kc, ks, km


def lx_pool_quantize_qk_smooth(Q, K, km, out, stream=None):
    """Block means of Q and K and INT8 codes of Q and K - km, into out = (mq, mk, qc, qs, kc, ks)."""
    lib = _abi.load()
    mq, mk, qc, qs, kc, ks = out
    q, k = bhld(Q), bhld(K)
    _check(lib.lx_pool_quantize_qk_smooth(ctypes.byref(q), ctypes.byref(k), _ptr(km), _ptr(mq), _ptr(mk), _ptr(qc),
                                          _ptr(qs), _ptr(kc), _ptr(ks), _stream(stream)), "lx_pool_quantize_qk_smooth")
    return out


def lx_quantize_v(V, out=None, amax_ws=None, stream=None):
    lib = _abi.load()
    B, H, L, D = V.shape
    if out is None:
        out = (torch.empty((B, H, L, D), dtype=torch.uint8, device=V.device),
               torch.empty((B, H, D), dtype=torch.float32, device=V.device))
    if amax_ws is None:
        amax_ws = torch.empty((B, H, D), dtype=torch.int32, device=V.device)
    v = bhld(V)
    _check(lib.lx_quantize_v(ctypes.byref(v), _ptr(out[0]), _ptr(out[1]), _ptr(amax_ws), _stream(stream)),
           "lx_quantize_v")
    return out


def lx_quantize_v_noalloc(V, out=None, stream=None):
    lib = _abi.load()
    B, H, L, D = V.shape
    if out is None:
        out = (torch.empty((B, H, L, D), dtype=torch.uint8, device=V.device),
               torch.empty((B, H, D), dtype=torch.float32, device=V.device))
    v = bhld(V)
    _check(lib.lx_quantize_v_noalloc(ctypes.byref(v), _ptr(out[0]), _ptr(out[1]), _stream(stream)),
           "lx_quantize_v_noalloc")
    return out


def lx_attn_bf16(Q, K, V, plan: Plan, out=None, stream=None):
    lib = _abi.load()
    if out is None:
        out = torch.empty_like(Q)
    q, k, v, o, cp = bhld(Q), bhld(K), bhld(V), bhld(out), plan.c()
    _check(lib.lx_attn_bf16(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), ctypes.byref(cp), ctypes.byref(o),
                            _stream(stream)), "lx_attn_bf16")
    return out


def lx_attn_int8fp8(qc, qs, kc, ks, vc, vs, plan: Plan, out=None, stream=None):
    lib = _abi.load()
    if out is None:
        out = torch.empty(qc.shape, dtype=torch.bfloat16, device=qc.device)
    o, cp = bhld(out), plan.c()
    _check(lib.lx_attn_int8fp8(_ptr(qc), _ptr(qs), _ptr(kc), _ptr(ks), _ptr(vc), _ptr(vs), ctypes.byref(cp),
                               ctypes.byref(o), _stream(stream)), "lx_attn_int8fp8")
    return out


def lx_fwd_workspace_size(Q, mode) -> int:
    lib = _abi.load()
    n = ctypes.c_size_t()
    q = bhld(Q)
    _check(lib.lx_fwd_workspace_size(ctypes.byref(q), MODES[mode], ctypes.byref(n)), "lx_fwd_workspace_size")
    return n.value


def lx_sparse_attn_fwd(Q, K, V, plan: Plan, mode="int8fp8", out=None, ws=None, stream=None):
    lib = _abi.load()
    if out is None:
        out = torch.empty_like(Q)
    if ws is None:
        n = lx_fwd_workspace_size(Q, mode)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=Q.device)
    q, k, v, o, cp = bhld(Q), bhld(K), bhld(V), bhld(out), plan.c()
    _check(lib.lx_sparse_attn_fwd(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), ctypes.byref(cp), MODES[mode],
                                  ctypes.byref(o), _ptr(ws), ws.numel(), _stream(stream)), "lx_sparse_attn_fwd")
    return out


def lx_sparse_attn_ws_size(Q, keep, mode="int8fp8") -> int:
    lib = _abi.load()
    n = ctypes.c_size_t()
    q = bhld(Q)
    _check(lib.lx_sparse_attn_ws_size(ctypes.byref(q), float(keep), MODES[mode], ctypes.byref(n)),
           "lx_sparse_attn_ws_size")
    return n.value


def lx_sparse_attn(Q, K, V, keep, mode="int8fp8", plan: Plan | None = None, out=None, ws=None, stream=None):
    """Plan and forward in one call (Q and K read once for means and codes): (O, plan)."""
    lib = _abi.load()
    B, H, L, D = Q.shape
    if plan is None:
        plan = empty_plan(B, H, L, D, keep, Q.device)
    if out is None:
        out = torch.empty_like(Q)
    if ws is None:
        ws = torch.empty(max(lx_sparse_attn_ws_size(Q, keep, mode), 256), dtype=torch.uint8, device=Q.device)
    q, k, v, o, cp = bhld(Q), bhld(K), bhld(V), bhld(out), plan.c()
    _check(lib.lx_sparse_attn(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), float(keep), MODES[mode],
                              ctypes.byref(cp), ctypes.byref(o), _ptr(ws), ws.numel(), _stream(stream)),
           "lx_sparse_attn")
    return out, plan


# ---------------------------------------------------------------- packed sequences
# These calls serve single tokens, where marshalling counts: sizes of workspaces are
# kept per shape, and the stream is asked for by device.  (The public forms of the two functions take
# longer; a torch build without CUDA has only them, and the sizes and checks work there too.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _with_stream(stream, t, call):
    """call() with `stream` as the current one: what is allocated there belongs to the stream that uses it."""
    if t.get_device() != stream.device_index:
        raise ValueError("the stream is on another device than the tensors")
    with torch.cuda.stream(stream):
        return call()


def _same_device(tensors, optional=()):
    """The device index of CUDA tensors that are all on one device (those that are None are skipped)."""
    d = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != d:
            raise ValueError("tensors are on different devices")
    for t in optional:
        if t is not None and t.get_device() != d:
            raise ValueError("tensors are on different devices")
    if d < 0:
        raise ValueError("expected CUDA tensors")
    return d


def _shape_only(H, L, D):
    return LxBhld(4096, 1, H, L, D, 8, D, H * D)


@lru_cache(maxsize=4096)
def _packed_ws(Hq, Tq, Hkv, Tk, D, n) -> int:
    b = ctypes.c_size_t()
    q, k = _shape_only(Hq, Tq, D), _shape_only(Hkv, Tk, D)
    _check(_abi.load().lx_attn_packed_ws_size(ctypes.byref(q), ctypes.byref(k), n, ctypes.byref(b)),
           "lx_attn_packed_ws_size")
    return b.value


@lru_cache(maxsize=4096)
def _prefix_ws(Hq, Tq, D) -> int:
    b = ctypes.c_size_t()
    q = _shape_only(Hq, Tq, D)
    _check(_abi.load().lx_attn_prefix_ws_size(ctypes.byref(q), ctypes.byref(b)), "lx_attn_prefix_ws_size")
    return b.value


def lx_attn_packed_ws_size(Q, K, n) -> int:
    return _packed_ws(Q.shape[1], Q.shape[2], K.shape[1], K.shape[2], Q.shape[3], int(n))


def lx_attn_prefix_ws_size(Q) -> int:
    return _prefix_ws(Q.shape[1], Q.shape[2], Q.shape[3])


def _attn_packed(prefix, Q, K, V, cu_q, cu_k, causal, scale, len_k, out, lse, ws, stream):
    if stream is not None:
        return _with_stream(stream, Q, lambda: _attn_packed(prefix, Q, K, V, cu_q, cu_k, causal, scale, len_k, out,
                                                            lse, ws, None))
    if out is None:
        out = torch.empty_like(Q)
    dev = _same_device((Q, K, V, out, cu_q, cu_k), (len_k, lse, ws, *prefix))
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _attn_packed(prefix, Q, K, V, cu_q, cu_k, causal, scale, len_k, out, lse, ws, None)
    starts = cu_q.shape
    n = starts[0] - 1 if len(starts) == 1 else -1
    if (cu_k.shape != starts or cu_q.dtype is not torch.int32 or cu_k.dtype is not torch.int32 or n < 0
            or not cu_q.is_contiguous() or not cu_k.is_contiguous()
            or len_k is not None and (len_k.dtype is not torch.int32 or len_k.shape != (n,) or not len_k.is_contiguous())):
        raise ValueError("cu_q and cu_k: contiguous int32 tensors of n + 1 entries, len_k of n")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != Q.shape[1:3] or not lse.is_contiguous()):
        raise ValueError("lse: a contiguous fp32 [Hq, Tq] tensor")
    q, k, v, o = bhld(Q), bhld(K), bhld(V), bhld(out)
    D = q.D
    if ws is None:
        size = _prefix_ws(q.H, q.L, D) if prefix else _packed_ws(q.H, q.L, k.H, k.L, D, n)
        if size:
            ws = Q.new_empty(size, dtype=torch.uint8)
    pk = LxPack(cu_q.data_ptr(), cu_k.data_ptr(), None if len_k is None else len_k.data_ptr(), n)
    tail = (k, v, pk, 1 if causal else 0, D ** -0.5 if scale is None else scale, o,
            None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel() * ws.element_size(), _raw_stream(dev))
    if prefix:   # (ctypes passes a structure's address where a pointer to it is declared)
        status = _abi.load().lx_attn_prefix(q, bhld(prefix[0]), bhld(prefix[1]), *tail)
    else:
        status = _abi.load().lx_attn_packed(q, *tail)
    if status:
        _check(status, "lx_attn_prefix" if prefix else "lx_attn_packed")
    return out


def lx_attn_packed(Q, K, V, cu_q, cu_k, causal=True, scale=None, len_k=None, out=None, lse=None, ws=None,
                   stream=None):
    """Attention over packed sequences of different lengths, causal or full, with grouped heads.

    Q: bf16 [1, Hq, Tq, D]; K, V: [1, Hkv, Tk, D]; cu_q, cu_k: int32 [n + 1] starts and ends; len_k: int32 [n]
    keys in use (caches).  scale None: 1 / sqrt(D).  lse: fp32 [Hq, Tq] to be filled, or None.  Rows outside
    [cu_q[0], cu_q[n]) of `out` and `lse` are left as they were.  Returns out."""
    return _attn_packed((), Q, K, V, cu_q, cu_k, causal, scale, len_k, out, lse, ws, stream)


def lx_attn_prefix(Q, Kp, Vp, K, V, cu_q, cu_k, causal=True, scale=None, len_k=None, out=None, lse=None, ws=None,
                   stream=None):
    """lx_attn_packed for a batch whose rows all see the keys Kp, Vp [1, Hkv, Lp, D] before their own."""
    return _attn_packed((Kp, Vp), Q, K, V, cu_q, cu_k, causal, scale, len_k, out, lse, ws, stream)


# ---------------------------------------------------------------- NVFP4
@dataclass
class NvFp4Tensor:
    """An NVFP4 tensor [R, K] in the layouts of lx_nvfp4_quantize: codes uint8
    [R, K/2], tiled E4M3 scales (uint8, rows padded to 128), fp32 global scale [1]."""
    codes: torch.Tensor
    sf: torch.Tensor
    gscale: torch.Tensor
    R: int
    K: int


def lx_nvfp4_sizes(R, K):
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_abi.load().lx_nvfp4_sizes(int(R), int(K), ctypes.byref(cb), ctypes.byref(sb)), "lx_nvfp4_sizes")
    return cb.value, sb.value


def lx_nvfp4_quantize(x, gscale=None, out: NvFp4Tensor | None = None, stream=None) -> NvFp4Tensor:
    """x: bf16 [R, K] CUDA tensor with contiguous rows.  gscale None: the global
    scale is computed from x; else a CUDA fp32 tensor of one element used as given."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("expected a bf16 [R, K] tensor with contiguous rows")
    R, K = x.shape
    if out is None:
        cb, sb = lx_nvfp4_sizes(R, K)
        g = torch.empty(1, dtype=torch.float32, device=x.device)
        out = NvFp4Tensor(torch.empty((R, K // 2), dtype=torch.uint8, device=x.device),
                          torch.empty(sb, dtype=torch.uint8, device=x.device), g, R, K)
    compute = gscale is None
    if not compute:
        out.gscale.copy_(gscale.reshape(1))
    _check(_abi.load().lx_nvfp4_quantize(_ptr(x), R, K, x.stride(0), int(compute), _ptr(out.gscale), _ptr(out.codes),
                                         _ptr(out.sf), _stream(stream)), "lx_nvfp4_quantize")
    return out


def lx_nvfp4_gemm(xq: NvFp4Tensor, wq: NvFp4Tensor, bias=None, out=None, stream=None):
    """Y = X W^T + bias in bf16 [M, N] from NVFP4 X [M, K] and W [N, K]; bias fp32 [N] or None."""
    if xq.K != wq.K:
        raise ValueError("X and W differ in K")
    M, N, K = xq.R, wq.R, xq.K
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=xq.codes.device)
    if bias is not None and (bias.dtype != torch.float32 or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous fp32 tensor")
    _check(_abi.load().lx_nvfp4_gemm(_ptr(xq.codes), _ptr(xq.sf), _ptr(xq.gscale), _ptr(wq.codes), _ptr(wq.sf),
                                     _ptr(wq.gscale), _ptr(bias), M, N, K, _ptr(out), out.stride(0), _stream(stream)),
           "lx_nvfp4_gemm")
    return out


@lru_cache(maxsize=4096)
def lx_nvfp4_gemv_ws_size(M, N, K) -> int:
    b = ctypes.c_size_t()
    _check(_abi.load().lx_nvfp4_gemv_ws_size(int(M), int(N), int(K), ctypes.byref(b)), "lx_nvfp4_gemv_ws_size")
    return b.value


def lx_nvfp4_gemv(x, wq: NvFp4Tensor, bias=None, out=None, ws=None, stream=None):
    """Y = x W^T + bias in bf16 [M, N] for M <= 16 bf16 rows x [M, K] and NVFP4 W [N, K]; bias fp32 [N] or None.

    `out` overlaps neither x nor the weights."""
    if stream is not None:
        return _with_stream(stream, x, lambda: lx_nvfp4_gemv(x, wq, bias, out, ws))
    strides = x.stride()
    if x.dtype is not torch.bfloat16 or len(strides) != 2 or strides[1] != 1:
        raise ValueError("expected a bf16 [M, K] tensor with contiguous rows")
    M, K = x.shape
    N, codes, sf, gw = wq.R, wq.codes, wq.sf, wq.gscale
    if K != wq.K:
        raise ValueError("x and W differ in K")
    if (codes.numel() * 2 != N * K or sf.numel() < (N + 127) // 128 * 8 * K or codes.element_size() != 1
            or sf.element_size() != 1 or not codes.is_contiguous() or not sf.is_contiguous()
            or gw.dtype is not torch.float32 or gw.numel() != 1):
        raise ValueError("W: not the codes, scales and global scale of an [N, K] tensor")
    if bias is not None and (bias.dtype is not torch.float32 or not bias.is_contiguous() or bias.numel() != N):
        raise ValueError("bias must be a contiguous fp32 tensor of N elements")
    dev = _same_device((x, codes, sf, gw), (bias, out, ws))
    if dev != _current_device():
        with torch.cuda.device(dev):
            return lx_nvfp4_gemv(x, wq, bias, out, ws)
    if out is None:
        out = x.new_empty((M, N))
        ldy = N
    elif out.dtype is torch.bfloat16 and out.shape == (M, N) and out.stride(1) == 1:
        ldy = out.stride(0) if M > 1 else N
    else:
        raise ValueError("out must be a bf16 [M, N] tensor with contiguous rows")
    if ws is None:
        size = lx_nvfp4_gemv_ws_size(M, N, K)
        if size:
            ws = x.new_empty(size, dtype=torch.uint8)
    status = _abi.load().lx_nvfp4_gemv(
        x.data_ptr(), M, strides[0] if M > 1 else K, codes.data_ptr(), sf.data_ptr(), gw.data_ptr(),
        None if bias is None else bias.data_ptr(), N, K, out.data_ptr(), ldy,
        None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size(), _raw_stream(dev))
    if status:
        _check(status, "lx_nvfp4_gemv")
    return out


def nvfp4_gemm_flops(M, N, K) -> float:
    return 2.0 * M * N * K


def lx_last_device_status(stream=None) -> int:
    return _abi.load().lx_last_device_status(_stream(stream))


def lx_debug_wait_timeout(limit_ns: int, stream=None):
    _check(_abi.load().lx_debug_wait_timeout(int(limit_ns), _stream(stream)), "lx_debug_wait_timeout")


def keep_count(nB: int, keep: float) -> int:
    """k for a plan, from the library's own size query (nB blocks of 64)."""
    return lx_plan_size(1, 1, nB * LX_BLOCK, 64, keep)[0]


def effective_flops(B, H, L, D, keep) -> float:
    """4 L^2 D H B * k/nB: the attention work on the kept tiles only."""
    nB = math.ceil(L / LX_BLOCK)
    k = keep_count(nB, keep)
    return 4.0 * L * L * D * H * B * k / nB
