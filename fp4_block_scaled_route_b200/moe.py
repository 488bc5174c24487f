"""Thin ctypes binding of ``libmoe.so`` (include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  The entry points keep the C names (``moe_create``, ``moe_forward``
...).  :class:`MoeLayer` wraps a context for torch tensors: it passes
``data_ptr()`` values and the current CUDA stream handle, nothing else.

There is no fallback: if the library is missing, or a call fails, this module
raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_CUDA = 3
MOE_ERR_NO_MEMORY = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_BAD_ROUTING = 6

MOE_DT_BF16 = 0
MOE_DT_FP16 = 1
MOE_DT_FP32 = 2

MOE_WFMT_FP8_E4M3_B128 = 0
MOE_WFMT_MXFP4_E2M1_E8M0_K32 = 1
MOE_WFMT_NVFP4_E2M1_E4M3_K16 = 2
MOE_WFMT_MXFP4_W4A4 = 3
MOE_WFMT_MXFP8_E4M3_E8M0_K32 = 4

# Every entry point declared in include/moe.h: name -> (restype, argtypes)
_vp = ctypes.c_void_p
_i = ctypes.c_int
_ll = ctypes.c_longlong
SIGNATURES = {
    "moe_create": (_i, [_i, _i, _i, _i, _i, ctypes.POINTER(_vp)]),
    "moe_create_ex": (_i, [_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_vp)]),
    "moe_destroy": (None, [_vp]),
    "moe_forward": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_forward_nvfp4": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_forward_partial": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_finalize_bf16": (_i, [_vp, _vp, ctypes.c_longlong, _vp]),
    "moe_pack_mxfp4_scales": (_i, [_vp, _vp, _i, _i, _vp]),
    "moe_pack_nvfp4_scales": (_i, [_vp, _vp, _i, _i, _vp]),
    "moe_declare_packed_scales": (_i, [_vp, ctypes.c_longlong, _i]),
    "moe_get_routing": (_i, [_vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_get_activations": (_i, [_vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_get_block_scales": (_i, [_vp, _vp, _vp, _vp]),
    "moe_get_device_status": (_i, [_vp, _vp]),
    "moe_last_config": (_i, [_vp, ctypes.POINTER(_i), ctypes.POINTER(_i)]),
    "moe_set_fault_injection": (_i, [_vp, _i]),
    "moe_profile_enable": (_i, [_vp, _i]),
    "moe_profile_read": (_i, [_vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(_i)]),
    "moe_forward_noalloc": (_i, [_i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_router_topk": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp]),
    "moe_set_green_ctx": (_i, [_vp, _i]),
    "moe_green_ctx_sms": (_i, [_vp, ctypes.POINTER(_i), ctypes.POINTER(_i)]),
    "moe_set_dispatch_overlap": (_i, [_vp, _i]),
    "moe_dispatch_overlap_ctas": (_i, [_vp, ctypes.POINTER(_i)]),
    "moe_route": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_permute": (_i, [_i, _i, _i, _i, _i, _vp, _ll, _vp, _vp, _ll, _vp]),
    "moe_combine": (_i, [_i, _i, _i, _i, _i, _i, _vp, _ll, _vp, _vp, _vp, _ll, _vp]),
    "moe_combine_backward": (_i, [_i, _i, _i, _i, _i, _i, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _ll, _vp, _vp]),
    "moe_grouped_gemm": (_i, [_i, _i, _i, _i, _i, _i, _vp, _vp, _ll, _vp, _ll, _ll, _vp, _ll, _vp, _vp]),
    "moe_grouped_gemm_dgrad": (_i, [_i, _i, _i, _i, _i, _i, _vp, _vp, _ll, _vp, _ll, _ll, _vp, _ll, _vp, _vp]),
    "moe_grouped_gemm_wgrad": (_i, [_i, _i, _i, _i, _i, _i, _vp, _vp, _ll, _vp, _ll, _vp, _vp, _vp]),
    "moe_quant_int8": (_i, [_i, _i, _i, _i, _i, _vp, _ll, _vp, _vp, _ll, _vp, _vp]),
    "moe_int8_gemm": (_i, [_i, _i, _i, _i, _i, _vp, _vp, _ll, _vp, _vp, _ll, _ll, _vp, _vp, _ll, _vp, _vp]),
    "moe_ops_status": (_i, [_vp]),
    "moe_status_string": (ctypes.c_char_p, [_i]),
}

_lib: Optional[ctypes.CDLL] = None


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built by ``python -m fp4_block_scaled_route_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m fp4_block_scaled_route_b200.build` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where)


# ---- C entry points under their own names --------------------------------
def moe_create(H, I, E, k, wfmt):
    ctx = _vp()
    _check(lib().moe_create(H, I, E, k, wfmt, ctypes.byref(ctx)), "moe_create")
    return ctx


def moe_create_ex(H, I, E, k, wfmt, max_T, n_shared):
    ctx = _vp()
    _check(lib().moe_create_ex(H, I, E, k, wfmt, max_T, n_shared, ctypes.byref(ctx)), "moe_create_ex")
    return ctx


def moe_destroy(ctx) -> None:
    lib().moe_destroy(ctx)


def moe_forward(ctx, T, x, topk_ids, topk_w, w13, s13, w2, s2, out, stream) -> int:
    return lib().moe_forward(ctx, T, x, topk_ids, topk_w, w13, s13, w2, s2, out, stream)


def moe_forward_nvfp4(ctx, T, x, topk_ids, topk_w, w13, s13, g13, w2, s2, g2, out, stream) -> int:
    return lib().moe_forward_nvfp4(ctx, T, x, topk_ids, topk_w, w13, s13, g13, w2, s2, g2, out, stream)


def moe_forward_partial(ctx, T, x, topk_ids, topk_w, w13, s13, g13, w2, s2, g2, out_f32, stream) -> int:
    return lib().moe_forward_partial(ctx, T, x, topk_ids, topk_w, w13, s13, g13, w2, s2, g2, out_f32, stream)


def moe_finalize_bf16(inp, out, n, stream) -> int:
    return lib().moe_finalize_bf16(inp, out, n, stream)


def moe_forward_noalloc(H, I, E, k, wfmt, n_shared, T, x, topk_ids, topk_w, w13, s13, w2, s2, out, d_status,
                        stream) -> int:
    return lib().moe_forward_noalloc(H, I, E, k, wfmt, n_shared, T, x, topk_ids, topk_w, w13, s13, w2, s2, out,
                                     d_status, stream)


def moe_pack_mxfp4_scales(src, dst, rows, K, stream) -> int:
    return lib().moe_pack_mxfp4_scales(src, dst, rows, K, stream)


def moe_pack_nvfp4_scales(src, dst, rows, K, stream) -> int:
    return lib().moe_pack_nvfp4_scales(src, dst, rows, K, stream)


def moe_declare_packed_scales(p, nbytes, wfmt) -> int:
    return lib().moe_declare_packed_scales(p, nbytes, wfmt)


def moe_get_block_scales(ctx, xsc, hsc, stream) -> int:
    return lib().moe_get_block_scales(ctx, xsc, hsc, stream)


def moe_get_routing(ctx, counts, offsets, perm, inv, stream) -> int:
    return lib().moe_get_routing(ctx, counts, offsets, perm, inv, stream)


def moe_get_activations(ctx, xq, xs, hq, hs, stream) -> int:
    return lib().moe_get_activations(ctx, xq, xs, hq, hs, stream)


def moe_get_device_status(ctx, stream) -> int:
    return lib().moe_get_device_status(ctx, stream)


def moe_last_config(ctx):
    bn, grid = _i(), _i()
    _check(lib().moe_last_config(ctx, ctypes.byref(bn), ctypes.byref(grid)), "moe_last_config")
    return bn.value, grid.value


MOE_NUM_STAGES = 5
STAGE_NAMES = ("route", "quant", "gemm1_swiglu_requant", "gemm2_combine", "finalize")


def moe_set_fault_injection(ctx, mode) -> int:
    return lib().moe_set_fault_injection(ctx, mode)


def moe_router_topk(ctx, T, x, wr, topk_ids, topk_w, stream) -> int:
    return lib().moe_router_topk(ctx, T, x, wr, topk_ids, topk_w, stream)


def moe_set_green_ctx(ctx, dispatch_sms) -> int:
    return lib().moe_set_green_ctx(ctx, dispatch_sms)


def moe_green_ctx_sms(ctx):
    d, g = _i(), _i()
    _check(lib().moe_green_ctx_sms(ctx, ctypes.byref(d), ctypes.byref(g)), "moe_green_ctx_sms")
    return d.value, g.value


def moe_set_dispatch_overlap(ctx, dispatch_ctas) -> int:
    return lib().moe_set_dispatch_overlap(ctx, dispatch_ctas)


def moe_dispatch_overlap_ctas(ctx) -> int:
    d = _i()
    _check(lib().moe_dispatch_overlap_ctas(ctx, ctypes.byref(d)), "moe_dispatch_overlap_ctas")
    return d.value


def moe_profile_enable(ctx, on) -> int:
    return lib().moe_profile_enable(ctx, on)


def moe_profile_read(ctx):
    """Mean milliseconds per stage over the recorded calls, and their number."""
    arr = (ctypes.c_float * MOE_NUM_STAGES)()
    n = _i()
    _check(lib().moe_profile_read(ctx, arr, ctypes.byref(n)), "moe_profile_read")
    return list(arr), n.value


def moe_route(ctx, T, topk_ids, counts, offsets, perm, inv, stream) -> int:
    return lib().moe_route(ctx, T, topk_ids, counts, offsets, perm, inv, stream)


def moe_permute(dtype, rows, H, T, k, x, ldx, perm, y, ldy, stream) -> int:
    return lib().moe_permute(dtype, rows, H, T, k, x, ldx, perm, y, ldy, stream)


def moe_combine(dtype, rows, H, T, k, n_shared, y, ldy, inv, topk_w, out, ldo, stream) -> int:
    return lib().moe_combine(dtype, rows, H, T, k, n_shared, y, ldy, inv, topk_w, out, ldo, stream)


def moe_combine_backward(dtype, rows, H, T, k, n_shared, dout, lddout, y, ldy, inv, topk_w, dy, lddy, dtopk_w,
                         stream) -> int:
    return lib().moe_combine_backward(dtype, rows, H, T, k, n_shared, dout, lddout, y, ldy, inv, topk_w, dy, lddy,
                                      dtopk_w, stream)


def moe_grouped_gemm(dtype, out_dtype, E, P, N, K, offsets, x, ldx, w, ldw, stride_w, y, ldy, d_status, stream) -> int:
    return lib().moe_grouped_gemm(dtype, out_dtype, E, P, N, K, offsets, x, ldx, w, ldw, stride_w, y, ldy, d_status,
                                  stream)


def moe_grouped_gemm_dgrad(dtype, out_dtype, E, P, N, K, offsets, dy, lddy, w, ldw, stride_w, dx, lddx, d_status,
                           stream) -> int:
    return lib().moe_grouped_gemm_dgrad(dtype, out_dtype, E, P, N, K, offsets, dy, lddy, w, ldw, stride_w, dx, lddx,
                                        d_status, stream)


def moe_grouped_gemm_wgrad(dtype, out_dtype, E, P, N, K, offsets, dy, lddy, x, ldx, dw, d_status, stream) -> int:
    return lib().moe_grouped_gemm_wgrad(dtype, out_dtype, E, P, N, K, offsets, dy, lddy, x, ldx, dw, d_status, stream)


def moe_quant_int8(dtype, rows, K, T, k, x, ldx, perm, q, ldq, scale, stream) -> int:
    return lib().moe_quant_int8(dtype, rows, K, T, k, x, ldx, perm, q, ldq, scale, stream)


def moe_int8_gemm(out_dtype, E, P, N, K, offsets, q, ldq, q_scale, w, ldw, stride_w, w_scale, y, ldy, d_status,
                  stream) -> int:
    return lib().moe_int8_gemm(out_dtype, E, P, N, K, offsets, q, ldq, q_scale, w, ldw, stride_w, w_scale, y, ldy,
                               d_status, stream)


def moe_ops_status(stream) -> int:
    return lib().moe_ops_status(stream)


# ---- torch convenience wrapper (marshalling only) ------------------------
def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


class MoeLayer:
    """One context of the library; tensors are torch CUDA tensors."""

    def __init__(self, H, I, E, k, wfmt=MOE_WFMT_FP8_E4M3_B128, max_T=4096, n_shared=0):
        self.H, self.I, self.E, self.k, self.wfmt = H, I, E, k, wfmt
        self.max_T, self.n_shared = max_T, n_shared
        self.ctx = moe_create_ex(H, I, E, k, wfmt, max_T, n_shared)
        import torch
        self.device = torch.cuda.current_device()   # the context's

    def close(self):
        if self.ctx:
            moe_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, x, topk_ids, topk_w, w13, s13, w2, s2, out=None, stream=None, g13=None, g2=None):
        """One layer; NVFP4 contexts also take the global scales g13 / g2 (moe_forward_nvfp4)."""
        import torch
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.bfloat16, device=x.device)
        nv = self.wfmt == MOE_WFMT_NVFP4_E2M1_E4M3_K16
        ts = (x, topk_ids, topk_w, w13, s13, w2, s2, out) + ((g13, g2) if nv else ())
        for t in ts:
            if t is None or not t.is_cuda or not t.is_contiguous():
                raise ValueError("MoeLayer.forward needs contiguous CUDA tensors")
        if nv:
            _check(moe_forward_nvfp4(self.ctx, T, _ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13), _ptr(s13),
                                     _ptr(g13), _ptr(w2), _ptr(s2), _ptr(g2), _ptr(out), _stream_handle(stream)),
                   "moe_forward_nvfp4")
        else:
            _check(moe_forward(self.ctx, T, _ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13), _ptr(s13),
                               _ptr(w2), _ptr(s2), _ptr(out), _stream_handle(stream)), "moe_forward")
        return out

    def forward_partial(self, x, topk_ids, topk_w, w13, s13, w2, s2, out=None, stream=None, g13=None, g2=None):
        """fp32 [T, H] partial combine result of this context's I slice (moe_forward_partial)."""
        import torch
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.float32, device=x.device)
        for t in (x, topk_ids, topk_w, w13, s13, w2, s2, out):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("MoeLayer.forward_partial needs contiguous CUDA tensors")
        _check(moe_forward_partial(self.ctx, T, _ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13), _ptr(s13),
                                   _ptr(g13), _ptr(w2), _ptr(s2), _ptr(g2), _ptr(out), _stream_handle(stream)),
               "moe_forward_partial")
        return out

    def routing(self, T, stream=None):
        """(counts, offsets, perm, inv) of the last forward, as host int32 numpy arrays."""
        import numpy as np
        P = T * self.k + self.n_shared * T
        NG = self.E + self.n_shared
        counts = np.zeros(NG, np.int32)
        offsets = np.zeros(NG + 1, np.int32)
        perm = np.zeros(max(P, 1), np.int32)
        inv = np.zeros(max(P, 1), np.int32)
        _check(moe_get_routing(self.ctx, counts.ctypes.data, offsets.ctypes.data, perm.ctypes.data,
                               inv.ctypes.data, _stream_handle(stream)), "moe_get_routing")
        return counts, offsets, perm[:P], inv[:P]

    def activations(self, T, stream=None):
        """(xq, xs, hq, hs) of the last forward, host numpy arrays in routing-position order
        (NVFP4: xq / hq packed, two codes per byte)."""
        import numpy as np
        P = T * self.k + self.n_shared * T
        cw = 2 if self.wfmt in (MOE_WFMT_NVFP4_E2M1_E4M3_K16, MOE_WFMT_MXFP4_W4A4) else 1
        xq = np.zeros((max(P, 1), self.H // cw), np.uint8)
        xs = np.zeros((max(P, 1), self.H // 128), np.float32)
        hq = np.zeros((max(P, 1), self.I // cw), np.uint8)
        hs = np.zeros((max(P, 1), self.I // 128), np.float32)
        _check(moe_get_activations(self.ctx, xq.ctypes.data, xs.ctypes.data, hq.ctypes.data, hs.ctypes.data,
                                   _stream_handle(stream)), "moe_get_activations")
        return xq[:P], xs[:P], hq[:P], hs[:P]

    def block_scales(self, T, stream=None):
        """4-bit activations: (xsc, hsc) block codes of the last forward, host numpy
        (NVFP4: E4M3 [P, H/16], [P, I/16]; MXFP4 x MXFP4: E8M0 [P, H/32], [P, I/32])."""
        import numpy as np
        P = T * self.k + self.n_shared * T
        bs = 16 if self.wfmt == MOE_WFMT_NVFP4_E2M1_E4M3_K16 else 32
        xsc = np.zeros((max(P, 1), self.H // bs), np.uint8)
        hsc = np.zeros((max(P, 1), self.I // bs), np.uint8)
        _check(moe_get_block_scales(self.ctx, xsc.ctypes.data, hsc.ctypes.data, _stream_handle(stream)),
               "moe_get_block_scales")
        return xsc[:P], hsc[:P]

    def device_status(self, stream=None) -> int:
        return moe_get_device_status(self.ctx, _stream_handle(stream))

    def last_config(self):
        return moe_last_config(self.ctx)

    def router(self, x, wr, ids=None, w=None, stream=None):
        """Fused router: (topk_ids int32 [T,k], topk_w fp32 [T,k]) from x bf16 [T,H] and wr bf16 [E,H]."""
        import torch
        T = x.shape[0]
        if ids is None:
            ids = torch.empty((T, self.k), dtype=torch.int32, device=x.device)
        if w is None:
            w = torch.empty((T, self.k), dtype=torch.float32, device=x.device)
        for t in (x, wr, ids, w):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("MoeLayer.router needs contiguous CUDA tensors")
        _check(moe_router_topk(self.ctx, T, _ptr(x), _ptr(wr), _ptr(ids), _ptr(w), _stream_handle(stream)),
               "moe_router_topk")
        return ids, w

    def route(self, topk_ids, stream=None):
        """Device int32 (counts, offsets, perm, inv) of topk_ids [T, k], in stream order (moe_route)."""
        import torch
        T = topk_ids.shape[0]
        if topk_ids.shape != (T, self.k):
            raise ValueError(f"topk_ids has shape {tuple(topk_ids.shape)}, not [T, {self.k}]")
        NG, P = self.E + self.n_shared, T * (self.k + self.n_shared)
        _vector(topk_ids, P - T * self.n_shared, "route", "topk_ids")
        dev = self.device
        _on("route", dev, "topk_ids", topk_ids, torch.int32)

        def body(s):
            counts, offsets, perm, inv = (torch.empty(n, dtype=torch.int32, device=dev) for n in (NG, NG + 1, P, P))
            _check(moe_route(self.ctx, T, _ptr(topk_ids), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), s),
                   "moe_route")
            return counts, offsets, perm, inv
        return _call("route", dev, stream, body)

    def set_green_ctx(self, dispatch_sms):
        """Green-Context partition: dispatch kernels on >= dispatch_sms SMs, GEMMs on the rest (0 = off)."""
        _check(moe_set_green_ctx(self.ctx, dispatch_sms), "moe_set_green_ctx")
        return moe_green_ctx_sms(self.ctx)

    def set_dispatch_overlap(self, dispatch_ctas):
        """Dispatch overlap: the last dispatch_ctas CTAs of the GEMM1 launch quantise first (0 = off)."""
        _check(moe_set_dispatch_overlap(self.ctx, dispatch_ctas), "moe_set_dispatch_overlap")
        return moe_dispatch_overlap_ctas(self.ctx)


def pack_nvfp4_scales(s, stream=None):
    """Plain E4M3 block codes [NE, rows, K/16] (uint8 CUDA tensor) -> the layout moe_forward_nvfp4 reads."""
    NE, rows, kg = s.shape
    dst = __import__("torch").empty_like(s)
    _check(moe_pack_nvfp4_scales(_ptr(s.contiguous()), _ptr(dst), NE * rows, kg * 16, _stream_handle(stream)),
           "moe_pack_nvfp4_scales")
    return dst


def pack_mxfp4_scales(s, stream=None):
    """Plain E8M0 scales [NE, rows, K/32] (uint8 CUDA tensor) -> the layout moe_forward reads."""
    import torch
    NE, rows, kg = s.shape
    dst = torch.empty_like(s)
    _check(moe_pack_mxfp4_scales(_ptr(s.contiguous()), _ptr(dst), NE * rows, kg * 32, _stream_handle(stream)),
           "moe_pack_mxfp4_scales")
    return dst


def finalize_bf16(acc, out=None, stream=None):
    """bf16 rounding of a summed fp32 [T, H] result (moe_finalize_bf16)."""
    import torch
    if out is None:
        out = torch.empty(acc.shape, dtype=torch.bfloat16, device=acc.device)
    _check(moe_finalize_bf16(_ptr(acc.contiguous()), _ptr(out), acc.numel(), _stream_handle(stream)),
           "moe_finalize_bf16")
    return out


# ---- expert operators on torch tensors (marshalling only) -----------------
# Small calls are bound by the host, so the checks below are flat and build
# their messages only when they fail.
def _on(what, dev, name, t, dtype):
    """Refuses t (None passes) unless it is a `dtype` tensor on CUDA device `dev`."""
    if t is None:
        return
    if t.get_device() != dev:
        raise ValueError(f"{what}: {name} is on {t.device}, not on cuda:{dev}" if t.is_cuda else
                         f"{what}: {name} is not a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {name} is {t.dtype}, not {dtype}")


def _call(what, dev, stream, body):
    """body(stream handle) with device `dev` current and `stream` (default: that device's current one) the stream that
    results are allocated on."""
    import torch
    if dev < 0:
        raise ValueError(f"{what}: the first argument is not a CUDA tensor")
    if stream is None and torch.cuda.current_device() == dev:
        # the handle alone: torch.cuda.current_stream() builds an object around it, 2 us
        return body(torch._C._cuda_getCurrentRawStream(dev))
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"{what}: the stream is on {stream.device}, the tensors on cuda:{dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return body(torch._C._cuda_getCurrentRawStream(dev))


def ops_status(stream=None) -> int:
    """Errors of the expert operators called without `status` on the stream's device (default: the current one) since the
    last such question: MOE_OK, MOE_ERR_BAD_ROUTING (unusable offsets: a result made by the call is unset) or
    MOE_ERR_TIMEOUT (moe_ops_status).  Waits for the stream."""
    import torch
    with torch.cuda.stream(stream):
        return moe_ops_status(_stream_handle(stream))


_no_formula = None


def _results(what, made, given, *inputs):
    """`made`, the result of a call, as autograd has to see it.

    These operators have no autograd formula: their gradients are calls of their own.  If an input records a gradient, a
    backward pass through what is returned raises.  A caller's tensor that the result was written into (`given`) has a
    new version, so that a graph which kept its old values notices."""
    if given is not None:
        from torch.autograd.graph import increment_version
        increment_version(given)
    for t in inputs:
        if t.requires_grad:
            break
    else:
        return made
    import torch
    if not torch.is_grad_enabled():
        return made
    global _no_formula
    if _no_formula is None:
        class NoFormula(torch.autograd.Function):
            @staticmethod
            def forward(ctx, what, made, *inputs):
                ctx.what = what
                return made   # (another tensor of the same memory: a caller's own stays outside of the graph)

            @staticmethod
            def backward(ctx, *grads):
                raise NotImplementedError(f"moe.{ctx.what} has no autograd formula: its gradient is a call of its own")
        _no_formula = NoFormula
    return _no_formula.apply(what, made, *inputs)


def _dtype_code(dtype, what):
    import torch
    if dtype is torch.bfloat16:
        return MOE_DT_BF16
    if dtype is torch.float16:
        return MOE_DT_FP16
    if dtype is torch.float32:
        return MOE_DT_FP32
    raise ValueError(f"{what}: type {dtype} is not supported")


def _rows_out(out, rows, n, dtype, dev, what, name="out"):
    """(matrix, row stride): `out`, checked, or an unset [rows, n] matrix whose row stride is a multiple of 16 bytes
    (contiguous where n allows it)."""
    if out is not None:
        return out, _matrix(out, rows, n, what, name)
    import torch
    step = 16 // dtype.itemsize
    ld = -(-n // step) * step
    return torch.empty_strided((rows, n), (ld, 1), dtype=dtype, device=dev), ld


def _matrix(t, rows, cols, what, name):
    """Row stride in elements of a [rows, cols] matrix with contiguous rows; None: any size."""
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{what}: {name} has shape {tuple(shape)}, not "
                         f"[{'any' if rows is None else rows}, {'any' if cols is None else cols}]")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{what}: {name}: rows are not contiguous")
    if shape[0] > 1:
        return s0
    step = 16 // t.element_size()      # a single row: its stride is never used
    return -(-shape[1] // step) * step


_INT_MAX = 2 ** 31 - 1


def _too_large(what):
    """What the library does not take, and ctypes would pass the low 32 bits of."""
    raise MoeError(MOE_ERR_UNSUPPORTED, what)


def _missing(what, name):
    raise ValueError(f"{what}: {name} is None")


def _vector(t, n, what, name):
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: {name}: expected {n} contiguous elements, got shape {tuple(t.shape)}")


def _weights(w, offsets, what):
    """(E, N, K, row stride, expert stride) of the weights; offsets [E + 1] fit them."""
    shape = w.shape
    if len(shape) != 3:
        raise ValueError(f"{what}: w has shape {tuple(shape)}, not [E, N, K]")
    E, N, K = shape
    if offsets is not None and (offsets.numel() != E + 1 or offsets.dim() != 1 or not offsets.is_contiguous()):
        raise ValueError(f"{what}: offsets has shape {tuple(offsets.shape)}, not [{E + 1}]")
    se, sn, sk = w.stride()
    if sk != 1 and K > 1:
        raise ValueError(f"{what}: w: rows are not contiguous")
    step = 16 // w.element_size()
    return E, N, K, sn if N > 1 else -(-K // step) * step, se if E > 1 else 0


def _grouped(entry, what, name, rows, forward, w, offsets, out, out_dtype, status, stream):
    import torch
    if offsets is None:
        _missing(what, "offsets")
    E, N, K, ldw, sw = _weights(w, offsets, what)
    P = rows.shape[0]
    if E + P + N + K > _INT_MAX:
        _too_large(what)
    R, M = (K, N) if forward else (N, K)
    ld = _matrix(rows, P, R, what, name)
    dtype = rows.dtype
    if out is not None:
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = dtype
    dt = _dtype_code(dtype, what)
    odt = dt if out_dtype is dtype else _dtype_code(out_dtype, what)
    dev = rows.get_device()
    _on(what, max(dev, 0), name, rows, dtype)
    _on(what, dev, "w", w, dtype)
    _on(what, dev, "offsets", offsets, torch.int32)
    _on(what, dev, "out", out, out_dtype)
    _on(what, dev, "status", status, torch.int32)

    def body(s):
        y, ldy = _rows_out(out, P, M, out_dtype, dev, what)
        st = getattr(lib(), entry)(dt, odt, E, P, N, K, offsets.data_ptr(), rows.data_ptr(), ld, w.data_ptr(), ldw, sw,
                                   y.data_ptr(), ldy, _ptr(status), s)
        if st != MOE_OK:
            raise MoeError(st, entry)
        return y
    y = _call(what, dev, stream, body)
    if out is None and not (rows.requires_grad or w.requires_grad):
        return y
    return _results(what, y, out, rows, w)


def grouped_gemm(x, w, offsets, out=None, out_dtype=None, status=None, stream=None):
    """y[p] = x[p] w[e]^T for the rows offsets[e] .. offsets[e+1]-1 of every expert e (moe_grouped_gemm).

    x [P, K] and w [E, N, K] bf16 or fp16 with contiguous rows (any row and expert strides that are multiples of 16
    bytes), offsets device int32 [E+1]; out [P, N] in the same type or fp32.  Rows outside every group are left as
    they were (unspecified in an `out` made here).  status: device int32 that errors found on the device are ORed into
    (see moe.h); without one, ops_status() tells of them."""
    return _grouped("moe_grouped_gemm", "grouped_gemm", "x", x, True, w, offsets, out, out_dtype, status, stream)


def grouped_gemm_dgrad(dy, w, offsets, out=None, out_dtype=None, status=None, stream=None):
    """dx[p] = dy[p] w[e], the gradient of grouped_gemm for x (moe_grouped_gemm_dgrad): dy [P, N] -> [P, K]."""
    return _grouped("moe_grouped_gemm_dgrad", "grouped_gemm_dgrad", "dy", dy, False, w, offsets, out, out_dtype, status,
                    stream)


def grouped_gemm_wgrad(dy, x, offsets, out=None, out_dtype=None, status=None, stream=None):
    """dw[e] = sum over the rows of e of dy[p]^T x[p], the gradient of grouped_gemm for w (moe_grouped_gemm_wgrad):
    dy [P, N], x [P, K] -> [E, N, K], zeros for an expert without rows."""
    import torch
    what = "grouped_gemm_wgrad"
    lddy = _matrix(dy, None, None, what, "dy")
    ldx = _matrix(x, dy.shape[0], None, what, "x")
    if offsets is None:
        _missing(what, "offsets")
    (P, N), K, E = dy.shape, x.shape[1], offsets.shape[0] - 1
    if E + P + N + K > _INT_MAX:
        _too_large(what)
    _vector(offsets, E + 1, what, "offsets")
    dtype = dy.dtype
    out_dtype = out.dtype if out is not None else (out_dtype or dtype)
    dt, odt = _dtype_code(dtype, what), _dtype_code(out_dtype, what)
    dev = dy.get_device()
    _on(what, max(dev, 0), "dy", dy, dy.dtype)
    _on(what, dev, "x", x, dtype)
    _on(what, dev, "offsets", offsets, torch.int32)
    _on(what, dev, "out", out, out_dtype)
    _on(what, dev, "status", status, torch.int32)
    if out is not None and (out.shape != (E, N, K) or not out.is_contiguous()):
        raise ValueError(f"{what}: out is not contiguous [{E}, {N}, {K}]")

    def body(s):
        dw = torch.empty((E, N, K), dtype=out_dtype, device=dev) if out is None else out
        _check(lib().moe_grouped_gemm_wgrad(dt, odt, E, P, N, K, offsets.data_ptr(), dy.data_ptr(), lddy, x.data_ptr(),
                                            ldx, dw.data_ptr(), _ptr(status), s), "moe_grouped_gemm_wgrad")
        return dw
    return _results(what, _call(what, dev, stream, body), out, dy, x)


def quant_int8(x, perm=None, k=1, out=None, scale=None, stream=None):
    """(q int8 [rows, K], scale fp32 [rows]) of x [T, K] bf16 or fp16, one scale amax / 127 per row (moe_quant_int8).
    With perm (device int32 [rows]) row p is token perm[p] // k, quantised in expert order."""
    import torch
    what = "quant_int8"
    ldx = _matrix(x, None, None, what, "x")
    T, K = x.shape
    rows = T if perm is None else perm.shape[0]
    if T + K + rows + abs(k) > _INT_MAX:
        _too_large(what)
    dt = _dtype_code(x.dtype, what)
    dev = x.get_device()
    _on(what, max(dev, 0), "x", x, x.dtype)
    _on(what, dev, "perm", perm, torch.int32)
    _on(what, dev, "out", out, torch.int8)
    _on(what, dev, "scale", scale, torch.float32)
    if perm is not None:
        _vector(perm, rows, what, "perm")

    def body(s):
        q, ldq = _rows_out(out, rows, K, torch.int8, dev, what)
        sc = torch.empty_strided((rows,), (1,), dtype=torch.float32, device=dev) if scale is None else scale
        _vector(sc, rows, what, "scale")
        _check(lib().moe_quant_int8(dt, rows, K, T, k, x.data_ptr(), ldx, _ptr(perm), q.data_ptr(), ldq,
                                    sc.data_ptr(), s), "moe_quant_int8")
        return q, sc
    q, sc = _call(what, dev, stream, body)
    if out is None and scale is None and not x.requires_grad:
        return q, sc
    return _results(what, q, out), _results(what, sc, scale, x)


def int8_gemm(q, q_scale, w, w_scale, offsets=None, out=None, out_dtype=None, status=None, stream=None):
    """y[p, n] = q_scale[p] w_scale[e, n] sum_k q[p, k] w[e, n, k] (moe_int8_gemm).

    q int8 [P, K], q_scale fp32 [P], w int8 [E, N, K] and w_scale fp32 [E, N] (or [N, K] and [N] without offsets: one
    dense product), offsets device int32 [E+1].  out [P, N] bf16 (default), fp16 or fp32."""
    import torch
    what = "int8_gemm"
    if offsets is None and w.dim() == 2:
        (N, K), E, sw = w.shape, 1, 0
        ldw = _matrix(w, N, K, what, "w")
    elif offsets is None and (w.dim() != 3 or w.shape[0] != 1):
        raise ValueError(f"{what}: w has shape {tuple(w.shape)}; one matrix without offsets, [E, N, K] with them")
    else:
        E, N, K, ldw, sw = _weights(w, offsets, what)
    P = q.shape[0]
    if E + P + N + K > _INT_MAX:
        _too_large(what)
    ldq = _matrix(q, P, K, what, "q")
    _vector(q_scale, P, what, "q_scale")
    _vector(w_scale, E * N, what, "w_scale")
    out_dtype = out.dtype if out is not None else (out_dtype or torch.bfloat16)
    odt = _dtype_code(out_dtype, what)
    dev = q.get_device()
    _on(what, max(dev, 0), "q", q, torch.int8)
    _on(what, dev, "q_scale", q_scale, torch.float32)
    _on(what, dev, "w", w, torch.int8)
    _on(what, dev, "w_scale", w_scale, torch.float32)
    _on(what, dev, "offsets", offsets, torch.int32)
    _on(what, dev, "out", out, out_dtype)
    _on(what, dev, "status", status, torch.int32)

    def body(s):
        y, ldy = _rows_out(out, P, N, out_dtype, dev, what)
        _check(lib().moe_int8_gemm(odt, E, P, N, K, _ptr(offsets), q.data_ptr(), ldq, q_scale.data_ptr(), w.data_ptr(),
                                   ldw, sw, w_scale.data_ptr(), y.data_ptr(), ldy, _ptr(status), s), "moe_int8_gemm")
        return y
    y = _call(what, dev, stream, body)
    if out is None and not (q_scale.requires_grad or w_scale.requires_grad):
        return y
    return _results(what, y, out, q_scale, w_scale)


def permute(x, perm, k, out=None, stream=None):
    """y[p] = x[perm[p] // k]: rows of x [T, H] (bf16, fp16 or fp32) in expert order (moe_permute).  Rows whose slot is
    -1 are left as they were (unspecified in an `out` made here)."""
    import torch
    what = "permute"
    ldx = _matrix(x, None, None, what, "x")
    T, H = x.shape
    if perm is None:
        _missing(what, "perm")
    rows = perm.shape[0]
    if T + H + rows + abs(k) > _INT_MAX:
        _too_large(what)
    _vector(perm, rows, what, "perm")
    dt = _dtype_code(x.dtype, what)
    dev = x.get_device()
    _on(what, max(dev, 0), "x", x, x.dtype)
    _on(what, dev, "perm", perm, torch.int32)
    _on(what, dev, "out", out, x.dtype)

    def body(s):
        y, ldy = _rows_out(out, rows, H, x.dtype, dev, what)
        _check(lib().moe_permute(dt, rows, H, T, k, x.data_ptr(), ldx, perm.data_ptr(), y.data_ptr(), ldy, s),
               "moe_permute")
        return y
    y = _call(what, dev, stream, body)
    if out is None and not x.requires_grad:
        return y
    return _results(what, y, out, x)


def _combine_sizes(inv, topk_w, k, n_shared, what):
    """(T, k) from the slots' count; topk_w [T, k], or None with k given."""
    if inv is None:
        _missing(what, "inv")
    if topk_w is not None:
        if topk_w.dim() != 2 or (k is not None and topk_w.shape[1] != k):
            raise ValueError(f"{what}: topk_w has shape {tuple(topk_w.shape)}, not [T, k]")
        T, k = topk_w.shape
        _vector(topk_w, T * k, what, "topk_w")
    else:
        if k is None:
            raise ValueError(f"{what}: without topk_w, k has to be given")
        if k < 1 or n_shared < 0:
            raise ValueError(f"{what}: k is {k}, n_shared is {n_shared}")
        T = inv.numel() // (k + n_shared)
    _vector(inv, T * (k + n_shared), what, "inv")
    return T, k


def combine(y, inv, topk_w=None, k=None, n_shared=0, out=None, stream=None):
    """out[t] = sum_j topk_w[t, j] y[inv[t*k + j]] (+ the shared expert's row) from y [rows, H] (moe_combine).
    topk_w fp32 [T, k], or None (ones; then k is given): the gradient of permute."""
    import torch
    what = "combine"
    ldy = _matrix(y, None, None, what, "y")
    rows, H = y.shape
    T, k = _combine_sizes(inv, topk_w, k, n_shared, what)
    if rows + H + T + k + n_shared > _INT_MAX:
        _too_large(what)
    dt = _dtype_code(y.dtype, what)
    dev = y.get_device()
    _on(what, max(dev, 0), "y", y, y.dtype)
    _on(what, dev, "inv", inv, torch.int32)
    _on(what, dev, "topk_w", topk_w, torch.float32)
    _on(what, dev, "out", out, y.dtype)

    def body(s):
        o, ldo = _rows_out(out, T, H, y.dtype, dev, what)
        _check(lib().moe_combine(dt, rows, H, T, k, n_shared, y.data_ptr(), ldy, inv.data_ptr(), _ptr(topk_w),
                                 o.data_ptr(), ldo, s), "moe_combine")
        return o
    o = _call(what, dev, stream, body)
    weights = y if topk_w is None else topk_w
    if out is None and not (y.requires_grad or weights.requires_grad):
        return o
    return _results(what, o, out, y, weights)


def combine_backward(dout, y, inv, topk_w, n_shared=0, dy=None, dtopk_w=None, stream=None):
    """(dy, dtopk_w): gradients of combine for y and topk_w (moe_combine_backward).  Rows of dy that no slot names are
    left as they were (unspecified in a `dy` made here)."""
    import torch
    what = "combine_backward"
    if topk_w is None:
        _missing(what, "topk_w")
    T, k = _combine_sizes(inv, topk_w, None, n_shared, what)
    ldy = _matrix(y, None, None, what, "y")
    rows, H = y.shape
    if rows + H + T + k + n_shared > _INT_MAX:
        _too_large(what)
    ldd = _matrix(dout, T, H, what, "dout")
    dt = _dtype_code(y.dtype, what)
    dev = y.get_device()
    _on(what, max(dev, 0), "y", y, y.dtype)
    _on(what, dev, "dout", dout, y.dtype)
    _on(what, dev, "inv", inv, torch.int32)
    _on(what, dev, "topk_w", topk_w, torch.float32)
    _on(what, dev, "dy", dy, y.dtype)
    _on(what, dev, "dtopk_w", dtopk_w, torch.float32)

    def body(s):
        gy, lddy = _rows_out(dy, rows, H, y.dtype, dev, what, "dy")
        gw = torch.empty_strided((T, k), (k, 1), dtype=torch.float32, device=dev) if dtopk_w is None else dtopk_w
        _vector(gw, T * k, what, "dtopk_w")
        _check(lib().moe_combine_backward(dt, rows, H, T, k, n_shared, dout.data_ptr(), ldd, y.data_ptr(), ldy,
                                          inv.data_ptr(), topk_w.data_ptr(), gy.data_ptr(), lddy, gw.data_ptr(), s),
               "moe_combine_backward")
        return gy, gw
    gy, gw = _call(what, dev, stream, body)
    return _results(what, gy, dy, dout, topk_w), _results(what, gw, dtopk_w, dout, y)
