"""Python binding of the C ABI (include/cc.h): the same entry points under the
same names, taking torch CUDA tensors instead of raw pointers.

Argument marshalling only: each function checks that its tensors are CUDA,
contiguous and of the expected dtype, reads the sizes off their shapes, and
calls the library on the current (or given) stream. All compute runs in
libcc.so's kernels. A non-OK status raises ``CCError`` with the library's
message.
"""

from __future__ import annotations

import math

import torch

from . import _lib

__all__ = [
    "CCError", "cc_version", "cc_check_device",
    "cc_conv3d_prepare", "cc_conv3d_causal",
    "cc_resample_prepare", "cc_resample_workspace_bytes", "cc_resample_phase_conv", "cc_resample_interleave",
    "cc_resample_up2", "cc_resample_up2_fused", "cc_resample_prepare_temporal",
    "cc_attn_ld", "cc_attn_workspace_bytes", "cc_attn_scores", "cc_attn_softmax", "cc_attn_pv", "cc_attn_frame",
    "cc_attn_exp_key_tiles", "cc_attn_exp_workspace_bytes", "cc_attn_scores_exp", "cc_attn_exp_rescale",
    "cc_attn_pv_exp", "cc_attn_frame_exp",
    "cc_head_prepare", "cc_head_workspace_bytes", "cc_head_temporal", "cc_head_stencil", "cc_head_out",
    "cc_attn_scores_stats", "cc_attn_fused_workspace_bytes", "cc_attn_frame_fused",
    "cc_head_out_fused", "cc_head_out_noalloc", "HEAD_NOALLOC_SCRATCH_BYTES", "cc_copy_to_host",
    "cc_group_norm_workspace_bytes", "cc_group_norm_act", "cc_group_norm_act_fp8",
    "cc_rms_norm_act", "cc_rms_norm_act_fp8",
    "cc_fp8_quantize", "cc_gemm_fp8_prepare", "cc_gemm_fp8",
    "cc_qk_norm_rope", "cc_qk_norm_rope_append",
    "cc_attn_paged_workspace_bytes", "cc_attn_paged", "cc_attn_cross_workspace_bytes", "cc_attn_cross",
    "cc_debug_im2col_tile", "cc_debug_wait_timeout", "cc_debug_conv_bad_tile_order",
    "HEAD_COUT", "HEAD_G_CH",
]

HEAD_COUT = 12
HEAD_G_CH = 112
HEAD_NOALLOC_SCRATCH_BYTES = 64 << 20  # CC_HEAD_NOALLOC_SCRATCH_BYTES

STATUS = {0: "CC_OK", 1: "CC_ERR_INVALID", 2: "CC_ERR_UNSUPPORTED", 3: "CC_ERR_CUDA", 4: "CC_ERR_TIMEOUT",
          5: "CC_ERR_DEVICE"}


class CCError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


def _check(st: int) -> None:
    if st != 0:
        msg = _lib.load().cc_last_error()
        raise CCError(st, msg.decode() if msg else "")


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None, dtype=torch.bfloat16, name: str = "tensor") -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def cc_version() -> int:
    return _lib.load().cc_version()


def cc_check_device(stream=None) -> None:
    _check(_lib.load().cc_check_device(_stream(stream)))


# ------------------------------------------------------- causal 3x3x3 conv --

def cc_conv3d_prepare(w: torch.Tensor, wp: torch.Tensor, stream=None) -> None:
    cout, cin = w.shape[:2]
    if tuple(w.shape) != (cout, cin, 3, 3, 3) or wp.numel() != 27 * cout * cin:
        raise ValueError("conv3d_prepare: w must be [Cout,Cin,3,3,3] and wp hold 27*Cout*Cin elements")
    _check(_lib.load().cc_conv3d_prepare(_ptr(w, name="w"), _ptr(wp, name="wp"), cout, cin, _stream(stream)))


def cc_conv3d_causal(x, wp, bias, y, hist: int = 0, stream=None) -> None:
    n, d, h, w, cout = y.shape
    cin = x.shape[-1]
    if tuple(x.shape) != (n, d + hist, h, w, cin):
        raise ValueError(f"conv3d_causal: x {tuple(x.shape)} does not match y {tuple(y.shape)} with hist={hist}")
    if wp.numel() != 27 * cout * cin:
        raise ValueError("conv3d_causal: wp must hold 27*Cout*Cin elements")
    if bias is not None and bias.numel() != cout:
        raise ValueError("conv3d_causal: bias must hold Cout elements")
    _check(_lib.load().cc_conv3d_causal(_ptr(x, name="x"), _ptr(wp, name="wp"), _ptr(bias, name="bias"),
                                        _ptr(y, name="y"), n, d, h, w, cin, cout, hist, _stream(stream)))


# ------------------------------------------------------- spatial resampler --

def cc_resample_prepare(w, pw, stream=None) -> None:
    cout, cin = w.shape[:2]
    if tuple(w.shape) != (cout, cin, 3, 3, 3) or pw.numel() != 48 * cout * cin:
        raise ValueError("resample_prepare: w must be [Cout,Cin,3,3,3] and pw hold 48*Cout*Cin elements")
    _check(_lib.load().cc_resample_prepare(_ptr(w, name="w"), _ptr(pw, name="pw"), cout, cin, _stream(stream)))


def cc_resample_workspace_bytes(n: int, d: int, hl: int, wl: int, cout: int) -> int:
    return _lib.load().cc_resample_workspace_bytes(n, d, hl, wl, cout)


def cc_resample_phase_conv(x, pw, phases, hist: int = 0, stream=None) -> None:
    four, n, d, hl, wl, cout = phases.shape
    cin = x.shape[-1]
    if four != 4 or tuple(x.shape) != (n, d + hist, hl, wl, cin) or pw.numel() != 48 * cout * cin:
        raise ValueError("resample_phase_conv: phases must be [4,N,D,HL,WL,Cout] matching x and pw")
    _check(_lib.load().cc_resample_phase_conv(_ptr(x, name="x"), _ptr(pw, name="pw"), _ptr(phases, name="phases"),
                                              n, d, hl, wl, cin, cout, hist, _stream(stream)))


def cc_resample_interleave(phases, bias, skip, out, stream=None) -> None:
    four, n, d, hl, wl, c = phases.shape
    if four != 4 or tuple(skip.shape) != (n, d, hl, wl, c) or tuple(out.shape) != (n, d, 2 * hl, 2 * wl, c) \
            or bias.numel() != c:
        raise ValueError("resample_interleave: shapes do not match")
    _check(_lib.load().cc_resample_interleave(_ptr(phases, name="phases"), _ptr(bias, name="bias"),
                                              _ptr(skip, name="skip"), _ptr(out, name="out"), n, d, hl, wl, c,
                                              _stream(stream)))


def cc_resample_up2(x, pw, bias, skip, out, ws, hist: int = 0, stream=None) -> None:
    n, d, h2, w2, cout = out.shape
    hl, wl = h2 // 2, w2 // 2
    cin = x.shape[-1]
    if h2 != 2 * hl or w2 != 2 * wl or tuple(x.shape) != (n, d + hist, hl, wl, cin):
        raise ValueError("resample_up2: out must be [N,D,2HL,2WL,Cout] of x [N,D+hist,HL,WL,Cin]")
    if tuple(skip.shape) != (n, d, hl, wl, cout) or bias.numel() != cout or pw.numel() != 48 * cout * cin:
        raise ValueError("resample_up2: skip, bias or pw shape mismatch")
    _check(_lib.load().cc_resample_up2(_ptr(x, name="x"), _ptr(pw, name="pw"), _ptr(bias, name="bias"),
                                       _ptr(skip, name="skip"), _ptr(out, name="out"), n, d, hl, wl, cin, cout, hist,
                                       _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def cc_resample_prepare_temporal(w, pw, stream=None) -> None:
    cout, cin = w.shape[:2]
    if tuple(w.shape) != (cout, cin, 3, 3, 3) or pw.numel() != 64 * cout * cin:
        raise ValueError("resample_prepare_temporal: w must be [Cout,Cin,3,3,3] and pw hold 64*Cout*Cin elements")
    _check(_lib.load().cc_resample_prepare_temporal(_ptr(w, name="w"), _ptr(pw, name="pw"), cout, cin,
                                                    _stream(stream)))


def cc_resample_up2_fused(x, pw, bias, skip, out, hist: int = 0, temporal: bool = False, stream=None) -> None:
    n, d2, h2, w2, cout = out.shape
    hl, wl = h2 // 2, w2 // 2
    d = d2 // 2 if temporal else d2
    cin = x.shape[-1]
    if h2 != 2 * hl or w2 != 2 * wl or (temporal and d2 != 2 * d) or tuple(x.shape) != (n, d + hist, hl, wl, cin):
        raise ValueError("resample_up2_fused: out must be [N,(2)D,2HL,2WL,Cout] of x [N,D+hist,HL,WL,Cin]")
    taps = 64 if temporal else 48
    if tuple(skip.shape) != (n, d, hl, wl, cout) or bias.numel() != cout or pw.numel() != taps * cout * cin:
        raise ValueError("resample_up2_fused: skip, bias or pw shape mismatch")
    _check(_lib.load().cc_resample_up2_fused(_ptr(x, name="x"), _ptr(pw, name="pw"), _ptr(bias, name="bias"),
                                             _ptr(skip, name="skip"), _ptr(out, name="out"), n, d, hl, wl, cin, cout,
                                             hist, 1 if temporal else 0, _stream(stream)))


# ------------------------------------------------------ per-frame attention --

def cc_attn_ld(hw: int) -> int:
    return _lib.load().cc_attn_ld(hw)


def cc_attn_workspace_bytes(t: int, hw: int) -> int:
    return _lib.load().cc_attn_workspace_bytes(t, hw)


def _rows(t: torch.Tensor, name: str):
    """(T, HW, C, ld) of a [T, HW, C] tensor whose rows may be strided (packed qkv slices)."""
    if t.dim() != 3 or (t.numel() and (t.stride(2) != 1 or t.stride(0) != t.shape[1] * t.stride(1))):
        raise ValueError(f"{name}: expected [T,HW,C] with unit channel stride and frame stride HW*ld")
    if t.device.type != "cuda" or t.dtype != torch.bfloat16:
        raise ValueError(f"{name}: expected a bf16 CUDA tensor")
    return t.shape[0], t.shape[1], t.shape[2], t.stride(1)


def cc_attn_scores(q, k, s, stream=None) -> None:
    t, hw, c, ld_q = _rows(q, "q")
    _, _, _, ld_k = _rows(k, "k")
    if tuple(k.shape) != (t, hw, c) or s.dim() != 3 or s.shape[0] != t or s.shape[1] != hw:
        raise ValueError("attn_scores: shapes do not match")
    _check(_lib.load().cc_attn_scores(q.data_ptr(), k.data_ptr(), _ptr(s, torch.float32, "s"), t, hw, c, ld_q, ld_k,
                                      s.shape[2], _stream(stream)))


def cc_attn_softmax(s, p, hw: int, scale: float, stream=None) -> None:
    t = s.shape[0]
    if s.dim() != 3 or p.dim() != 3 or s.shape[:2] != (t, hw) or p.shape[:2] != (t, hw):
        raise ValueError("attn_softmax: s and p must be [T,HW,ld]")
    _check(_lib.load().cc_attn_softmax(_ptr(s, torch.float32, "s"), _ptr(p, name="p"), t, hw, s.shape[2], p.shape[2],
                                       float(scale), _stream(stream)))


def cc_attn_pv(p, v, o, hw: int, stream=None) -> None:
    t, _, c, ld_v = _rows(v, "v")
    _, _, _, ld_o = _rows(o, "o")
    if p.dim() != 3 or p.shape[:2] != (t, hw):
        raise ValueError("attn_pv: p must be [T,HW,ld]")
    _check(_lib.load().cc_attn_pv(_ptr(p, name="p"), v.data_ptr(), o.data_ptr(), t, hw, c, p.shape[2], ld_v, ld_o,
                                  _stream(stream)))


def cc_attn_frame(q, k, v, o, ws, scale: float | None = None, stream=None) -> None:
    t, hw, c, ld_q = _rows(q, "q")
    _, _, _, ld_k = _rows(k, "k")
    _, _, _, ld_v = _rows(v, "v")
    _, _, _, ld_o = _rows(o, "o")
    if not (tuple(k.shape) == tuple(v.shape) == tuple(o.shape) == (t, hw, c)):
        raise ValueError("attn_frame: q, k, v, o must share [T,HW,C]")
    if scale is None:
        scale = c ** -0.5
    _check(_lib.load().cc_attn_frame(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), t, hw, c, ld_q, ld_k,
                                     ld_v, ld_o, float(scale), _ptr(ws, torch.uint8, "ws"), ws.numel(),
                                     _stream(stream)))


def cc_attn_exp_key_tiles(hw: int) -> int:
    return _lib.load().cc_attn_exp_key_tiles(hw)


def cc_attn_exp_workspace_bytes(t: int, hw: int) -> int:
    return _lib.load().cc_attn_exp_workspace_bytes(t, hw)


def cc_attn_scores_exp(q, k, e, stats, scale: float | None = None, stream=None) -> None:
    """e: bf16 [T, HW, ld]; stats: fp32 [T, HW, key_tiles, 2] (pairs c_t, l_t)."""
    t, hw, c, ld_q = _rows(q, "q")
    _, _, _, ld_k = _rows(k, "k")
    tiles = cc_attn_exp_key_tiles(hw)
    if tuple(k.shape) != (t, hw, c) or e.dim() != 3 or tuple(e.shape[:2]) != (t, hw):
        raise ValueError("attn_scores_exp: shapes do not match")
    if tuple(stats.shape) != (t, hw, tiles, 2):
        raise ValueError(f"attn_scores_exp: stats must be [T,HW,{tiles},2]")
    if scale is None:
        scale = c ** -0.5
    _check(_lib.load().cc_attn_scores_exp(q.data_ptr(), k.data_ptr(), _ptr(e, name="e"),
                                          _ptr(stats, torch.float32, "stats"), t, hw, c, ld_q, ld_k, e.shape[2],
                                          float(scale), _stream(stream)))


def cc_attn_exp_rescale(e, stats, hw: int, stream=None) -> None:
    t = e.shape[0]
    if e.dim() != 3 or tuple(e.shape[:2]) != (t, hw) or tuple(stats.shape) != (t, hw, cc_attn_exp_key_tiles(hw), 2):
        raise ValueError("attn_exp_rescale: e must be [T,HW,ld] and stats [T,HW,key_tiles,2]")
    _check(_lib.load().cc_attn_exp_rescale(_ptr(e, name="e"), _ptr(stats, torch.float32, "stats"), t, hw, e.shape[2],
                                           _stream(stream)))


def cc_attn_pv_exp(e, stats, v, o, stream=None) -> None:
    t, hw, c, ld_v = _rows(v, "v")
    _, _, _, ld_o = _rows(o, "o")
    if e.dim() != 3 or tuple(e.shape[:2]) != (t, hw) or tuple(stats.shape) != (t, hw, cc_attn_exp_key_tiles(hw), 2):
        raise ValueError("attn_pv_exp: e must be [T,HW,ld] and stats [T,HW,key_tiles,2]")
    _check(_lib.load().cc_attn_pv_exp(_ptr(e, name="e"), _ptr(stats, torch.float32, "stats"), v.data_ptr(),
                                      o.data_ptr(), t, hw, c, e.shape[2], ld_v, ld_o, _stream(stream)))


def cc_attn_frame_exp(q, k, v, o, ws, scale: float | None = None, stream=None) -> None:
    t, hw, c, ld_q = _rows(q, "q")
    _, _, _, ld_k = _rows(k, "k")
    _, _, _, ld_v = _rows(v, "v")
    _, _, _, ld_o = _rows(o, "o")
    if not (tuple(k.shape) == tuple(v.shape) == tuple(o.shape) == (t, hw, c)):
        raise ValueError("attn_frame_exp: q, k, v, o must share [T,HW,C]")
    if scale is None:
        scale = c ** -0.5
    _check(_lib.load().cc_attn_frame_exp(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), t, hw, c, ld_q, ld_k,
                                         ld_v, ld_o, float(scale), _ptr(ws, torch.uint8, "ws"), ws.numel(),
                                         _stream(stream)))


def cc_attn_scores_stats(q, k, stats, scale: float | None = None, stream=None) -> None:
    """stats: fp32 [T, HW, key_tiles, 2] (pairs c_t, l_t); E is not written."""
    t, hw, c, ld_q = _rows(q, "q")
    _, _, _, ld_k = _rows(k, "k")
    tiles = cc_attn_exp_key_tiles(hw)
    if tuple(k.shape) != (t, hw, c) or tuple(stats.shape) != (t, hw, tiles, 2):
        raise ValueError(f"attn_scores_stats: k must be [T,HW,C] and stats [T,HW,{tiles},2]")
    if scale is None:
        scale = c ** -0.5
    _check(_lib.load().cc_attn_scores_stats(q.data_ptr(), k.data_ptr(), _ptr(stats, torch.float32, "stats"), t, hw,
                                            c, ld_q, ld_k, float(scale), _stream(stream)))


def cc_attn_fused_workspace_bytes(t: int, hw: int) -> int:
    return _lib.load().cc_attn_fused_workspace_bytes(t, hw)


def cc_attn_frame_fused(q, k, v, o, ws, scale: float | None = None, stream=None) -> None:
    """Attention with the numerators kept on chip (statistics pass + one kernel)."""
    t, hw, c, ld_q = _rows(q, "q")
    _, _, _, ld_k = _rows(k, "k")
    _, _, _, ld_v = _rows(v, "v")
    _, _, _, ld_o = _rows(o, "o")
    if not (tuple(k.shape) == tuple(v.shape) == tuple(o.shape) == (t, hw, c)):
        raise ValueError("attn_frame_fused: q, k, v, o must share [T,HW,C]")
    if scale is None:
        scale = c ** -0.5
    _check(_lib.load().cc_attn_frame_fused(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), t, hw, c, ld_q,
                                           ld_k, ld_v, ld_o, float(scale), _ptr(ws, torch.uint8, "ws"), ws.numel(),
                                           _stream(stream)))


# -------------------------------------------------------------- output head --

def cc_head_prepare(w, wp, stream=None) -> None:
    cin = w.shape[1]
    if tuple(w.shape) != (HEAD_COUT, cin, 3, 3, 3) or wp.numel() != 3 * HEAD_G_CH * cin:
        raise ValueError("head_prepare: w must be [12,Cin,3,3,3] and wp hold 3*112*Cin elements")
    _check(_lib.load().cc_head_prepare(_ptr(w, name="w"), _ptr(wp, name="wp"), cin, _stream(stream)))


def cc_head_workspace_bytes(n: int, d: int, h: int, w: int) -> int:
    return _lib.load().cc_head_workspace_bytes(n, d, h, w)


def cc_head_temporal(x, wp, g, hist: int = 0, stream=None) -> None:
    n, d, h, w, ch = g.shape
    cin = x.shape[-1]
    if ch != HEAD_G_CH or tuple(x.shape) != (n, d + hist, h, w, cin) or wp.numel() != 3 * HEAD_G_CH * cin:
        raise ValueError("head_temporal: g must be [N,D,H,W,112] matching x and wp")
    _check(_lib.load().cc_head_temporal(_ptr(x, name="x"), _ptr(wp, name="wp"), _ptr(g, name="g"), n, d, h, w, cin,
                                        hist, _stream(stream)))


def cc_head_stencil(g, bias, out, stream=None) -> None:
    n, d, h, w, c = out.shape
    if c != HEAD_COUT or tuple(g.shape) != (n, d, h, w, HEAD_G_CH) or bias.numel() != HEAD_COUT:
        raise ValueError("head_stencil: g must be [N,D,H,W,112] and out [N,D,H,W,12]")
    _check(_lib.load().cc_head_stencil(_ptr(g, name="g"), _ptr(bias, name="bias"), _ptr(out, name="out"), n, d, h, w,
                                       _stream(stream)))


def cc_head_out(x, wp, bias, out, ws, hist: int = 0, stream=None) -> None:
    n, d, h, w, c = out.shape
    cin = x.shape[-1]
    if c != HEAD_COUT or tuple(x.shape) != (n, d + hist, h, w, cin) or bias.numel() != HEAD_COUT:
        raise ValueError("head_out: out must be [N,D,H,W,12] of x [N,D+hist,H,W,Cin]")
    _check(_lib.load().cc_head_out(_ptr(x, name="x"), _ptr(wp, name="wp"), _ptr(bias, name="bias"),
                                   _ptr(out, name="out"), n, d, h, w, cin, hist, _ptr(ws, torch.uint8, "ws"),
                                   ws.numel(), _stream(stream)))


def cc_head_out_fused(x, wp, bias, out, hist: int = 0, stream=None) -> None:
    """The whole head in one kernel (g kept in fp32 on chip), no workspace."""
    n, d, h, w, c = out.shape
    cin = x.shape[-1]
    if c != HEAD_COUT or tuple(x.shape) != (n, d + hist, h, w, cin) or bias.numel() != HEAD_COUT:
        raise ValueError("head_out_fused: out must be [N,D,H,W,12] of x [N,D+hist,H,W,Cin]")
    _check(_lib.load().cc_head_out_fused(_ptr(x, name="x"), _ptr(wp, name="wp"), _ptr(bias, name="bias"),
                                         _ptr(out, name="out"), n, d, h, w, cin, hist, _stream(stream)))


def cc_head_out_noalloc(x, wp, bias, out, hist: int = 0, stream=None) -> None:
    """cc_head_out without a workspace, for callers that cannot allocate device
    memory: g lives in the library's fixed 64 MiB static scratch (at most
    299,593 output positions per call; calls that overlap on the GPU race on
    it, so keep them on one stream)."""
    n, d, h, w, c = out.shape
    cin = x.shape[-1]
    if c != HEAD_COUT or tuple(x.shape) != (n, d + hist, h, w, cin) or bias.numel() != HEAD_COUT:
        raise ValueError("head_out_noalloc: out must be [N,D,H,W,12] of x [N,D+hist,H,W,Cin]")
    _check(_lib.load().cc_head_out_noalloc(_ptr(x, name="x"), _ptr(wp, name="wp"), _ptr(bias, name="bias"),
                                           _ptr(out, name="out"), n, d, h, w, cin, hist, _stream(stream)))


# ------------------------------------------------- norms with an activation --

ACTS = {"none": 0, "silu": 1}  # CC_ACT_*


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act: expected one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


def _arg(t, dtype, name: str, dev: int) -> int | None:
    """_ptr for a tensor on the current device `dev`, whose stream the call uses. A call's host time counts where its
    tensors are small, so the tests that all pass come first (a tensor off the GPU has device -1)."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype and t.is_contiguous():
        return t.data_ptr()
    _ptr(t, dtype, name)  # says what is wrong with it, unless it is
    raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _last_rows(t, dtype, name: str, dev: int):
    """(pointer, rows, C, ld) of a [..., C] tensor whose rows are C channels next to each other at one stride `ld`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.get_device() != dev or t.dtype is not dtype:
        if not t.is_cuda:
            raise ValueError(f"{name}: must be a CUDA tensor")
        if t.dtype is not dtype:
            raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")
    rows, c, ld = _row_layout(t, name)
    if rows > INT_MAX or c > INT_MAX:
        _too_large(name, rows, c)
    return t.data_ptr(), rows, c, ld


INT_MAX = 0x7FFFFFFF  # sizes are passed as C ints, of which ctypes keeps the low 32 bits without a word


def _too_large(name: str, *sizes):
    raise ValueError(f"{name}: sizes {sizes} must be at most {INT_MAX}")


def _row_layout(t, name: str):
    """(rows, C, ld)"""
    shape = t.shape
    if not shape:
        raise ValueError(f"{name}: expected [..., C]")
    c = shape[-1]
    if t.is_contiguous():
        return (shape[0] if len(shape) == 2 else t.numel() // c if c else 0), c, c
    if t.stride(-1) != 1 and c > 1:
        raise ValueError(f"{name}: channels must be contiguous")
    rows, ld = 1, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != ld * rows:
            raise ValueError(f"{name}: rows must lie at one stride")
        rows *= size
    return rows, c, c if ld is None else ld


def _scales_of(scales, t, rows: int, c: int, name: str) -> None:
    """`scales` has a value for each row and 128 channels of t [..., C], whose leading sizes it shares. (Up to two
    dimensions their number tells; more are compared.)"""
    blocks, dims = (c + 127) // 128, t.dim()
    if (scales.dim() != dims or scales.shape[-1] != blocks or scales.numel() != rows * blocks
            or (dims > 2 and scales.shape[:-1] != t.shape[:-1])):
        raise ValueError(f"{name} must be [..., {blocks}] for {tuple(t.shape)}, got {tuple(scales.shape)}")


def cc_group_norm_workspace_bytes(n: int, p: int, c: int, groups: int) -> int:
    if n > INT_MAX or p > INT_MAX or c > INT_MAX or groups > INT_MAX:
        return 0  # as for other sizes that the norm refuses
    return _lib.load().cc_group_norm_workspace_bytes(n, p, c, groups)


def _group_norm_sizes(x, gamma, beta, y, groups: int):
    shape = x.shape
    if len(shape) < 2 or shape != y.shape:
        raise ValueError(f"group_norm_act: x and y must share [N,...,C], got {tuple(shape)} and {tuple(y.shape)}")
    n, c = shape[0], shape[-1]
    if (gamma is not None and gamma.numel() != c) or (beta is not None and beta.numel() != c):
        raise ValueError("group_norm_act: gamma and beta must hold C elements")
    p = shape[1] if len(shape) == 3 else math.prod(shape[1:-1])
    if n > INT_MAX or p > INT_MAX or c > INT_MAX or abs(groups) > INT_MAX:
        _too_large("group_norm_act", n, p, c, groups)
    return n, p, c


def cc_group_norm_act(x, gamma, beta, y, groups: int, ws, eps: float = 1e-6, act: str = "silu", stream=None) -> None:
    """Group norm of x [N, ..., C] over everything but N (view [N, D, H, W, C] as [N*D, H, W, C] for a norm per
    frame) and an activation ("silu" or "none"). gamma, beta: [C] or None."""
    n, p, c = _group_norm_sizes(x, gamma, beta, y, groups)
    dev, bf16 = torch.cuda.current_device(), torch.bfloat16
    _check(_lib.load().cc_group_norm_act(
        _arg(x, bf16, "x", dev), _arg(gamma, bf16, "gamma", dev), _arg(beta, bf16, "beta", dev),
        _arg(y, bf16, "y", dev), n, p, c, groups, eps, _act(act), _arg(ws, torch.uint8, "ws", dev),
        0 if ws is None else ws.numel(), _raw_stream(stream, dev)))


def cc_group_norm_act_fp8(x, gamma, beta, y, scales, groups: int, ws, eps: float = 1e-6, act: str = "silu",
                          stream=None) -> None:
    """The same, written as e4m3 (y, torch.float8_e4m3fn) with scales [N, ..., ceil(C/128)]."""
    n, p, c = _group_norm_sizes(x, gamma, beta, y, groups)
    _scales_of(scales, x, n * p, c, "group_norm_act_fp8: scales")
    dev, bf16 = torch.cuda.current_device(), torch.bfloat16
    _check(_lib.load().cc_group_norm_act_fp8(
        _arg(x, bf16, "x", dev), _arg(gamma, bf16, "gamma", dev), _arg(beta, bf16, "beta", dev),
        _arg(y, torch.float8_e4m3fn, "y", dev), _arg(scales, torch.float32, "scales", dev), n, p, c, groups, eps,
        _act(act), _arg(ws, torch.uint8, "ws", dev), 0 if ws is None else ws.numel(), _raw_stream(stream, dev)))


def cc_rms_norm_act(x, gamma, y, eps: float = 1e-6, act: str = "silu", stream=None) -> None:
    """RMS norm over the channels of x [..., C] (rows may be strided) and an activation. gamma: [C] or None."""
    dev, bf16 = torch.cuda.current_device(), torch.bfloat16
    px, rows, c, ld = _last_rows(x, bf16, "x", dev)
    if x.shape != y.shape or (gamma is not None and gamma.numel() != c):
        raise ValueError("rms_norm_act: x and y must share [...,C] and gamma hold C elements")
    _check(_lib.load().cc_rms_norm_act(px, _arg(gamma, bf16, "gamma", dev), _arg(y, bf16, "y", dev), rows, c, ld, eps,
                                       _act(act), _raw_stream(stream, dev)))


def cc_rms_norm_act_fp8(x, gamma, y, scales, eps: float = 1e-6, act: str = "silu", stream=None) -> None:
    """The same, written as e4m3 (y, torch.float8_e4m3fn) with scales [..., ceil(C/128)]."""
    dev, bf16 = torch.cuda.current_device(), torch.bfloat16
    px, rows, c, ld = _last_rows(x, bf16, "x", dev)
    if x.shape != y.shape or (gamma is not None and gamma.numel() != c):
        raise ValueError("rms_norm_act_fp8: x and y must share [...,C] and gamma hold C elements")
    _scales_of(scales, x, rows, c, "rms_norm_act_fp8: scales")
    _check(_lib.load().cc_rms_norm_act_fp8(
        px, _arg(gamma, bf16, "gamma", dev), _arg(y, torch.float8_e4m3fn, "y", dev),
        _arg(scales, torch.float32, "scales", dev), rows, c, ld, eps, _act(act), _raw_stream(stream, dev)))


# ------------------------------------- product in 8 bits with block scales --

def cc_fp8_quantize(x, y, scales, stream=None) -> None:
    """bf16 rows x [..., C] (rows may be strided) to e4m3 y with scales [..., ceil(C/128)]."""
    dev = torch.cuda.current_device()
    px, rows, c, ld = _last_rows(x, torch.bfloat16, "x", dev)
    if x.shape != y.shape:
        raise ValueError("fp8_quantize: x and y must share [...,C]")
    _scales_of(scales, x, rows, c, "fp8_quantize: scales")
    _check(_lib.load().cc_fp8_quantize(px, _arg(y, torch.float8_e4m3fn, "y", dev),
                                       _arg(scales, torch.float32, "scales", dev), rows, c, ld,
                                       _raw_stream(stream, dev)))


def cc_gemm_fp8_prepare(w, wq, sw, stream=None) -> None:
    """Weights w [N, K] (a 1x1x1 convolution's [Cout, Cin]) to e4m3 wq with scales sw [ceil(N/128), ceil(K/128)]."""
    if w.dim() != 2 or w.shape != wq.shape or tuple(sw.shape) != tuple((s + 127) // 128 for s in w.shape):
        raise ValueError("gemm_fp8_prepare: wq must be [N,K] and sw [ceil(N/128),ceil(K/128)] of w [N,K]")
    if w.shape[0] > INT_MAX or w.shape[1] > INT_MAX:
        _too_large("gemm_fp8_prepare", *w.shape)
    dev = torch.cuda.current_device()
    _check(_lib.load().cc_gemm_fp8_prepare(
        _arg(w, torch.bfloat16, "w", dev), _arg(wq, torch.float8_e4m3fn, "wq", dev),
        _arg(sw, torch.float32, "sw", dev), w.shape[0], w.shape[1], _raw_stream(stream, dev)))


def cc_gemm_fp8(a, sa, wq, sw, bias, res, out, stream=None) -> None:
    """out [..., N] = a [..., K] wq^T with the block scales, plus bias [N] and res [..., N] (or None). out and res
    may be rows at a stride (a slice of packed qkv)."""
    dev, bf16, f8, f32 = torch.cuda.current_device(), torch.bfloat16, torch.float8_e4m3fn, torch.float32
    po, m, n, ld_out = _last_rows(out, bf16, "out", dev)
    dims = a.dim()
    k = a.shape[-1] if dims else 0
    if (dims != out.dim() or a.numel() != m * k or wq.shape != (n, k)
            or (dims > 2 and a.shape[:-1] != out.shape[:-1])):
        raise ValueError(f"gemm_fp8: a must be [...,K] and wq [N,K] of out [...,N], got {tuple(a.shape)}, "
                         f"{tuple(wq.shape)} and {tuple(out.shape)}")
    if k > INT_MAX:
        _too_large("gemm_fp8", m, n, k)
    _scales_of(sa, a, m, k, "gemm_fp8: sa")
    if sw.shape != ((n + 127) // 128, (k + 127) // 128):
        raise ValueError("gemm_fp8: sw must be [ceil(N/128),ceil(K/128)]")
    if bias is not None and bias.numel() != n:
        raise ValueError("gemm_fp8: bias must hold N elements")
    pr, ld_res = None, n
    if res is not None:
        if res.shape != out.shape:
            raise ValueError("gemm_fp8: res must have out's shape")
        pr, _, _, ld_res = _last_rows(res, bf16, "res", dev)
    _check(_lib.load().cc_gemm_fp8(_arg(a, f8, "a", dev), _arg(sa, f32, "sa", dev), _arg(wq, f8, "wq", dev),
                                   _arg(sw, f32, "sw", dev), _arg(bias, bf16, "bias", dev), pr, po, m, n, k, ld_res,
                                   ld_out, _raw_stream(stream, dev)))


# ---------------------------- heads: norm, rotation, a paged cache, attention --

ROT_STYLES = {"pairs": 0, "halves": 1}  # CC_ROT_*


def _on(t, dtype, name: str, dev: int) -> None:
    """`t` is a tensor of this type on the current device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")


def _head_rows(t, name: str, dev: int):
    """(pointer, shape, rows, ld) of a bf16 tensor [..., heads, D] whose rows hold their heads side by side and lie at
    one stride `ld`. (What usually comes, rows at a stride, is told first.)"""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.get_device() == dev:
        shape, strides = t.shape, t.stride()
        if len(shape) == 3:
            rows, heads, d = shape
            if rows > 1 and strides[2] == 1 and strides[1] == d and rows | heads | d <= INT_MAX:
                return t.data_ptr(), shape, rows, strides[0]
        elif len(shape) == 4:
            n, rows, heads, d = shape
            if rows > 1 and strides[3] == 1 and strides[2] == d and strides[0] == rows * strides[1] \
                    and n * rows | heads | d <= INT_MAX:
                return t.data_ptr(), shape, n * rows, strides[1]
    else:
        _on(t, torch.bfloat16, name, dev)
        shape, strides = t.shape, t.stride()
    if len(shape) < 3:
        raise ValueError(f"{name}: expected [..., heads, D]")
    heads, d = shape[-2:]
    if (strides[-1] != 1 and d > 1) or (strides[-2] != d and heads > 1):
        raise ValueError(f"{name}: a row's heads and channels must be contiguous")
    rows, ld = 1, None
    for size, stride in zip(reversed(shape[:-2]), reversed(strides[:-2])):
        if size != 1:
            if ld is None:
                ld = stride
            elif stride != ld * rows and rows:
                raise ValueError(f"{name}: rows must lie at one stride")
            rows *= size
    if rows > INT_MAX or heads > INT_MAX or d > INT_MAX:
        _too_large(name, rows, heads, d)
    return t.data_ptr(), shape, rows, heads * d if ld is None else ld


def _rotation(rot, pos, rows: int, name: str, dev: int):
    """(pointer of rot, positions, rd, pointer of pos)"""
    prot, positions, rd = None, 0, 0
    if rot is not None:
        prot = _arg(rot, torch.float32, "rot", dev)
        shape = rot.shape
        if len(shape) != 3 or shape[2] != 2:
            raise ValueError(f"{name}: rot must be [positions, rd/2, 2], got {tuple(shape)}")
        positions, rd = shape[0], 2 * shape[1]
        if positions > INT_MAX or rd > INT_MAX:
            _too_large(name, positions, rd)
    if pos is None:
        return prot, positions, rd, None
    if pos.numel() != rows:
        raise ValueError(f"{name}: pos must hold a position for each of {rows} rows")
    return prot, positions, rd, _arg(pos, torch.int32, "pos", dev)


def _style(style: str) -> int:
    if style not in ROT_STYLES:
        raise ValueError(f"style: expected one of {sorted(ROT_STYLES)}, got {style!r}")
    return ROT_STYLES[style]


def _gamma(gamma, d: int, name: str, dev: int):
    if gamma is None:
        return None
    if gamma.numel() != d:
        raise ValueError(f"{name} must hold D elements")
    return _arg(gamma, torch.bfloat16, name, dev)


def cc_qk_norm_rope(q, k, gamma_q, gamma_k, rot, pos, q_out, k_out, eps: float = 1e-6, style: str = "pairs",
                    stream=None) -> None:
    """RMS norm over the channels of every head of q [..., heads, D] and k [..., kv_heads, D] (rows may be strided;
    either may be None with its output) and the rotation of the first rd channels by pos[row] (None: the row's number)
    as rot [positions, rd/2, 2], fp32 (cos, sin), says (None: no rotation). style: "pairs" or "halves"."""
    dev = torch.cuda.current_device()
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (q is None and k is None):
        raise ValueError("qk_norm_rope: q and k come with their outputs, and one of them must be there")
    pq = pk = pqo = pko = None
    heads = kv_heads = ld_q = ld_k = ld_qo = ld_ko = 0
    if k is not None:
        pk, shape, rows, ld_k = _head_rows(k, "k", dev)
        pko, out, _, ld_ko = _head_rows(k_out, "k_out", dev)
        if out != shape:
            raise ValueError("qk_norm_rope: k_out must have k's shape")
        kv_heads, d = shape[-2:]
    if q is not None:
        pq, shape_q, rows, ld_q = _head_rows(q, "q", dev)
        pqo, out, _, ld_qo = _head_rows(q_out, "q_out", dev)
        heads, d = shape_q[-2:]
        if out != shape_q or (k is not None and (shape_q[:-2] != shape[:-2] or shape[-1] != d)):
            raise ValueError("qk_norm_rope: q, k and q_out must share rows and D")
    prot, positions, rd, ppos = _rotation(rot, pos, rows, "qk_norm_rope", dev)
    _check(_lib.load().cc_qk_norm_rope(
        pq, pk, _gamma(gamma_q, d, "gamma_q", dev), _gamma(gamma_k, d, "gamma_k", dev), prot, ppos, pqo, pko, rows,
        heads, kv_heads, d, rd, positions, ld_q, ld_k, ld_qo, ld_ko, eps, _style(style), _raw_stream(stream, dev)))


def _paged(k_cache, v_cache, q_offsets, kv_lens, page_table, name: str, dev: int):
    """Pointers, sizes and strides of a cache [pages, page_size, kv_heads, D] and of a step's plan."""
    bf16, i32 = torch.bfloat16, torch.int32
    for cache in (k_cache, v_cache):
        if not isinstance(cache, torch.Tensor) or cache.dtype is not bf16 or cache.get_device() != dev:
            _on(cache, bf16, "k_cache" if cache is k_cache else "v_cache", dev)
    shape, ks, vs = k_cache.shape, k_cache.stride(), v_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"{name}: k_cache and v_cache must share [pages, page_size, kv_heads, D]")
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError(f"{name}: a cached head's channels must be contiguous")
    plan = (_arg(q_offsets, i32, "q_offsets", dev), _arg(kv_lens, i32, "kv_lens", dev),
            _arg(page_table, i32, "page_table", dev))
    table = page_table.shape
    if len(table) != 2 or kv_lens.numel() != table[0] or q_offsets.numel() != table[0] + 1:
        raise ValueError(f"{name}: q_offsets must be [seqs + 1], kv_lens [seqs] and page_table [seqs, max_pages]")
    pages, page_size, kv_heads, d = shape
    seqs, max_pages = table
    if pages | page_size | kv_heads | d | seqs | max_pages > INT_MAX:
        _too_large(name, *shape, *table)
    return k_cache.data_ptr(), v_cache.data_ptr(), plan, (seqs, max_pages, pages, page_size), kv_heads, d, ks[:3] + vs[:3]


def cc_qk_norm_rope_append(q, k, v, gamma_q, gamma_k, rot, pos, q_out, k_cache, v_cache, q_offsets, kv_lens,
                           page_table, eps: float = 1e-6, style: str = "pairs", stream=None) -> None:
    """cc_qk_norm_rope of the rows of a step's plan, with the keys and the values v [rows, kv_heads, D] written to
    their tokens' slots in k_cache and v_cache [pages, page_size, kv_heads, D] (any strides). Sequence b owns rows
    q_offsets[b] .. q_offsets[b + 1] - 1, the newest of its kv_lens[b] tokens; page_table [seqs, max_pages]. All three
    are int32 on the GPU. pos None: a row's position is its token's in its sequence."""
    dev = torch.cuda.current_device()
    pq, shape, rows, ld_q = _head_rows(q, "q", dev)
    pqo, out, _, ld_qo = _head_rows(q_out, "q_out", dev)
    pk, shape_k, _, ld_k = _head_rows(k, "k", dev)
    pv, shape_v, _, ld_v = _head_rows(v, "v", dev)
    pkc, pvc, plan, sizes, kv_heads, d, strides = _paged(k_cache, v_cache, q_offsets, kv_lens, page_table,
                                                         "qk_norm_rope_append", dev)
    if (out != shape or shape_k[:-2] != shape[:-2] or shape_k != shape_v or shape[-1] != d or shape_k[-1] != d
            or shape_k[-2] != kv_heads):
        raise ValueError("qk_norm_rope_append: q, k, v and the cache must share rows, heads and D")
    prot, positions, rd, ppos = _rotation(rot, pos, rows, "qk_norm_rope_append", dev)
    _check(_lib.load().cc_qk_norm_rope_append(
        pq, pk, pv, _gamma(gamma_q, d, "gamma_q", dev), _gamma(gamma_k, d, "gamma_k", dev), prot, ppos, pqo, pkc, pvc,
        *plan, rows, *sizes, shape[-2], kv_heads, d, rd, positions, ld_q, ld_k, ld_v, ld_qo, *strides, eps,
        _style(style), _raw_stream(stream, dev)))


def cc_attn_paged_workspace_bytes(rows: int, seqs: int, heads: int, kv_heads: int, d: int) -> int:
    if max(rows, seqs, heads, kv_heads, d) > INT_MAX:
        return 0  # as for other sizes that the call refuses
    return _lib.load().cc_attn_paged_workspace_bytes(rows, seqs, heads, kv_heads, d)


def cc_attn_paged(q, k_cache, v_cache, o, q_offsets, kv_lens, page_table, ws, scale: float | None = None,
                  causal_block: int = 1, stream=None) -> None:
    """Attention of a plan's rows q [rows, heads, D] over the cache (as for cc_qk_norm_rope_append). A token sees those
    up to the end of its own block of `causal_block` new tokens (1: up to itself; 0: all of its sequence)."""
    dev = torch.cuda.current_device()
    pq, shape, rows, ld_q = _head_rows(q, "q", dev)
    po, out, _, ld_o = _head_rows(o, "o", dev)
    pk, pv, plan, sizes, kv_heads, d, strides = _paged(k_cache, v_cache, q_offsets, kv_lens, page_table, "attn_paged", dev)
    if out != shape or shape[-1] != d:
        raise ValueError("attn_paged: q, o and the cache must share rows and D")
    if abs(causal_block) > INT_MAX:
        _too_large("attn_paged", causal_block)
    _check(_lib.load().cc_attn_paged(
        pq, pk, pv, po, *plan, rows, *sizes, shape[-2], kv_heads, d, ld_q, ld_o, *strides,
        d ** -0.5 if scale is None else scale, causal_block, _arg(ws, torch.uint8, "ws", dev),
        0 if ws is None else ws.numel(), _raw_stream(stream, dev)))


def cc_attn_cross_workspace_bytes(n: int, lq: int, lk: int, heads: int, kv_heads: int, d: int) -> int:
    if max(n, lq, lk, heads, kv_heads, d) > INT_MAX:
        return 0
    return _lib.load().cc_attn_cross_workspace_bytes(n, lq, lk, heads, kv_heads, d)


def cc_attn_cross(q, k, v, o, kv_lens, ws, scale: float | None = None, stream=None) -> None:
    """Attention of q [N, Lq, heads, D] to an encoder's k, v [N, Lk, kv_heads, D] (rows may be strided), of which
    kv_lens [N] (int32 on the GPU; None: all) count."""
    dev = torch.cuda.current_device()
    pq, shape, _, ld_q = _head_rows(q, "q", dev)
    pk, shape_k, _, ld_k = _head_rows(k, "k", dev)
    pv, shape_v, _, ld_v = _head_rows(v, "v", dev)
    po, out, _, ld_o = _head_rows(o, "o", dev)
    if len(shape) != 4 or len(shape_k) != 4 or shape[0] != shape_k[0] or out != shape or shape_v != shape_k \
            or shape_k[3] != shape[3]:
        raise ValueError("attn_cross: q and o must be [N,Lq,heads,D], k and v [N,Lk,kv_heads,D]")
    n, lq, heads, d = shape
    if kv_lens is not None and kv_lens.numel() != n:
        raise ValueError("attn_cross: kv_lens must hold N values")
    _check(_lib.load().cc_attn_cross(
        pq, pk, pv, po, _arg(kv_lens, torch.int32, "kv_lens", dev), n, lq, shape_k[1], heads, shape_k[2], d, ld_q,
        ld_k, ld_v, ld_o, d ** -0.5 if scale is None else scale, _arg(ws, torch.uint8, "ws", dev),
        0 if ws is None else ws.numel(), _raw_stream(stream, dev)))


# -------------------------------------------------------- result read-back --

def cc_copy_to_host(dst: torch.Tensor, src: torch.Tensor, ctas: int = 8, stream=None) -> None:
    """Copies the CUDA tensor `src` into the pinned CPU tensor `dst` (same
    number of bytes, both contiguous) with a copy kernel of `ctas` CTAs."""
    if not isinstance(dst, torch.Tensor) or not isinstance(src, torch.Tensor):
        raise TypeError("copy_to_host: expected torch tensors")
    if dst.device.type != "cpu" or not dst.is_pinned():
        raise ValueError("copy_to_host: dst must be a pinned CPU tensor")
    if src.device.type != "cuda":
        raise ValueError("copy_to_host: src must be a CUDA tensor")
    if not (dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("copy_to_host: tensors must be contiguous")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("copy_to_host: dst and src hold different numbers of bytes")
    _check(_lib.load().cc_copy_to_host(dst.data_ptr(), src.data_ptr(), nbytes, int(ctas), _stream(stream)))


# ------------------------------------------------------------- self tests --

def cc_debug_im2col_tile(x, tile, lower, upper, c0, start, offsets, stream=None) -> None:
    n, d_in, h, w, c = x.shape
    if tile.numel() != 128 * 64:
        raise ValueError("debug_im2col_tile: tile must hold 128*64 elements")
    _check(_lib.load().cc_debug_im2col_tile(_ptr(x, name="x"), _ptr(tile, name="tile"), n, d_in, h, w, c, *lower,
                                            *upper, c0, *start, *offsets, _stream(stream)))


def cc_debug_wait_timeout(limit_ns: int, stream=None) -> None:
    _check(_lib.load().cc_debug_wait_timeout(int(limit_ns), _stream(stream)))


def cc_debug_conv_bad_tile_order(x, wp, y, entry: int, stream=None) -> None:
    n, d, h, w, cout = y.shape
    cin = x.shape[-1]
    if tuple(x.shape) != (n, d, h, w, cin) or wp.numel() != 27 * cout * cin:
        raise ValueError("debug_conv_bad_tile_order: x must be [N,D,H,W,Cin] of y and wp hold 27*Cout*Cin elements")
    _check(_lib.load().cc_debug_conv_bad_tile_order(_ptr(x, name="x"), _ptr(wp, name="wp"), _ptr(y, name="y"), n, d,
                                                    h, w, cin, cout, int(entry), _stream(stream)))
