"""B200-native decode-time latent attention for looped (weight-tied) Transformers.

Thin Python binding over the C ABI in ``include/lla.h`` (``liblla.so``): the
functions below only turn torch tensors into pointers, sizes and strides and
call the library entry points of the same names.  Every step of the
computation runs in the library's CUDA kernels; there is no CPU path.  Tensors
must be CUDA tensors; PyTorch provides device memory and streams only.

Entry points (names as in the C ABI):

* ``lla_write_latents``  -- HLA latent writer (eq. 2), LLA per-head and LLA-2D
  encoders; appends rows to a caller-owned latent cache.
* ``lla_decode_attn``    -- LLA reconstruct-on-read decode attention.
* ``hla_decode_attn``    -- absorbed latent read: HLA (eqs. 3-4) and LLA-D.
* ``lla_kv8_write``, ``lla_kv8_attn``, ``lla_kv8_evict`` -- an 8-bit K/V cache
  with a scale for each block of tokens and head: its writer, the attention
  that reads it beside the exact window, eviction by accumulated weight.
"""

import ctypes
import struct

from . import _abi
from ._abi import (LLA_BF16, LLA_ERR_CUDA, LLA_F32, LLA_FP8_E4M3, LLA_KV8_E4M3, LLA_KV8_I8,  # noqa: F401
                   LLA_WRITE_FOLDED, LLA_WRITE_HLA, LLA_WRITE_PERHEAD, LibraryMissing)

__all__ = [
    "LLAError", "lla_status_str", "lla_abi_version",
    "lla_write_latents", "lla_write_workspace_bytes",
    "lla_decode_attn", "lla_decode_workspace_bytes",
    "hla_decode_attn", "hla_decode_workspace_bytes",
    "lla_kv8_write", "lla_kv8_attn", "lla_kv8_attn_workspace_bytes",
    "lla_kv8_evict", "lla_kv8_evict_workspace_bytes",
    "LLA_WRITE_HLA", "LLA_WRITE_PERHEAD", "LLA_WRITE_FOLDED",
]


class LLAError(RuntimeError):
    """A non-zero lla_status returned by the library."""

    def __init__(self, status, where):
        self.status = status
        msg = f"{where}: status {status} ({lla_status_str(status)})"
        self.cuda_error = None
        if status == LLA_ERR_CUDA:
            self.cuda_error = lib().lla_last_cuda_error()
            msg += f": {lib().lla_cuda_error_name(self.cuda_error).decode()} ({self.cuda_error})"
        super().__init__(msg)


def lib():
    return _abi.load()


def lla_status_str(status):
    return lib().lla_status_str(int(status)).decode()


def lla_abi_version():
    return lib().lla_abi_version()


# ---------------------------------------------------------------- helpers --
def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return LLA_F32
    if t.dtype == torch.bfloat16:
        return LLA_BF16
    if t.dtype == torch.uint8:
        return LLA_FP8_E4M3          # byte rows: e4m3 codes, then the two fp32 scales and 8 zero bytes
    raise TypeError(f"unsupported dtype {t.dtype}; use float32, bfloat16 or uint8 (fp8 rows)")


FP8_ROW_EXTRA = 16   # bytes after the codes of an fp8 row: s^K, s^V (fp32), 8 zero bytes


def _row_width(t):
    """Elements of one latent row: the codes only, for fp8 byte rows."""
    return t.shape[-1] - (FP8_ROW_EXTRA if t.dtype == _torch().uint8 else 0)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("every tensor must be a CUDA tensor (this library has no CPU path)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors are on different devices")
    if dev is None:
        raise ValueError("no tensor given")
    return dev


def _dense_inner(t, ndim_inner, name):
    """Check that the last ``ndim_inner`` axes of t are dense row-major."""
    exp = 1
    for ax in range(t.dim() - 1, t.dim() - 1 - ndim_inner, -1):
        if t.shape[ax] != 1 and t.stride(ax) != exp:
            raise ValueError(f"{name}: inner axes must be dense (axis {ax} stride {t.stride(ax)}, want {exp})")
        exp *= t.shape[ax]


def _stream_handle(stream, device):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _scratch(nbytes, device, stream):
    """A call's scratch, taken from the allocator's blocks of the stream that the call runs on: whoever had the block
    before or gets it next is ordered with the call by that stream."""
    torch = _torch()
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _workspace(nbytes, device, workspace, stream):
    """(address, bytes, tensor) of a call's scratch; the caller holds the tensor until the call is issued."""
    if nbytes == 0:
        return None, 0, None
    if workspace is None:
        workspace = _scratch(nbytes, device, stream)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace too small: {workspace.numel()} < {nbytes} bytes")
    return ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(), workspace


def _call(fn, params, ws, nbytes, stream, where):
    st = fn(ctypes.byref(params), ws, nbytes, stream)
    if st != 0:
        raise LLAError(st, where)


# ----------------------------------------------------------------- writer --
def _write_params(mode, x, xv, E_main, E_1, E_K, E_V, out0, out1, pos0, d_h, r_k, r_v, r_1,
                  rotate_keys, rope_base):
    p = _abi.WriteParams()
    p.mode = mode
    p.pos0 = pos0
    p.rope_base = float(rope_base)
    p.rotate_keys = int(bool(rotate_keys))
    if mode == LLA_WRITE_HLA:
        B, n, T, D = x.shape
        _dense_inner(x, 1, "h")
        p.B, p.n, p.T, p.D, p.H, p.d_h = B, n, T, D, 1, d_h
        p.r_k, p.r_v, p.r_1 = r_k, _row_width(out0) - r_k, _row_width(out1) // 2
        p.out_stride_b, p.out_stride_n = out0.stride(0), out0.stride(1)
        p.out1_stride_b, p.out1_stride_n = out1.stride(0), out1.stride(1)
        p.Ncap = min(out0.shape[1], out1.shape[1])
        _dense_inner(out0, 1, "out0")
        _dense_inner(out1, 1, "out1")
    else:
        B, n, T, H, dh = x.shape
        _dense_inner(x, 2, "k")
        _dense_inner(xv, 2, "v")
        if xv.stride() != x.stride() or xv.shape != x.shape:
            raise ValueError("k and v must have the same shape and strides")
        p.B, p.n, p.T, p.H, p.d_h, p.D = B, n, T, H, dh, 0
        if mode == LLA_WRITE_PERHEAD:
            r = out0.shape[-1]
            p.r_k = p.r_v = r
            _dense_inner(out0, 1, "cK")
            _dense_inner(out1, 1, "cV")
            if out1.stride() != out0.stride():
                raise ValueError("cK and cV must share strides")
            p.out_stride_b, p.out_stride_h, p.out_stride_n = out0.stride(0), out0.stride(1), out0.stride(2)
            p.Ncap = out0.shape[2]
        else:
            p.r_k = E_K.shape[2]
            p.r_v = E_V.shape[2]
            _dense_inner(out0, 1, "lat")
            p.out_stride_b, p.out_stride_n = out0.stride(0), out0.stride(1)
            p.Ncap = out0.shape[1]
    p.x, p.xv = _ptr(x), _ptr(xv)
    p.x_stride_b, p.x_stride_n, p.x_stride_t = x.stride(0), x.stride(1), x.stride(2)
    p.E_main, p.E_1, p.E_K, p.E_V = _ptr(E_main), _ptr(E_1), _ptr(E_K), _ptr(E_V)
    p.out0, p.out1 = _ptr(out0), _ptr(out1)
    p.out_dtype = _dtype_code(out0)
    for t in (x, xv, E_main, E_1, E_K, E_V):
        if t is not None and t.dtype != _torch().float32:
            raise TypeError("writer inputs and codecs are float32")
    for t in (E_main, E_1, E_K, E_V):
        if t is not None and not t.is_contiguous():
            raise ValueError("codec tensors must be contiguous")
    return p


def lla_write_workspace_bytes(mode, **kw):
    p = _write_params(mode, **_write_kw(kw))
    return lib().lla_write_workspace_bytes(ctypes.byref(p))


def _write_kw(kw):
    keys = ["x", "xv", "E_main", "E_1", "E_K", "E_V", "out0", "out1", "pos0", "d_h", "r_k",
            "r_v", "r_1", "rotate_keys", "rope_base"]
    d = {k: None for k in keys}
    d.update(pos0=0, d_h=0, r_k=0, r_v=0, r_1=0, rotate_keys=True, rope_base=10000.0)
    unknown = set(kw) - set(keys) - {"workspace", "stream"}
    if unknown:
        raise TypeError(f"unknown arguments {sorted(unknown)}")
    d.update({k: v for k, v in kw.items() if k in keys})
    return d


def lla_write_latents(mode, *, workspace=None, stream=None, **kw):
    """Append latents of n tokens per sequence at rows pos0..pos0+n-1.

    HLA:     x=h [B,n,T,D], E_main [T-1,r_k+r_v,D], E_1 [2r_1,D],
             out0 [B,Ncap,r_k+r_v], out1 [B,Ncap,2r_1], r_k=..., d_h=...
    PERHEAD: x=k, xv=v [B,n,T,H,d_h], E_K, E_V [T,H,r,d_h], out0=cK, out1=cV [B,H,Ncap,r]
    FOLDED:  x=k, xv=v, E_K [T,H,r_K,d_h], E_V [T,H,r_V,d_h], out0 [B,Ncap,r_K+r_V]
    """
    args = _write_kw(kw)
    dev = _cuda(args["x"], args["xv"], args["E_main"], args["E_1"], args["E_K"], args["E_V"],
                args["out0"], args["out1"])
    p = _write_params(mode, **args)
    L = lib()
    need = L.lla_write_workspace_bytes(ctypes.byref(p))
    ws, nb, _keep = _workspace(need, dev, workspace, stream)
    _call(L.lla_write_latents, p, ws, nb, _stream_handle(stream, dev), "lla_write_latents")


# ----------------------------------------------------------------- decode --
def _ring_fields(p, win_k, win_v):
    if win_k.shape != win_v.shape or win_k.stride() != win_v.stride() or win_k.dtype != win_v.dtype:
        raise ValueError("win_k and win_v must match in shape, strides and dtype")
    _dense_inner(win_k, 4, "win_k")
    p.win_k, p.win_v = _ptr(win_k), _ptr(win_v)
    p.win_dtype = _dtype_code(win_k)
    p.Wcap = win_k.shape[2]
    p.win_stride_b = win_k.stride(0)


def _events(p, timing_events):
    """Attach the optional (begin, end) torch.cuda.Event pair (timing hook)."""
    if timing_events is None:
        p.timing_events = None
        return
    ev0, ev1 = timing_events
    for ev in (ev0, ev1):
        if ev.cuda_event == 0:
            raise ValueError("record each timing event once before passing it (creates the handle)")
    arr = (ctypes.c_void_p * 2)(ev0.cuda_event, ev1.cuda_event)
    p._keep = arr
    p.timing_events = ctypes.cast(arr, ctypes.c_void_p)


def _win_side(p, win_stream, win_events):
    """Attach the optional window stream and its (fork, join) torch.cuda.Event pair."""
    if win_stream is None:
        p.win_stream = None
        p.win_events = None
        return
    if win_events is None:
        raise ValueError("win_stream needs win_events: a (fork, join) pair of torch.cuda.Event")
    ev0, ev1 = win_events
    for ev in (ev0, ev1):
        if ev.cuda_event == 0:
            raise ValueError("record each window event once before passing it (creates the handle)")
    arr = (ctypes.c_void_p * 2)(ev0.cuda_event, ev1.cuda_event)
    p._keep_win = arr
    p.win_stream = ctypes.c_void_p(win_stream.cuda_stream)
    p.win_events = ctypes.cast(arr, ctypes.c_void_p)


def _hla_params(lat, A, Bm, q, win_k, win_v, out, N, W, t0, r_k, rotate_query, rope_base, scale,
                timing_events=None, win_stream=None, win_events=None):
    p = _abi.HlaDecodeParams()
    if q.dim() == 5:                       # [B, nq, nt, H, d_h]: the last nq positions at once
        B, nq, nt, H, d_h = q.shape
        _dense_inner(q, 4, "q")
        _dense_inner(out, 4, "out")
    else:
        B, nt, H, d_h = q.shape
        nq = 1
        _dense_inner(q, 3, "q")
        _dense_inner(out, 3, "out")
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError("out must have q's shape")
    p.nq = nq
    for t, nm in ((A, "A"), (Bm, "Bm")):
        if not t.is_contiguous() or t.dtype != _torch().float32:
            raise ValueError(f"{nm} must be a contiguous float32 tensor")
    if tuple(A.shape[:3]) != (nt, H, d_h) or tuple(Bm.shape[:2]) != (nt, H) or Bm.shape[3] != d_h:
        raise ValueError("A is [nt,H,d_h,r_k], Bm is [nt,H,r_v,d_h]")
    r_k = A.shape[3] if r_k is None else r_k
    p.B, p.H, p.d_h, p.nt, p.t0 = B, H, d_h, nt, t0
    p.T = win_k.shape[1]
    p.N, p.W = N, W
    p.r_k, p.r_v = r_k, Bm.shape[2]
    if lat is not None:
        _dense_inner(lat, 1, "lat")
        p.lat = _ptr(lat)
        p.lat_dtype = _dtype_code(lat)
        p.lat_stride_b, p.lat_stride_n = lat.stride(0), lat.stride(1)
    p.A, p.Bm, p.q = _ptr(A), _ptr(Bm), _ptr(q)
    p.q_stride_b = q.stride(0)
    p.rotate_query = int(bool(rotate_query))
    p.rope_base = float(rope_base)
    _ring_fields(p, win_k, win_v)
    p.out = _ptr(out)
    p.out_stride_b = out.stride(0)
    p.scale = float(scale)
    _events(p, timing_events)
    _win_side(p, win_stream, win_events)
    return p


def hla_decode_workspace_bytes(**kw):
    p = _hla_params(**_hla_kw(kw))
    return lib().hla_decode_workspace_bytes(ctypes.byref(p))


def _hla_kw(kw):
    d = dict(lat=None, A=None, Bm=None, q=None, win_k=None, win_v=None, out=None, N=None, W=None,
             t0=0, r_k=None, rotate_query=True, rope_base=10000.0, scale=0.0, timing_events=None,
             win_stream=None, win_events=None)
    unknown = set(kw) - set(d) - {"workspace", "stream"}
    if unknown:
        raise TypeError(f"unknown arguments {sorted(unknown)}")
    d.update({k: v for k, v in kw.items() if k in d})
    return d


def hla_decode_attn(*, workspace=None, stream=None, **kw):
    """Absorbed latent read (HLA eqs. 3-4, or LLA-D with rotate_query=False).

    lat [B,Ncap,r_k+r_v] (key part stored as R~_j c^K_j; bf16, float32, or
    uint8 fp8 rows of r_k+r_v+16 bytes), A [nt,H,d_h,r_k], Bm [nt,H,r_v,d_h],
    q [B,nt,H,d_h] (or [B,nq,nt,H,d_h]: the last nq positions of the context
    at once), ring win_k/win_v [B,T,Wcap,H,d_h], out shaped like q, float32;
    N = context length, W = exact window, t0 = first loop served.  Optional
    win_stream (torch.cuda.Stream) with win_events (a (fork, join) pair of
    torch.cuda.Event, each recorded once beforehand): the window runs on
    win_stream beside the query map and the latent read.
    """
    args = _hla_kw(kw)
    dev = _cuda(args["lat"], args["A"], args["Bm"], args["q"], args["win_k"], args["win_v"], args["out"])
    p = _hla_params(**args)
    L = lib()
    need = L.hla_decode_workspace_bytes(ctypes.byref(p))
    ws, nb, _keep = _workspace(need, dev, workspace, stream)
    _call(L.hla_decode_attn, p, ws, nb, _stream_handle(stream, dev), "hla_decode_attn")


def _lla_params(cK, cV, UK, UV, q, win_k, win_v, out, N, W, t0, scale, timing_events=None):
    p = _abi.LlaDecodeParams()
    B, nt, H, d_h = q.shape
    _dense_inner(q, 3, "q")
    _dense_inner(out, 3, "out")
    for t, nm in ((UK, "UK"), (UV, "UV")):
        if not t.is_contiguous() or t.dtype != _torch().float32:
            raise ValueError(f"{nm} must be a contiguous float32 tensor")
    r = UK.shape[3]
    p.B, p.H, p.d_h, p.r, p.nt, p.t0 = B, H, d_h, r, nt, t0
    p.T = win_k.shape[1]
    p.N, p.W = N, W
    if cK is not None:
        _dense_inner(cK, 2, "cK")
        if cK.stride() != cV.stride() or cK.dtype != cV.dtype:
            raise ValueError("cK and cV must share strides and dtype")
        p.cK, p.cV = _ptr(cK), _ptr(cV)
        p.lat_dtype = _dtype_code(cK)
        p.lat_stride_b, p.lat_stride_h = cK.stride(0), cK.stride(1)
    p.UK, p.UV, p.q = _ptr(UK), _ptr(UV), _ptr(q)
    p.q_stride_b = q.stride(0)
    _ring_fields(p, win_k, win_v)
    p.out = _ptr(out)
    p.out_stride_b = out.stride(0)
    p.scale = float(scale)
    _events(p, timing_events)
    return p


def _lla_kw(kw):
    d = dict(cK=None, cV=None, UK=None, UV=None, q=None, win_k=None, win_v=None, out=None,
             N=None, W=0, t0=0, scale=0.0, timing_events=None)
    unknown = set(kw) - set(d) - {"workspace", "stream"}
    if unknown:
        raise TypeError(f"unknown arguments {sorted(unknown)}")
    d.update({k: v for k, v in kw.items() if k in d})
    return d


def lla_decode_workspace_bytes(**kw):
    p = _lla_params(**_lla_kw(kw))
    return lib().lla_decode_workspace_bytes(ctypes.byref(p))


def lla_decode_attn(*, workspace=None, stream=None, **kw):
    """LLA reconstruct-on-read decode attention.

    cK, cV [B,H,Ncap,r], UK, UV [nt,H,d_h,r], q [B,nt,H,d_h] post-rotary,
    ring win_k/win_v [B,T,Wcap,H,d_h], out [B,nt,H,d_h] float32.
    """
    args = _lla_kw(kw)
    dev = _cuda(args["cK"], args["cV"], args["UK"], args["UV"], args["q"], args["win_k"],
                args["win_v"], args["out"])
    p = _lla_params(**args)
    L = lib()
    need = L.lla_decode_workspace_bytes(ctypes.byref(p))
    ws, nb, _keep = _workspace(need, dev, workspace, stream)
    _call(L.lla_decode_attn, p, ws, nb, _stream_handle(stream, dev), "lla_decode_attn")


# -------------------------------------------------------- 8-bit K/V cache --
# These are called once for each layer, loop and token, so they keep the host's
# share small: each tensor's attributes are read once, and a call's parameters
# are packed in one go.
_CACHE_FMT = "6i2P2q2P2q"
_I32_FMT = "Pi4x"


def _packer(struct_type, fmt):
    s = struct.Struct("@" + fmt)
    if s.size != ctypes.sizeof(struct_type):
        raise AssertionError(f"{struct_type.__name__}: {s.size} packed bytes, {ctypes.sizeof(struct_type)} expected")
    return lambda *values: struct_type.from_buffer_copy(s.pack(*values))


_pack_write = _packer(_abi.Kv8WriteParams, _CACHE_FMT + "2P3i4x3qi4x" + 3 * _I32_FMT)
_pack_attn = _packer(_abi.Kv8AttnParams, _CACHE_FMT + _I32_FMT + "2i2Pi4x4q2P2i3q" + 2 * _I32_FMT + "f4xP2q")
_pack_evict = _packer(_abi.Kv8EvictParams, 2 * _CACHE_FMT + "P2qP2q2P3i4xP")


def _unlike(shape, sa, sb):
    """Whether strides that are not equal make two layouts of shape: an axis of one element may carry any."""
    return any(n > 1 and x != y for n, x, y in zip(shape, sa, sb))


def _kv8_cache(k8, v8, k_scale, v_scale):
    """[B,H,Ncap,d] codes and [B,H,Ncap/block] scales as the values of the ABI's struct."""
    torch = _torch()
    dtype, shape, st, sshape, ss = k8.dtype, k8.shape, k8.stride(), k_scale.shape, k_scale.stride()
    if dtype is torch.int8:
        code = LLA_KV8_I8
    elif dtype is torch.float8_e4m3fn:
        code = LLA_KV8_E4M3
    else:
        raise TypeError(f"unsupported code dtype {dtype}; use int8 or float8_e4m3fn")
    if v8.dtype is not dtype or k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32:
        raise TypeError("k8 and v8 share a dtype, scales are float32")
    if len(shape) != 4 or v8.shape != shape or (v8.stride() != st and _unlike(shape, v8.stride(), st)):
        raise ValueError("k8 and v8 are [B,H,Ncap,d] with the same strides")
    if len(sshape) != 3 or v_scale.shape != sshape or (v_scale.stride() != ss and _unlike(sshape, v_scale.stride(), ss)):
        raise ValueError("k_scale and v_scale are [B,H,Ncap/block] with the same strides")
    B, H, cap, d = shape
    sB, sH, nb = sshape
    if sB != B or sH != H or (cap % nb if nb else cap):
        raise ValueError("k_scale and v_scale are [B,H,Ncap/block] of k8's B, H and Ncap")
    sb, sh, sn, sd = st
    if sd != 1 or (sn != d and cap > 1):
        raise ValueError("k8 and v8: inner axes must be dense")
    if ss[2] != 1 and nb > 1:
        raise ValueError("k_scale and v_scale: inner axis must be dense")
    # an axis of one element may carry any stride
    if H == 1:
        sh = cap * d
    if B == 1:
        sb = H * sh
    qh = ss[1] if H > 1 else nb
    qb = ss[0] if B > 1 else H * qh
    return (B, H, d, cap // nb if nb else 16, cap, code, k8.data_ptr(), v8.data_ptr(), sb, sh, k_scale.data_ptr(),
            v_scale.data_ptr(), qb, qh)


def _i32(v, B, name):
    """An int for every sequence, or an int32 tensor [B]: (address, value)."""
    if v.__class__ is int:
        return 0, v
    torch = _torch()
    if isinstance(v, torch.Tensor):
        if v.dtype is not torch.int32 or v.shape != (B,) or (v.stride(0) != 1 and B > 1):
            raise ValueError(f"{name} is an int or a contiguous int32 tensor [B]")
        return v.data_ptr(), 0
    return 0, int(v)


def _kv8_device(*ts):
    """The one CUDA device of the tensors among the arguments."""
    Tensor, dev = _torch().Tensor, None
    for t in ts:
        if isinstance(t, Tensor):
            i = t.get_device()
            if i != dev:
                if dev is not None or i < 0:
                    _cuda(*[x for x in ts if isinstance(x, Tensor)])     # raises
                dev = i
    return dev


def _rows16(t, what):
    """Strides of the outer axes of t [B,rows,H,d], those of one element replaced by 0."""
    n0, n1, n2, d = t.shape
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 and d > 1:
        raise ValueError(f"{what}: the inner axis must be dense")
    return s0 if n0 > 1 else 0, s1 if n1 > 1 else 0, s2 if n2 > 1 else 0


def _on(dev, fn, where, params, *mid, stream):
    """Call fn on a stream of device number dev, with that device current."""
    cuda = _torch().cuda
    handle = (cuda.current_stream(dev) if stream is None else stream).cuda_stream
    if dev == cuda.current_device():
        st = fn(params, *mid, handle)
    else:
        with cuda.device(dev):
            st = fn(params, *mid, handle)
    if st != 0:
        raise LLAError(st, where)


def _kv8_size(size, params, dev):
    """Bytes of scratch on device number dev (its processor count decides on splits); negative: no device."""
    cuda = _torch().cuda
    if dev < 0 or dev == cuda.current_device():
        return size(params)
    with cuda.device(dev):
        return size(params)


def _kv8_workspace(size, params, dev, workspace, stream):
    """(address, bytes, tensor) of a call's scratch."""
    need = _kv8_size(size, params, dev)
    if need and workspace is None:
        workspace = _scratch(need, _torch().device("cuda", dev), stream)
    elif need and workspace.get_device() != dev:
        raise ValueError("workspace is on another device")
    elif need and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if not need:
        return None, 0, None
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace too small: {have} < {need} bytes")
    return workspace.data_ptr(), have, workspace


def lla_kv8_write(*, k, v, k8, v8, k_scale, v_scale, n=None, max_n=None, src0=0, row0=0, ring=False, stream=None):
    """Quantise tokens of k, v [B,rows,H,d] (float32 or bfloat16) into the cache.

    Cache: codes k8, v8 [B,H,Ncap,d] (int8 or float8_e4m3fn) and scales
    k_scale, v_scale [B,H,Ncap/block] float32, block in 16..256.  Sequence b's
    tokens src0[b] .. src0[b]+n[b]-1 (ring=True: positions, in rows mod `rows`)
    go to cache rows row0[b].., row0 a multiple of block.  n, src0, row0: an int
    for all sequences or an int32 CUDA tensor [B]; n defaults to `rows`, and a
    tensor n needs max_n, its bound (default: the least of rows and Ncap).
    """
    dev = _kv8_device(k, v, k8, v8, k_scale, v_scale, n, src0, row0)
    c = _kv8_cache(k8, v8, k_scale, v_scale)
    B, shape = c[0], k.shape
    if (len(shape) != 4 or v.shape != shape or k.dtype is not v.dtype
            or (k.stride() != v.stride() and _unlike(shape, k.stride(), v.stride()))):
        raise ValueError("k and v are [B,rows,H,d] and match in shape, strides and dtype")
    rows = shape[1]
    if shape[0] != B or shape[2] != c[1] or shape[3] != c[2]:
        raise ValueError("k and v are [B,rows,H,d] of the cache's B, H and d")
    if n is None:
        n = rows
    if max_n is None:
        max_n = n if isinstance(n, int) else min(rows, c[4])
    p = _pack_write(*c, k.data_ptr(), v.data_ptr(), _dtype_code(k), rows, 1 if ring else 0, *_rows16(k, "k and v"),
                    max_n, *_i32(n, B, "n"), *_i32(src0, B, "src0"), *_i32(row0, B, "row0"))
    _on(dev, lib().lla_kv8_write, "lla_kv8_write", p, stream=stream)


def _kv8_attn_params(q, k8, v8, k_scale, v_scale, lens, out, win_k=None, win_v=None, ctx=None, tail=0, scale=0.0,
                     weights=None):
    c = _kv8_cache(k8, v8, k_scale, v_scale)
    B, H, d = c[:3]
    shape = q.shape
    if len(shape) != 4 or shape[0] != B or shape[3] != d or shape[2] % H or shape[2] == 0:
        raise ValueError("q is [B,nq,H*G,d] of the cache's B, H and d")
    if out.shape != shape or out.dtype is not q.dtype:
        raise ValueError("out must have q's shape and dtype")
    _, nq, heads, _ = shape
    row = heads * d
    qb, qn, qh, qd = q.stride()
    ob, on, oh, od = out.stride()
    if qd != 1 or od != 1 or (heads > 1 and (qh != d or oh != d)):
        raise ValueError("q and out: inner axes must be dense")
    win = (0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    if win_k is not None:
        ws = win_k.shape
        if (win_v is None or len(ws) != 4 or win_v.shape != ws or win_k.dtype is not win_v.dtype
                or (win_k.stride() != win_v.stride() and _unlike(ws, win_k.stride(), win_v.stride()))):
            raise ValueError("win_k and win_v are [B,Wcap,H,d] and match in shape, strides and dtype")
        if ws[0] != B or ws[2] != H or ws[3] != d:
            raise ValueError("win_k and win_v are [B,Wcap,H,d] of the cache's B, H and d")
        if ctx is None:
            raise ValueError("win_k needs ctx, the context length")
        win = (win_k.data_ptr(), win_v.data_ptr(), _dtype_code(win_k), ws[1], *_rows16(win_k, "win_k and win_v"),
               *_i32(ctx, B, "ctx"), *_i32(tail, B, "tail"))
    elif win_v is not None:
        raise ValueError("win_v without win_k")
    w = (0, 0, 0) if weights is None else _kv8_weights(weights, c)
    return _pack_attn(*c, *_i32(lens, B, "lens"), nq, heads // H, q.data_ptr(), out.data_ptr(), _dtype_code(q),
                      qb if B > 1 else 0, qn if nq > 1 else 0, ob if B > 1 else nq * row, on if nq > 1 else row,
                      *win, scale, *w)


def _kv8_weights(w, c):
    B, H, cap = c[0], c[1], c[4]
    if w.dtype is not _torch().float32 or w.shape != (B, H, cap):
        raise ValueError("weights are float32 [B,H,Ncap]")
    sb, sh, sn = w.stride()
    if sn != 1 and cap > 1:
        raise ValueError("weights: the inner axis must be dense")
    if H == 1:
        sh = cap
    return w.data_ptr(), sb if B > 1 else H * sh, sh


def lla_kv8_attn_workspace_bytes(**kw):
    kw.pop("workspace", None)
    kw.pop("stream", None)
    return _kv8_size(lib().lla_kv8_attn_workspace_bytes, _kv8_attn_params(**kw), kw["k8"].get_device())


def lla_kv8_attn(*, q, k8, v8, k_scale, v_scale, lens, out, win_k=None, win_v=None, ctx=None, tail=0, scale=0.0,
                 weights=None, workspace=None, stream=None):
    """Attention over an 8-bit cache and the exact tokens after it, one softmax.

    q [B,nq,H*G,d] (float32 or bfloat16; head h reads cache head h // G), out
    likewise; cache as lla_kv8_write fills it, of which each query sees the
    first lens[b] tokens; ring win_k, win_v [B,Wcap,H,d] holds the last tail[b]
    (at most ctx[b]) positions of a context of ctx[b] tokens, position j in row
    j mod Wcap, and query p (context position ctx - nq + p) sees those up to
    its own.  lens, ctx, tail: an int for all sequences or an int32 CUDA tensor
    [B].  weights [B,H,Ncap] float32, optional: the softmax weights of the
    cached tokens are added, summed over the queries of their head.  scale 0:
    1/sqrt(d).
    """
    dev = _kv8_device(q, k8, v8, k_scale, v_scale, out, win_k, win_v, weights, lens, ctx, tail)
    p = _kv8_attn_params(q, k8, v8, k_scale, v_scale, lens, out, win_k, win_v, ctx, tail, scale, weights)
    L = lib()
    ws, nb, _keep = _kv8_workspace(L.lla_kv8_attn_workspace_bytes, p, dev, workspace, stream)
    _on(dev, L.lla_kv8_attn, "lla_kv8_attn", p, ws, nb, stream=stream)


def _kv8_evict_params(k8, v8, k_scale, v_scale, weights, lens, keep, first=0, last=1, to=None, kept=None):
    torch = _torch()
    c = _kv8_cache(k8, v8, k_scale, v_scale)
    w = _kv8_weights(weights, c)
    if to is None:
        t, tw, to_lens = c, w, lens
    else:
        t = _kv8_cache(to["k8"], to["v8"], to["k_scale"], to["v_scale"])
        tw, to_lens = _kv8_weights(to["weights"], t), to["lens"]
    for x in (lens, to_lens):
        if x.dtype is not torch.int32 or x.shape != (c[0],) or not x.is_contiguous():
            raise ValueError("lens (and to['lens']) are contiguous int32 tensors [B]")
    if kept is not None and (kept.dtype is not torch.int32 or kept.shape != (c[0], c[1], keep)
                             or not kept.is_contiguous()):
        raise ValueError("kept is a contiguous int32 tensor [B,H,keep]")
    return _pack_evict(*c, *t, *w, *tw, lens.data_ptr(), to_lens.data_ptr(), keep, first, last,
                       0 if kept is None else kept.data_ptr())


def lla_kv8_evict_workspace_bytes(**kw):
    kw.pop("workspace", None)
    kw.pop("stream", None)
    return _kv8_size(lib().lla_kv8_evict_workspace_bytes, _kv8_evict_params(**kw), kw["k8"].get_device())


def lla_kv8_evict(*, k8, v8, k_scale, v_scale, weights, lens, keep, first=0, last=1, to=None, kept=None,
                  workspace=None, stream=None):
    """Keep the `keep` blocks of each head that gathered the most weight.

    Cache (at most 8192 blocks a head) and weights [B,H,Ncap] as lla_kv8_attn
    reads and adds them; lens int32 [B].  Of a sequence of more than `keep` blocks the first `first`, the last
    `last` (>= 1) and, of the others, those whose tokens' weights sum highest
    stay, in order, moved to the front.  In place, or into `to`: a dict of k8,
    v8, k_scale, v_scale, weights and lens of another cache (which may have
    another Ncap).  kept [B,H,keep] int32, optional: source block of each block
    that stays, -1 where there is none.
    """
    dev = _kv8_device(k8, v8, k_scale, v_scale, weights, lens, kept, *(to.values() if to else ()))
    p = _kv8_evict_params(k8, v8, k_scale, v_scale, weights, lens, keep, first, last, to, kept)
    L = lib()
    ws, nb, _keep = _kv8_workspace(L.lla_kv8_evict_workspace_bytes, p, dev, workspace, stream)
    _on(dev, L.lla_kv8_evict, "lla_kv8_evict", p, ws, nb, stream=stream)
