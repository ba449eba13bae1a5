"""Thin Python binding over the state-space operators of libwkv_b200.so
(include/wkv_ssm.h): the short causal convolution, the per-head norm with
position rotation and the selective scan.

Like ``wkv``, argument marshalling only: every function checks tensor dtypes,
shapes, devices and contiguity, allocates outputs and workspaces with torch
and calls the C entry point of the same name on the tensors' device and its
current stream.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import wkv as _wkv
from .wkv import WkvError, _check, _dtype_code, _want, device_error  # noqa: F401  (WkvError, device_error: re-exported)

SCAN_CKPT_LEN = 16  # WKV_SCAN_CKPT_LEN

_i64, _int, _vp, _sz, _f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
# Every symbol include/wkv_ssm.h declares, with its ctypes signature.
SIGNATURES = {
    "wkv_conv_forward": (_int, [_i64, _i64, _i64, _int, _i64, _int] + [_vp] * 6),
    "wkv_conv_backward_workspace_bytes": (_sz, [_i64, _i64, _i64, _int, _i64]),
    "wkv_conv_backward": (_int, [_i64, _i64, _i64, _int, _i64, _int] + [_vp] * 10 + [_sz, _vp]),
    "wkv_conv_chunk_step": (_int, [_i64, _i64, _int, _i64, _int] + [_vp] * 4 + [_i64, _vp, _vp, _vp]),
    "wkv_conv_decode_step": (_int, [_i64, _i64, _int, _i64, _int] + [_vp] * 6),
    "wkv_norm_rotate": (_int, [_i64] * 6 + [_int] + [_vp] * 4 + [_f32, _vp, _vp, _i64, _int] + [_vp] * 3),
    "wkv_norm_rotate_backward_workspace_bytes": (_sz, [_i64] * 5),
    "wkv_norm_rotate_backward": (_int, [_i64] * 6 + [_int] + [_vp] * 6 + [_f32, _vp, _vp, _i64, _int] + [_vp] * 5 +
                                 [_sz, _vp]),
    "wkv_scan_forward": (_int, [_i64] * 5 + [_int] + [_vp] * 8 + [_int] + [_vp] * 5 + [_sz, _vp]),
    "wkv_scan_forward_workspace_bytes": (_sz, [_i64] * 5),
    "wkv_scan_ckpt_floats": (_sz, [_i64] * 4),
    "wkv_scan_backward_workspace_bytes": (_sz, [_i64] * 5 + [_int]),
    "wkv_scan_backward": (_int, [_i64] * 5 + [_int] + [_vp] * 8 + [_int] + [_vp] * 14 + [_sz, _vp]),
    "wkv_scan_chunk_step": (_int, [_i64] * 4 + [_int] + [_vp] * 8 + [_int, _vp, _i64, _vp, _vp, _vp]),
    "wkv_scan_decode_step": (_int, [_i64] * 4 + [_int] + [_vp] * 8 + [_int, _vp, _vp, _vp]),
}

_lib = _wkv.lib()
for _name, (_res, _args) in SIGNATURES.items():
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args


# The current stream's handle without the torch.cuda.Stream object around it
# (0.3 of the 11 microseconds that a small call takes on the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_fn = {name: getattr(_lib, name) for name in SIGNATURES}


def _call(name: str, dev: torch.device, *args):
    """Calls the C entry point on the device's current stream, with `dev` current."""
    if dev.index == torch.cuda.current_device():
        status = _fn[name](*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            status = _fn[name](*args, _raw_stream(dev.index))
    if status:
        _check(status, name)


def _has(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, dev: torch.device) -> int:
    """The tensor's address, once it is known to be what the call reads or writes."""
    if not (t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous()):
        _want(t, name, dtype=dtype, shape=shape, device=dev)
    return t.data_ptr()


def _may(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple, dev: torch.device):
    return None if t is None else _has(t, name, dtype, shape, dev)


_CODES = {torch.float32: _wkv.WKV_F32, torch.bfloat16: _wkv.WKV_BF16}


def _first(t: torch.Tensor, name: str, dims: int):
    """(device, dtype code) of the tensor that the sizes are taken from."""
    if not (t.is_cuda and t.is_contiguous()):
        _want(t, name)
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    code = _CODES.get(t.dtype)
    return t.device, _dtype_code(t) if code is None else code


def _like(t: Optional[torch.Tensor], given: Optional[torch.Tensor], name: str, dtype, shape, dev):
    """(tensor, address) of an output: the one given, checked, or a new one like `t`."""
    if given is None:
        given = torch.empty_like(t)
        return given, given.data_ptr()
    return given, _has(given, name, dtype, shape, dev)


def _float32(want: bool, given: Optional[torch.Tensor], like: torch.Tensor, name: str, shape, dev):
    """(tensor, address) of a float32 output: the one given, checked, or where
    wanted a new one on the device of the float32 tensor `like`; else (None, None)."""
    if given is not None:
        return given, _has(given, name, torch.float32, shape, dev)
    if not want:
        return None, None
    given = like.new_empty(shape)
    return given, given.data_ptr()


def _space(workspace: Optional[torch.Tensor], nbytes: int, dev: torch.device):
    """(address, bytes, the tensor) of a workspace of at least `nbytes`."""
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        return workspace.data_ptr(), nbytes, workspace
    _want(workspace, "workspace", device=dev)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# ----------------------------------------------------------------------------
# short causal convolution
# ----------------------------------------------------------------------------

def _taps(weight: torch.Tensor, C: int) -> int:
    if weight.dim() != 2:
        raise ValueError("weight must be [W, C]")
    return weight.shape[0]


def wkv_conv_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                     x_prev: Optional[torch.Tensor] = None, *, silu: bool = True,
                     y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Depthwise causal convolution over the last W tokens. x: [B, T, C];
    weight: [W, C] float32 (W 2..4, the last row meets the current token);
    bias: [C] float32; x_prev: [B, W-1, C], the tokens before x (None: zeros).
    Returns y like x, put through silu unless ``silu`` is false."""
    dev, code = _first(x, "x", 3)
    B, T, C = x.shape
    W, f32 = _taps(weight, C), torch.float32
    y, yp = _like(x, y, "y", x.dtype, x.shape, dev)
    _call("wkv_conv_forward", dev, B, T, C, code, W, int(silu), x.data_ptr(),
          _has(weight, "weight", f32, (W, C), dev), _may(bias, "bias", f32, (C,), dev),
          _may(x_prev, "x_prev", x.dtype, (B, W - 1, C), dev), yp)
    return y


def wkv_conv_backward(x, weight, gy, bias=None, x_prev=None, *, silu: bool = True, want_gx_prev: bool = False,
                      gx=None, gweight=None, gbias=None, gx_prev=None, workspace: Optional[torch.Tensor] = None):
    """Gradients of sum(gy * wkv_conv_forward(x, weight, bias, x_prev)).
    Returns (gx, gweight, gbias, gx_prev); gbias is None without a bias,
    gx_prev unless wanted (or a buffer is passed)."""
    dev, code = _first(x, "x", 3)
    B, T, C = x.shape
    W, f32, e = _taps(weight, C), torch.float32, x.dtype
    wp = _has(weight, "weight", f32, (W, C), dev)
    bp = _may(bias, "bias", f32, (C,), dev)
    gx, gxp = _like(x, gx, "gx", e, x.shape, dev)
    gweight, gwp = _like(weight, gweight, "gweight", f32, (W, C), dev)
    gbp = None
    if bias is not None or gbias is not None:
        gbias, gbp = _like(bias, gbias, "gbias", f32, (C,), dev)
    if gx_prev is None and want_gx_prev:
        gx_prev = torch.empty((B, W - 1, C), dtype=e, device=dev)
    ptr, nbytes, workspace = _space(workspace, _fn["wkv_conv_backward_workspace_bytes"](B, T, C, code, W), dev)
    _call("wkv_conv_backward", dev, B, T, C, code, W, int(silu), x.data_ptr(), wp, bp,
          _may(x_prev, "x_prev", e, (B, W - 1, C), dev), _has(gy, "gy", e, x.shape, dev), gxp, gwp, gbp,
          _may(gx_prev, "gx_prev", e, (B, W - 1, C), dev), ptr, nbytes)
    return gx, gweight, gbias, gx_prev


def wkv_conv_chunk_step(x, weight, cu_tokens: torch.Tensor, state: torch.Tensor, bias=None, *, silu: bool = True,
                        y=None) -> torch.Tensor:
    """The convolution over slots. x: [n, C], the tokens of all slots packed;
    cu_tokens: int32 [S+1] on the device; state: [S, W-1, C] like x, the last
    tokens of each slot, read and written in place. Returns y like x."""
    dev, code = _first(x, "x", 2)
    n, C = x.shape
    W, S, f32 = _taps(weight, C), state.shape[0], torch.float32
    y, yp = _like(x, y, "y", x.dtype, x.shape, dev)
    _call("wkv_conv_chunk_step", dev, S, C, code, W, int(silu), x.data_ptr(),
          _has(weight, "weight", f32, (W, C), dev), _may(bias, "bias", f32, (C,), dev), yp, n,
          _has(cu_tokens, "cu_tokens", torch.int32, (S + 1,), dev), _has(state, "state", x.dtype, (S, W - 1, C), dev))
    return y


def wkv_conv_decode_step(x, weight, state: torch.Tensor, bias=None, *, silu: bool = True, y=None) -> torch.Tensor:
    """One token for every slot: x, y [S, C]; state as for wkv_conv_chunk_step."""
    dev, code = _first(x, "x", 2)
    S, C = x.shape
    W, f32 = _taps(weight, C), torch.float32
    y, yp = _like(x, y, "y", x.dtype, x.shape, dev)
    _call("wkv_conv_decode_step", dev, S, C, code, W, int(silu), x.data_ptr(),
          _has(weight, "weight", f32, (W, C), dev), _may(bias, "bias", f32, (C,), dev), yp,
          _has(state, "state", x.dtype, (S, W - 1, C), dev))
    return y


# ----------------------------------------------------------------------------
# per-head norm with position rotation
# ----------------------------------------------------------------------------

def _norm_operands(q, k, q_weight, k_weight, inv_freq, positions, K, pos_offset):
    """(device, dtype, dtype code, sizes B T Hq Hk K R, the addresses of the
    operands) of a call; q or k may be None."""
    if K < 1:
        raise ValueError("head_size must be at least 1")
    if not -(1 << 63) <= pos_offset < 1 << 63:
        raise ValueError("pos_offset must fit 64 bits")
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("q and k are both None")
    dev, code = _first(lead, "q" if q is not None else "k", 3)
    B, T, width = lead.shape
    e, f32 = lead.dtype, torch.float32
    qp = kp = None
    Hq = Hk = 0
    if q is not None:
        Hq, odd = divmod(width, K)
        qp = q.data_ptr()
    else:
        Hk, odd = divmod(width, K)
        kp = k.data_ptr()
    if q is not None and k is not None:
        if k.dim() != 3:
            raise ValueError(f"k must have 3 dimensions, got shape {tuple(k.shape)}")
        Hk, more = divmod(k.shape[2], K)
        odd = odd or more
        kp = _has(k, "k", e, (B, T, k.shape[2]), dev)
    if odd:
        raise ValueError(f"q and k must be [B, T, H * {K}]")
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    return dev, e, code, (B, T, Hq, Hk, K, R), (
        qp, kp, _may(q_weight, "q_weight", f32, (K,), dev), _may(k_weight, "k_weight", f32, (K,), dev),
        _may(inv_freq, "inv_freq", f32, (R // 2,), dev), _may(positions, "positions", torch.int32, (B, T), dev))


def wkv_norm_rotate(q, k, q_weight=None, k_weight=None, inv_freq=None, positions=None, *, head_size: int,
                    eps: float = 1e-6, pos_offset: int = 0, interleaved: bool = False, q_out=None, k_out=None):
    """Root-mean-square norm of every head of q and k and rotation of its first
    2 * len(inv_freq) entries by position, in one pass. q: [B, T, Hq*K], k:
    [B, T, Hk*K] (either may be None); q_weight, k_weight: [K] float32;
    inv_freq: [R/2] float32 (None: no rotation); positions: int32 [B, T] (None:
    pos_offset + t, within 2^53). q_out=q and k_out=k work in place. Returns (q_out, k_out)."""
    dev, e, code, sizes, (qp, kp, wq, wk, fr, po) = _norm_operands(
        q, k, q_weight, k_weight, inv_freq, positions, head_size, pos_offset)
    qo = ko = None
    if q is not None:
        q_out, qo = _like(q, q_out, "q_out", e, q.shape, dev)
    if k is not None:
        k_out, ko = _like(k, k_out, "k_out", e, k.shape, dev)
    _call("wkv_norm_rotate", dev, *sizes, code, qp, kp, wq, wk, eps, fr, po, pos_offset, int(interleaved), qo, ko)
    return q_out if q is not None else None, k_out if k is not None else None


def wkv_norm_rotate_backward(q, k, gq_out, gk_out, q_weight=None, k_weight=None, inv_freq=None, positions=None, *,
                             head_size: int, eps: float = 1e-6, pos_offset: int = 0, interleaved: bool = False,
                             gq=None, gk=None, workspace: Optional[torch.Tensor] = None):
    """Gradients of sum(gq_out * q_out) + sum(gk_out * k_out) for wkv_norm_rotate
    with the same arguments. Returns (gq, gk, gq_weight, gk_weight); a weight's
    gradient is None where there is no such weight."""
    dev, e, code, sizes, (qp, kp, wq, wk, fr, po) = _norm_operands(
        q, k, q_weight, k_weight, inv_freq, positions, head_size, pos_offset)
    gop = kop = gqp = gkp = gwqp = gwkp = gwq = gwk = None
    if q is not None:
        gop = _has(gq_out, "gq_out", e, q.shape, dev)
        gq, gqp = _like(q, gq, "gq", e, q.shape, dev)
    if k is not None:
        kop = _has(gk_out, "gk_out", e, k.shape, dev)
        gk, gkp = _like(k, gk, "gk", e, k.shape, dev)
    if q_weight is not None:
        gwq = torch.empty_like(q_weight)
        gwqp = gwq.data_ptr()
    if k_weight is not None:
        gwk = torch.empty_like(k_weight)
        gwkp = gwk.data_ptr()
    ptr, nbytes, workspace = _space(workspace, _fn["wkv_norm_rotate_backward_workspace_bytes"](*sizes[:5]), dev)
    _call("wkv_norm_rotate_backward", dev, *sizes, code, qp, kp, gop, kop, wq, wk, eps, fr, po, pos_offset,
          int(interleaved), gqp, gkp, gwqp, gwkp, ptr, nbytes)
    return gq if q is not None else None, gk if k is not None else None, gwq, gwk


# ----------------------------------------------------------------------------
# selective scan
# ----------------------------------------------------------------------------

def scan_ckpt_shape(B: int, T: int, C: int, N: int):
    return (B, (T + SCAN_CKPT_LEN - 1) // SCAN_CKPT_LEN, C, N)


def _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, dims):
    """(device, dtype code, sizes, addresses of the operands) of a scan over x of `dims` dimensions."""
    dev, code = _first(x, "x", dims)
    shape, f32, e = x.shape, torch.float32, x.dtype
    *lead, C = shape
    rates, bc = A.shape, Bm.shape
    if len(rates) != 2 or rates[0] != C:
        raise ValueError(f"A must be [C, N] with C = {C}, got {tuple(rates)}")
    N = rates[1]
    if len(bc) != dims or N == 0 or bc[-1] % N:
        raise ValueError(f"Bm must be [..., G * N] with N = {N}, got {tuple(bc)}")
    GN = bc[-1]
    bc = (*lead, GN)
    return dev, code, lead, C, N, GN // N, (
        x.data_ptr(), _has(dt, "dt", e, shape, dev), _has(A, "A", f32, (C, N), dev), _has(Bm, "Bm", e, bc, dev),
        _has(Cm, "Cm", e, bc, dev), _may(D, "D", f32, (C,), dev), _may(z, "z", e, shape, dev),
        _may(dt_bias, "dt_bias", f32, (C,), dev))


def wkv_scan_forward(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, init_state=None, *, dt_softplus: bool = True,
                     want_final_state: bool = True, want_ckpt: bool = False, y=None, final_state=None, ckpt=None,
                     workspace: Optional[torch.Tensor] = None):
    """Selective scan. x, dt, z: [B, T, C]; A: [C, N] float32; Bm, Cm: [B, T,
    G*N]; D, dt_bias: [C] float32; init_state: [B, C, N] float32.
    Returns (y, final_state or None), or (y, final_state or None, ckpt) when
    ``want_ckpt`` (or a ckpt buffer is passed)."""
    dev, code, (B, T), C, N, G, ptrs = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, 3)
    y, yp = _like(x, y, "y", x.dtype, x.shape, dev)
    final_state, fp = _float32(want_final_state, final_state, A, "final_state", (B, C, N), dev)
    ckpt, cp = _float32(want_ckpt, ckpt, A, "ckpt", scan_ckpt_shape(B, T, C, N), dev)
    ptr, nbytes, workspace = _space(workspace, _fn["wkv_scan_forward_workspace_bytes"](B, T, C, N, G), dev)
    _call("wkv_scan_forward", dev, B, T, C, N, G, code, *ptrs, int(dt_softplus),
          _may(init_state, "init_state", torch.float32, (B, C, N), dev), yp, fp, cp, ptr, nbytes)
    return (y, final_state) if ckpt is None else (y, final_state, ckpt)


def wkv_scan_backward(x, dt, A, Bm, Cm, gy, D=None, z=None, dt_bias=None, init_state=None, g_final=None, ckpt=None, *,
                      dt_softplus: bool = True, want_g_init: bool = False, gx=None, gdt=None, gz=None,
                      workspace: Optional[torch.Tensor] = None):
    """Gradients of sum(gy * y) + sum(g_final * final_state) for
    wkv_scan_forward with the same arguments. ckpt: the checkpoints it wrote
    (None: regenerated). Returns (gx, gdt, gA, gB, gC, gD, gz, gdt_bias,
    g_init); the gradient of an operand that is None is None, and so is g_init
    unless wanted."""
    dev, code, (B, T), C, N, G, ptrs = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, 3)
    f32, e = torch.float32, x.dtype
    gx, gxp = _like(x, gx, "gx", e, x.shape, dev)
    gdt, gdtp = _like(x, gdt, "gdt", e, x.shape, dev)
    gzp = None
    if z is None:
        gz = None
    else:
        gz, gzp = _like(z, gz, "gz", e, x.shape, dev)
    gA, gB, gC = torch.empty_like(A), torch.empty_like(Bm), torch.empty_like(Cm)
    gD = None if D is None else torch.empty_like(D)
    gbias = None if dt_bias is None else torch.empty_like(dt_bias)
    g_init = A.new_empty((B, C, N)) if want_g_init else None
    ptr, nbytes, workspace = _space(
        workspace, _fn["wkv_scan_backward_workspace_bytes"](B, T, C, N, G, int(ckpt is not None)), dev)
    _call("wkv_scan_backward", dev, B, T, C, N, G, code, *ptrs, int(dt_softplus),
          _may(init_state, "init_state", f32, (B, C, N), dev), _has(gy, "gy", e, x.shape, dev),
          _may(g_final, "g_final", f32, (B, C, N), dev), _may(ckpt, "ckpt", f32, scan_ckpt_shape(B, T, C, N), dev),
          gxp, gdtp, gA.data_ptr(), gB.data_ptr(), gC.data_ptr(), None if gD is None else gD.data_ptr(), gzp,
          None if gbias is None else gbias.data_ptr(), None if g_init is None else g_init.data_ptr(), ptr, nbytes)
    return gx, gdt, gA, gB, gC, gD, gz, gbias, g_init


def wkv_scan_chunk_step(x, dt, A, Bm, Cm, cu_tokens: torch.Tensor, state: torch.Tensor, D=None, z=None, dt_bias=None,
                        *, dt_softplus: bool = True, y=None) -> torch.Tensor:
    """The scan over slots. x, dt, z: [n, C], Bm, Cm: [n, G*N], the tokens of all
    slots packed; cu_tokens: int32 [S+1] on the device; state: [S, C, N]
    float32, read and written in place. Returns y like x."""
    dev, code, (n,), C, N, G, ptrs = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, 2)
    S = state.shape[0]
    y, yp = _like(x, y, "y", x.dtype, x.shape, dev)
    _call("wkv_scan_chunk_step", dev, S, C, N, G, code, *ptrs, int(dt_softplus), yp, n,
          _has(cu_tokens, "cu_tokens", torch.int32, (S + 1,), dev), _has(state, "state", torch.float32, (S, C, N), dev))
    return y


def wkv_scan_decode_step(x, dt, A, Bm, Cm, state: torch.Tensor, D=None, z=None, dt_bias=None, *,
                         dt_softplus: bool = True, y=None) -> torch.Tensor:
    """One token for every slot: x, dt, z, y [S, C], Bm, Cm [S, G*N]; state as for
    wkv_scan_chunk_step."""
    dev, code, (S,), C, N, G, ptrs = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, 2)
    y, yp = _like(x, y, "y", x.dtype, x.shape, dev)
    _call("wkv_scan_decode_step", dev, S, C, N, G, code, *ptrs, int(dt_softplus), yp,
          _has(state, "state", torch.float32, (S, C, N), dev))
    return y
