"""Binding of the operators around the layer: the short causal convolution before
it, and the selective scan with a diagonal A. Argument marshalling only.

Inputs may be slices of wider rows (a projection's output): channels contiguous,
any non-negative strides of tokens and batch rows. Outputs are contiguous. Every
tensor is on one device, whichever is current; a call runs on that device's
current stream, or on `stream`, which the caller orders behind the work that made
the inputs (new outputs come from the current stream's memory).
"""
from __future__ import annotations

import struct

import torch

from ._lib import SSD_BF16, SSD_F32, check, lib

_DT = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}
_F32 = torch.float32

# ssd_conv_shape_t and ssd_selective_shape_t as bytes: building the ctypes structures costs more than
# the rest of a decoding step's call
_conv_shape = struct.Struct("=9q2i").pack
_selective_shape = struct.Struct("=15q4i").pack


def _refuse(t, name, shape, dtype, device, inner):
    """Raises what is wrong with an input."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if inner == len(shape):
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name}: the last {inner} dimension(s) must be contiguous")


def _inner_contiguous(t, inner):
    step = 1
    for size, stride in zip(reversed(t.shape[-inner:]), reversed(t.stride()[-inner:])):
        if size > 1 and stride != step:
            return False
        step *= size
    return True


def _in(t, name, shape, dtype, device, inner=1):
    """An input: its shape, type and device, and its last `inner` dimensions contiguous."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and (t.is_contiguous() or _inner_contiguous(t, inner))):
        return t
    _refuse(t, name, shape, dtype, device, inner)


def _whole(t, name, shape, dtype, device):
    """A tensor that has to be contiguous throughout."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return t
    _refuse(t, name, shape, dtype, device, len(shape))


def _first(t, name, dim):
    """The call's first input, whose type and device the others share."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DT:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")


def _like(u):
    """A new contiguous tensor of u's shape and type."""
    return torch.empty_like(u) if u.is_contiguous() else u.new_empty(u.shape)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _current_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# the raw handle of the device's current stream, without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_entries = {}


def _call(name, t, stream, *args):
    """The entry point on t's device and its current stream, or on `stream`."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(lib(), name)
    index = t.get_device()
    if stream is None:
        handle = _raw_stream(index) if _raw_stream is not None else _current_stream(t.device)
    elif stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    else:
        handle = stream.cuda_stream
    if index == _current_device():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st:
        check(st, name)


def _offsets(cu_seqlens, T, device, stream=None):
    """Device offsets of a pack: a device int32 tensor as is, a host list checked and copied. The
    copy is made, and its memory used again, in the order of the stream that reads it."""
    if isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.is_cuda:
        if (cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous()
                or cu_seqlens.numel() < 1):
            raise ValueError("device cu_seqlens must be a contiguous 1-D int32 tensor of n_docs + 1 offsets")
        if cu_seqlens.device != device:
            raise ValueError(f"cu_seqlens must be on {device}, got {cu_seqlens.device}")
        return cu_seqlens
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    from . import check_cu_seqlens
    cu = torch.tensor(check_cu_seqlens(cu_seqlens, T), dtype=torch.int32)
    if stream is None:
        return cu.to(device)
    with torch.cuda.stream(stream):
        return cu.to(device)


# ---- the short causal convolution ------------------------------------------

def _check_conv(u, weight, bias):
    """Raises what is wrong with the convolution's inputs."""
    _first(u, "u", 3)
    _in(u, "u", u.shape, u.dtype, u.device)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [channels, width]")
    _whole(weight, "weight", (u.shape[2], weight.shape[1]), _F32, u.device)
    if bias is not None:
        _whole(bias, "bias", (u.shape[2],), _F32, u.device)


def _conv_args(u, weight, bias, silu, split, out):
    """The width, the checked shape as bytes, the outputs and three pointers to them."""
    try:       # the checks of _check_conv at once; it says which one failed
        b, T, C = u.shape
        s, index = u.stride(), u.get_device()
        Cw, W = weight.shape
        good = (index >= 0 and (s[2] == 1 or C == 1) and u.dtype in _DT and Cw == C and weight.dtype is _F32
                and weight.get_device() == index and weight.is_contiguous()
                and (bias is None or (bias.dtype is _F32 and bias.shape == (C,) and bias.get_device() == index
                                      and bias.is_contiguous())))
    except (AttributeError, TypeError, ValueError, IndexError):
        good = False
    if not good:
        _check_conv(u, weight, bias)
        b, T, C = u.shape
        s, W = u.stride(), weight.shape[1]
    sizes = (C,) if split is None else tuple(split)
    if not 1 <= len(sizes) <= 3 or min(sizes) < 0 or sum(sizes) != C:
        raise ValueError(f"split must be up to three sizes that add up to {C}, got {split}")
    if out is None:
        ys = [_like(u)] if len(sizes) == 1 else [u.new_empty((b, T, c)) for c in sizes]
    else:
        ys = [out] if split is None else list(out)
        if len(ys) != len(sizes):
            raise ValueError(f"out must be {len(sizes)} tensors")
        for i, (y, c) in enumerate(zip(ys, sizes)):
            _whole(y, f"out[{i}]", (b, T, c), u.dtype, u.device)
    pad = (0,) * (3 - len(sizes))
    shape = _conv_shape(b, T, C, W, *sizes, *pad, s[0], s[1], _DT[u.dtype], 1 if silu else 0)
    return W, shape, ys, [y.data_ptr() for y in ys] + [None] * len(pad)


def _conv_states(u, W, nseq, initial_states, return_final_states, final_states):
    size = (nseq, W - 1, u.shape[2])
    if initial_states is not None:
        _whole(initial_states, "initial_states", size, u.dtype, u.device)
    if final_states is not None:
        _whole(final_states, "final_states", size, u.dtype, u.device)
    elif return_final_states:
        final_states = u.new_empty(size)
    return final_states


def _conv_result(ys, split, final_states, return_final_states):
    y = ys[0] if split is None else tuple(ys)
    return (y, final_states) if return_final_states else y


def ssd_causal_conv1d(u, weight, bias=None, silu: bool = True, split=None, initial_states=None,
                      return_final_states: bool = False, out=None, final_states=None, stream=None):
    """Depthwise causal convolution of u [b, T, C] along T, with SiLU (Knowl 6, before the layer).

    weight [C, W] fp32, W = 2..4, the last tap on the current token; bias [C] fp32 or None.
    split: sizes of up to three parts of the channels, each returned as its own contiguous
    tensor (a tuple), as ssd_fwd takes x, B and C; None: one tensor.
    initial_states, final_states [b, W-1, C] in u's type: the last tokens before and of the
    sequence. Returns y, or (y, final_states).
    """
    W, shape, ys, yp = _conv_args(u, weight, bias, silu, split, out)
    fin = _conv_states(u, W, u.shape[0], initial_states, return_final_states, final_states)
    _call("ssd_causal_conv1d", u, stream, shape, u.data_ptr(), weight.data_ptr(),
          _ptr(bias), _ptr(initial_states), *yp, _ptr(fin))
    return _conv_result(ys, split, fin, return_final_states)


def ssd_causal_conv1d_varlen(u, weight, bias=None, cu_seqlens=None, silu: bool = True, split=None,
                             initial_states=None, return_final_states: bool = False, out=None,
                             final_states=None, stream=None):
    """ssd_causal_conv1d on a pack of documents (u [1, T, C], as ssd_fwd_varlen): document k is
    tokens cu_seqlens[k] .. cu_seqlens[k+1]-1, with its own states [n_docs, W-1, C].

    cu_seqlens: a device int32 tensor [n_docs + 1] (from 0, at most T; rows behind the last
    document are left as they were), or a host list or tensor from 0 to T (copied).
    """
    W, shape, ys, yp = _conv_args(u, weight, bias, silu, split, out)
    if u.shape[0] != 1:
        raise ValueError("packed documents need batch 1 (u [1, T, C])")
    cu = _offsets(cu_seqlens, u.shape[1], u.device, stream)
    n = cu.numel() - 1
    fin = _conv_states(u, W, n, initial_states, return_final_states, final_states)
    _call("ssd_causal_conv1d_varlen", u, stream, shape, u.data_ptr(), weight.data_ptr(),
          _ptr(bias), cu.data_ptr(), n, _ptr(initial_states), *yp, _ptr(fin))
    return _conv_result(ys, split, fin, return_final_states)


def ssd_causal_conv1d_step(u, weight, bias, state, silu: bool = True, split=None, out=None, stream=None):
    """The convolution of the next tokens u [b, T, C] (or [b, C] for one) from `state`
    [b, W-1, C], which is updated in place; returns y (a tuple with split)."""
    one = isinstance(u, torch.Tensor) and u.dim() == 2
    if one:
        u = u.unsqueeze(1)
        if out is not None:
            out = out.unsqueeze(1) if split is None else [y.unsqueeze(1) for y in out]
    W, shape, ys, yp = _conv_args(u, weight, bias, silu, split, out)
    _whole(state, "state", (u.shape[0], W - 1, u.shape[2]), u.dtype, u.device)
    _call("ssd_causal_conv1d_step", u, stream, shape, u.data_ptr(), weight.data_ptr(),
          _ptr(bias), state.data_ptr(), *yp)
    if one:
        ys = [y.squeeze(1) for y in ys]
    return ys[0] if split is None else tuple(ys)


# ---- the selective scan ----------------------------------------------------

def _check_selective(u, dt, A, B, C, D, z, dt_bias):
    """Raises what is wrong with the scan's inputs."""
    _first(u, "u", 3)
    b, T, Dc = u.shape
    dev, dtype = u.device, u.dtype
    _in(u, "u", u.shape, dtype, dev)
    if not isinstance(dt, torch.Tensor) or dt.dtype not in (_F32, dtype):
        raise TypeError(f"dt must be a float32 or {dtype} tensor")
    _in(dt, "dt", u.shape, dt.dtype, dev)
    if not isinstance(B, torch.Tensor) or B.dim() != 4:
        raise ValueError("B must be [batch, seqlen, ngroups, dstate]")
    G, N = B.shape[2], B.shape[3]
    _in(B, "B", (b, T, G, N), dtype, dev, 2)
    _in(C, "C", (b, T, G, N), dtype, dev, 2)
    _whole(A, "A", (Dc, N), _F32, dev)
    if D is not None:
        _whole(D, "D", (Dc,), _F32, dev)
    if dt_bias is not None:
        _whole(dt_bias, "dt_bias", (Dc,), _F32, dev)
    if z is not None:
        _in(z, "z", u.shape, dtype, dev)


def _vector_ok(t, n, index):
    return t is None or (t.dtype is _F32 and t.shape == (n,) and t.get_device() == index and t.is_contiguous())


def _selective_args(u, dt, A, B, C, D, z, dt_bias, dt_softplus, y):
    """The state size, the checked shape as bytes, the input pointers in the C order, and y."""
    try:       # the checks of _check_selective at once; it says which one failed
        size = u.shape
        b, T, Dc = size
        dtype, index = u.dtype, u.get_device()
        us, ds, bs, cs = u.stride(), dt.stride(), B.stride(), C.stride()
        shape = B.shape
        Bb, BT, G, N = shape
        zs = (0, 0, 1) if z is None else z.stride()
        good = (index >= 0 and dtype in _DT and (dt.dtype is _F32 or dt.dtype is dtype) and dt.shape == size
                and dt.get_device() == index and Bb == b and BT == T and C.shape == shape and B.dtype is dtype
                and C.dtype is dtype and B.get_device() == index and C.get_device() == index
                and (Dc == 1 or us[2] == ds[2] == zs[2] == 1) and (N == 1 or bs[3] == cs[3] == 1)
                and (G == 1 or bs[2] == cs[2] == N) and A.dtype is _F32 and A.shape == (Dc, N)
                and A.get_device() == index and A.is_contiguous() and _vector_ok(D, Dc, index)
                and _vector_ok(dt_bias, Dc, index)
                and (z is None or (z.dtype is dtype and z.shape == size and z.get_device() == index)))
    except (AttributeError, TypeError, ValueError, IndexError):
        good = False
    if not good:
        _check_selective(u, dt, A, B, C, D, z, dt_bias)
        size, dtype = u.shape, u.dtype
        (b, T, Dc), (G, N) = size, B.shape[2:]
        us, ds, bs, cs = u.stride(), dt.stride(), B.stride(), C.stride()
        zs = (0, 0) if z is None else z.stride()
    if y is None:
        y = _like(u)
    else:
        _whole(y, "y", size, dtype, u.device)
    shape = _selective_shape(b, T, Dc, G, N, us[0], us[1], ds[0], ds[1], zs[0], zs[1], bs[0], bs[1], cs[0], cs[1],
                             _DT[dtype], _DT[dt.dtype], 1 if dt_softplus else 0, 0)
    return N, shape, (u.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D),
                      _ptr(z), _ptr(dt_bias)), y


def _selective_states(u, nseq, N, initial_states, return_final_states, final_states):
    size = (nseq, u.shape[2], N)
    if initial_states is not None:
        _whole(initial_states, "initial_states", size, torch.float32, u.device)
    if final_states is not None:
        _whole(final_states, "final_states", size, torch.float32, u.device)
    elif return_final_states:
        final_states = u.new_empty(size, dtype=_F32)
    return final_states


def ssd_selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
                       initial_states=None, return_final_states: bool = False, y=None,
                       final_states=None, stream=None):
    """The selective scan: each of u's [b, T, D] channels with its own steps and decay rates.

        h_t[d, n] = exp(dt_t[d] A[d, n]) h_{t-1}[d, n] + dt_t[d] u_t[d] B_t[g, n]
        y_t[d] = (C_t[g, :] . h_t[d, :] + D[d] u_t[d]) * SiLU(z_t[d])

    dt [b, T, D] fp32 or u's type, through softplus(dt + dt_bias) with dt_softplus (dt + dt_bias
    without); A [D, N] fp32, N up to 256; B, C [b, T, G, N]; D, dt_bias [D] fp32 or None;
    z [b, T, D] or None (no gate). States [b, D, N] fp32. Returns y, or (y, final_states).
    """
    N, shape, ins, y = _selective_args(u, dt, A, B, C, D, z, dt_bias, dt_softplus, y)
    fin = _selective_states(u, u.shape[0], N, initial_states, return_final_states, final_states)
    _call("ssd_selective_scan", u, stream, shape, *ins, _ptr(initial_states), y.data_ptr(),
          _ptr(fin))
    return (y, fin) if return_final_states else y


def ssd_selective_scan_varlen(u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
                              cu_seqlens=None, initial_states=None, return_final_states: bool = False,
                              y=None, final_states=None, stream=None):
    """ssd_selective_scan on a pack of documents (u [1, T, D]) with states [n_docs, D, N];
    cu_seqlens as for ssd_causal_conv1d_varlen."""
    N, shape, ins, y = _selective_args(u, dt, A, B, C, D, z, dt_bias, dt_softplus, y)
    if u.shape[0] != 1:
        raise ValueError("packed documents need batch 1 (u [1, T, D])")
    cu = _offsets(cu_seqlens, u.shape[1], u.device, stream)
    n = cu.numel() - 1
    fin = _selective_states(u, n, N, initial_states, return_final_states, final_states)
    _call("ssd_selective_scan_varlen", u, stream, shape, *ins, cu.data_ptr(), n,
          _ptr(initial_states), y.data_ptr(), _ptr(fin))
    return (y, fin) if return_final_states else y


def ssd_selective_step(u, dt, A, B, C, D, state, z=None, dt_bias=None, dt_softplus: bool = False, y=None,
                       stream=None):
    """The scan of the next tokens from `state` [b, D, N] fp32, which is updated in place; returns y.

    u, dt, z [b, T, D] (or [b, D] for one token), B, C [b, T, G, N] (or [b, G, N]).
    """
    one = isinstance(u, torch.Tensor) and u.dim() == 2
    if one:
        u, dt, B, C, z, y = (t.unsqueeze(1) if isinstance(t, torch.Tensor) else t for t in (u, dt, B, C, z, y))
    N, shape, ins, y = _selective_args(u, dt, A, B, C, D, z, dt_bias, dt_softplus, y)
    _whole(state, "state", (u.shape[0], u.shape[2], N), _F32, u.device)
    _call("ssd_selective_step", u, stream, shape, *ins, state.data_ptr(), y.data_ptr())
    return y.squeeze(1) if one else y
