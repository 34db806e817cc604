"""torch conveniences of the sequence operators: the short causal conv1d and the
selective scan of a state-space block, over prompts and for single tokens.

Like ``conv2d`` and its relatives in ``binding`` they check their arguments (the C
ABI sees pointers only), allocate the output and the workspace with torch, and
enqueue on torch's current stream of the tensors' device; all arithmetic runs in
the library's kernels.  A decoding step is a few microseconds of kernel, so the
checks are kept short: one comparison each, the message made only on failure.
"""
from __future__ import annotations

from ctypes import byref

import torch

from . import binding as B

_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_F32, _I32 = torch.float32, torch.int32
_CONTIGUOUS = torch.contiguous_format
_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty_like = torch.empty_like
_NO_STRIDES = (0, 0, 0)


def _refuse(t, name, shape, dtype, index, contiguous):
    """Raise for the first thing that is wrong with an operand."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, x on cuda:{index}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous" if contiguous else f"the last dimension of {name} must be contiguous")


def _whole(t, name, shape, dtype, index):
    """The pointer of a contiguous operand."""
    try:
        if t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, shape, dtype, index, True)


def _rows(t, name, shape, dtype, index):
    """(pointer, strides) of an operand whose last dimension is contiguous."""
    try:
        if t.get_device() == index and t.dtype is dtype and t.shape == shape:
            s = t.stride()
            if s[-1] == 1 or shape[-1] == 1:
                return t.data_ptr(), s
    except AttributeError:
        pass
    _refuse(t, name, shape, dtype, index, False)


def _input(x, dims):
    """(type code, device index, shape, dtype) of the input that the other operands are held against."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor (the library has no CPU path)")
    dtype = x.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    shape = x.shape
    if len(shape) != dims:
        raise ValueError(f"x must have {dims} dimensions (tokens packed with offsets, or a step: [T, C]; a batch: [N, L, C])")
    return code, x.get_device(), shape, dtype


def _offsets(offsets, index):
    """(pointer, sequences)"""
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be a tensor of n + 1 values")
    return _whole(offsets, "offsets", offsets.shape, _I32, index), offsets.shape[0] - 1


def _cache(state, slots, n, rows, cols, dtype, index):
    """(state pointer, slots pointer, slots in the cache) for n sequences."""
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError(f"state must be a tensor of shape (slots, {rows}, {cols})")
    have = state.shape[0]
    ptr = _whole(state, "state", (have, rows, cols), dtype, index)
    if slots is None:
        if have < n:
            raise ValueError(f"state has {have} slots for {n} sequences")
        return ptr, 0, have
    if have < 1:
        raise ValueError("state has no slots")
    return ptr, _whole(slots, "slots", (n,), _I32, index), have


def _need_state(state, slots, carry):
    if state is None and (carry or slots is not None):
        raise ValueError("carry and slots need a state")


def _filter(w):
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a tensor of shape [C, K]")
    return w.shape[1]


def _activation(name):
    code = B.ACTIVATION.get(name)
    if code is None:
        raise ValueError(f"activation {name!r}: expected None or 'silu'")
    return code


def _enqueue(call, index, *args):
    """call(*args, stream) on torch's current stream of device `index`, that device current."""
    if index == _current_device():
        status = call(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, _stream(index))
    if status != 0:
        raise B.ConvError(status, call.__name__)


def conv1d_causal(x, w, bias=None, activation=None, offsets=None, state=None, slots=None, carry=False, out=None):
    """Short depthwise causal conv1d over prompts, w [C, K] with 2 <= K <= 8, the last
    tap on the token itself: x [N, L, C], or packed [T, C] with int32 offsets [n + 1]
    (rows outside every sequence, or of one whose slot is outside the cache, are left
    as they are: whatever memory held, where out is not given).  The K-1 tokens before a
    sequence are zero, or with carry its slot of state [slots, K-1, C]; the last K-1
    tokens are left in state where one is given.  x may be a slice of wider rows."""
    packed = offsets is not None
    code, index, shape, dtype = _input(x, 2 if packed else 3)
    _need_state(state, slots, carry)
    op, n = _offsets(offsets, index) if packed else (0, shape[0])
    c, k = shape[-1], _filter(w)
    xp, xs = _rows(x, "x", shape, dtype, index)
    wp = _whole(w, "w", (c, k), dtype, index)
    bp = 0 if bias is None else _whole(bias, "bias", (c,), dtype, index)
    sp, ip, have = (0, 0, 0) if state is None else _cache(state, slots, n, k - 1, c, dtype, index)
    if out is None:
        out = _empty_like(x, memory_format=_CONTIGUOUS)
    yp, ys = _rows(out, "out", shape, dtype, index)
    desc = B.CausalConvDesc(n, shape[-2], c, k, _activation(activation), 1 if carry else 0, have,
                            0 if packed else xs[0], xs[-2], 0 if packed else ys[0], ys[-2])
    _enqueue(B._conv1d_causal_forward, index, xp, wp, bp, op, sp, ip, yp, byref(desc), code)
    return out


def conv1d_causal_step(x, w, state, bias=None, activation=None, slots=None, out=None):
    """conv1d_causal for one new token of each of N sequences: x [N, C], the window of
    sequence i in slot i, or slots[i], of state [slots, K-1, C], shifted in place.  A
    sequence whose slot is outside the cache (-1) is left out, its row of out too (which
    holds whatever memory held, where out is not given)."""
    code, index, shape, dtype = _input(x, 2)
    (n, c), k = shape, _filter(w)
    xp, xs = _rows(x, "x", shape, dtype, index)
    wp = _whole(w, "w", (c, k), dtype, index)
    bp = 0 if bias is None else _whole(bias, "bias", (c,), dtype, index)
    sp, ip, have = _cache(state, slots, n, k - 1, c, dtype, index)
    if out is None:
        out = _empty_like(x, memory_format=_CONTIGUOUS)
    yp, ys = _rows(out, "out", shape, dtype, index)
    desc = B.CausalConvDesc(n, 1, c, k, _activation(activation), 1, have, xs[0], 0, ys[0], 0)
    _enqueue(B._conv1d_causal_step_forward, index, xp, wp, bp, sp, ip, yp, byref(desc), code)
    return out


def _states(t, name, lead, g, s, dtype, index):
    """(pointer, strides) of b or c, [..., G, S] with the last two dimensions contiguous."""
    p, st = _rows(t, name, (*lead, g, s), dtype, index)
    if g > 1 and st[-2] != s:
        raise ValueError(f"the last two dimensions of {name} must be contiguous")
    return p, st


def _groups(b, dims, d):
    if not isinstance(b, torch.Tensor) or b.dim() != dims + 1:
        raise ValueError("b must be a tensor of shape [..., G, S]")
    g, s = b.shape[-2:]
    if g < 1 or d % g:
        raise ValueError(f"{g} groups do not divide {d} channels")
    return g, s


def selective_scan(x, dt, a, b, c, d=None, z=None, dt_bias=None, softplus=False, offsets=None, state=None, slots=None,
                   carry=False, out=None, workspace=None):
    """The selective state space recurrence over prompts, per channel and state:
    h_t = exp(delta_t a) h_{t-1} + delta_t b_t x_t, out_t = (c_t . h_t + d x_t) silu(z_t),
    delta_t = dt_t + dt_bias, through log(1 + exp(.)) with softplus.

    x, dt, z [N, L, D], b, c [N, L, G, S], or packed [T, D], [T, G, S] with int32 offsets
    [n + 1] (rows outside every sequence, or of one whose slot is outside the cache, are
    left as they are: whatever memory held, where out is not given); a [D, S], d, dt_bias
    [D] in fp32.  h starts from zero, or with carry from state [slots, D, S] (fp32), and is
    left there where one is given.  x, dt, z, b, c may be slices of wider rows."""
    packed = offsets is not None
    code, index, shape, dtype = _input(x, 2 if packed else 3)
    _need_state(state, slots, carry)
    op, n = _offsets(offsets, index) if packed else (0, shape[0])
    lead, dim = shape[:-1], shape[-1]
    g, s = _groups(b, len(shape), dim)
    xp, xs = _rows(x, "x", shape, dtype, index)
    tp, ts = _rows(dt, "dt", shape, dtype, index)
    bp, bs = _states(b, "b", lead, g, s, dtype, index)
    cp, cs = _states(c, "c", lead, g, s, dtype, index)
    zp, zs = (0, _NO_STRIDES) if z is None else _rows(z, "z", shape, dtype, index)
    ap = _whole(a, "a", (dim, s), _F32, index)
    dp = 0 if d is None else _whole(d, "d", (dim,), _F32, index)
    up = 0 if dt_bias is None else _whole(dt_bias, "dt_bias", (dim,), _F32, index)
    sp, ip, have = (0, 0, 0) if state is None else _cache(state, slots, n, dim, s, _F32, index)
    if out is None:
        out = _empty_like(x, memory_format=_CONTIGUOUS)
    yp, ys = _rows(out, "out", shape, dtype, index)
    t = len(shape) - 2                                  # the token dimension; a packed call has no batch before it
    batch = (lambda st: 0) if packed else (lambda st: st[0])
    desc = B.ScanDesc(n, shape[t], dim, s, g, 1 if softplus else 0, 1 if carry else 0, have, 1 if packed else 0, batch(xs), xs[t], batch(ts),
                      ts[t], batch(zs), zs[t], batch(bs), bs[t], batch(cs), cs[t], batch(ys), ys[t])
    need = B._selective_scan_workspace_size(byref(desc), code, index)
    if workspace is not None:
        B._check_workspace(workspace, need, x)
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif need:
        workspace = x.new_empty(need, dtype=torch.uint8)
        wp, wn = workspace.data_ptr(), need
    else:
        wp = wn = 0
    tensors = B.ScanTensors(xp, tp, bp, cp, zp, ap, dp, up, op, ip, sp, yp)
    _enqueue(B._selective_scan_forward, index, byref(tensors), byref(desc), code, wp, wn)
    return out


def selective_scan_step(x, dt, a, b, c, state, d=None, z=None, dt_bias=None, softplus=False, slots=None, out=None):
    """selective_scan for one new token of each of N sequences: x, dt, z [N, D], b, c
    [N, G, S], the state of sequence i in slot i, or slots[i], of state [slots, D, S]
    (fp32), advanced in place.  A sequence whose slot is outside the cache (-1) is left
    out, its row of out too (which holds whatever memory held, where out is not given)."""
    code, index, shape, dtype = _input(x, 2)
    n, dim = shape
    g, s = _groups(b, 2, dim)
    xp, xs = _rows(x, "x", shape, dtype, index)
    tp, ts = _rows(dt, "dt", shape, dtype, index)
    bp, bs = _states(b, "b", (n,), g, s, dtype, index)
    cp, cs = _states(c, "c", (n,), g, s, dtype, index)
    zp, zs = (0, _NO_STRIDES) if z is None else _rows(z, "z", shape, dtype, index)
    ap = _whole(a, "a", (dim, s), _F32, index)
    dp = 0 if d is None else _whole(d, "d", (dim,), _F32, index)
    up = 0 if dt_bias is None else _whole(dt_bias, "dt_bias", (dim,), _F32, index)
    sp, ip, have = _cache(state, slots, n, dim, s, _F32, index)
    if out is None:
        out = _empty_like(x, memory_format=_CONTIGUOUS)
    yp, ys = _rows(out, "out", shape, dtype, index)
    desc = B.ScanDesc(n, 1, dim, s, g, 1 if softplus else 0, 1, have, 0, xs[0], 0, ts[0], 0, zs[0], 0, bs[0], 0, cs[0], 0,
                      ys[0], 0)
    tensors = B.ScanTensors(xp, tp, bp, cp, zp, ap, dp, up, 0, ip, sp, yp)
    _enqueue(B._selective_scan_step_forward, index, byref(tensors), byref(desc), code)
    return out
