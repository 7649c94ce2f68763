"""Python binding of the sequence-block operators in libcfc.so
(include/seq.h): layer norm, dropout, causal convolution and selective scan,
each forward and backward, the last two also for single tokens.

Argument marshalling only: every operator runs in the HIP kernels of libcfc.so
on the current stream; torch tensors provide device memory.  There is no
fallback: a missing library or a failed call raises.

Activations are float32, bfloat16 or float16 (one type per call), parameters,
states and parameter gradients float32.  An activation's last axis is dense
and its rows lie at one stride, so ``xz[..., :D]`` is passed as it is.
Sequences are [S, L, D], or packed rows [T, D] with ``cu_seqlens`` (int32,
S + 1 values from 0 to T, on the GPU); [T, D] alone is one sequence.  Outputs
given by the caller are overwritten and returned, others are allocated.
"""
import ctypes
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import cfc as _cfc

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_U64 = ctypes.c_uint64
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_LIB = None


def _raw_stream(index):
    """The current stream's handle (the raw getter where torch has it: the
    Stream object costs more than a small kernel)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


class _Scan(ctypes.Structure):
    _fields_ = [("u", _P), ("ldu", _I64), ("dt", _P), ("lddt", _I64), ("z", _P), ("ldz", _I64), ("B", _P), ("ldb", _I64),
                ("C", _P), ("ldc", _I64), ("A", _P), ("skip", _P), ("dt_bias", _P), ("h0", _P), ("cu_seqlens", _P),
                ("total", _I64), ("len", _I64), ("n_seq", _I), ("D", _I), ("N", _I), ("G", _I), ("softplus", _I), ("dtype", _I)]


class _ScanGrads(ctypes.Structure):
    _fields_ = [("du", _P), ("lddu", _I64), ("ddt", _P), ("ldddt", _I64), ("dz", _P), ("lddz", _I64), ("dB", _P), ("dC", _P),
                ("dA", _P), ("dskip", _P), ("ddt_bias", _P), ("dh0", _P)]


def lib():
    """libcfc.so with the sequence operators' signatures declared."""
    global _LIB
    if _LIB is None:
        L = _cfc.lib()
        SP = ctypes.POINTER(_Scan)
        ints = {
            "seq_layer_norm_fwd": [_P, _I64, _P, _P, _P, _I64, _P, _P, _I64, _I, _F, _I, _P],
            "seq_layer_norm_bwd": [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _P, _I64, _I, _I, _P, _SZ, _P],
            "seq_dropout_fwd": [_P, _I64, _P, _I64, _P, _I64, _I64, _I64, ctypes.c_double, _U64, _U64, _I, _P],
            "seq_dropout_bwd": [_P, _I64, _P, _I64, _I64, _I64, ctypes.c_double, _U64, _U64, _I, _P],
            "seq_causal_conv_fwd": [_P, _I64, _P, _P, _P, _P, _I64, _P, _P, _I, _I64, _I64, _I, _I, _I, _I, _P],
            "seq_causal_conv_bwd": [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _P, _P, _I, _I64, _I64, _I, _I, _I, _I,
                                    _P, _SZ, _P],
            "seq_causal_conv_step": [_P, _I64, _P, _P, _P, _P, _I64, _I64, _I, _I, _I, _I, _P],
            "seq_selective_scan_fwd": [SP, _P, _I64, _P, _P, _P, _SZ, _P],
            "seq_selective_scan_bwd": [SP, _P, _I64, _P, _P, ctypes.POINTER(_ScanGrads), _P, _SZ, _P],
            "seq_selective_scan_step": [_P, _P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _P, _I64, _P, _P, _I64,
                                        _I64, _I, _I, _I, _I, _I, _P],
        }
        sizes = {
            "seq_layer_norm_bwd_workspace_bytes": [_I64, _I, _I],
            "seq_causal_conv_bwd_workspace_bytes": [_I, _I64, _I64, _I, _I, _I],
            "seq_selective_scan_hist_floats": [SP],
            "seq_selective_scan_fwd_workspace_bytes": [SP],
            "seq_selective_scan_bwd_workspace_bytes": [SP],
        }
        for table, res in ((ints, _I), (sizes, _SZ)):
            for name, args in table.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = res
        _LIB = L
    return _LIB


# ---------------------------------------------------------------- arguments

def _rows(t, name, like=None):
    """(address, row stride) of an activation: the last axis dense, all other
    axes one run of rows.  `like`: the activation whose type, device and shape
    it shares."""
    if like is None:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("%s must be a GPU tensor" % name)
        if t.dtype not in _TYPES:
            raise TypeError("%s must be float32, bfloat16 or float16" % name)
        if t.dim() < 2:
            raise ValueError("%s needs rows and columns" % name)
    else:
        if not isinstance(t, torch.Tensor) or t.dtype != like.dtype or t.get_device() != like.get_device():
            raise TypeError("%s must be %s on %s" % (name, like.dtype, like.device))
        if t.shape != like.shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(like.shape)))
    if t.is_contiguous():
        return t.data_ptr(), t.shape[-1]
    return t.data_ptr(), _row_stride(t, name, t.dim() - 1)


def _out(t, name, like):
    """(tensor, address, row stride) of an output shaped as `like`, allocated if
    not given."""
    if t is None:
        t = torch.empty(like.shape, dtype=like.dtype, device=like.device)
        return t, t.data_ptr(), like.shape[-1]
    return (t,) + _rows(t, name, like)


def _row_stride(t, name, lead):
    """The stride of the rows that the first `lead` axes form, the others dense."""
    if t.is_contiguous():
        return math.prod(t.shape[lead:])
    shape, stride = t.shape, t.stride()
    n = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] != 1 and stride[i] != n:
            raise TypeError("%s must be dense from axis %d on" % (name, lead))
        n *= shape[i]
    ld = None
    step = 0
    for i in range(lead - 1, -1, -1):
        if shape[i] == 1:
            continue
        if ld is None:
            ld = stride[i]
            step = ld * shape[i]
        elif stride[i] != step:
            raise TypeError("the rows of %s must lie at one stride" % name)
        else:
            step *= shape[i]
    if ld is None:
        return n
    if ld < n:
        raise TypeError("the rows of %s overlap" % name)
    return ld


def _f32(t, name, shape, like):
    """Address of a contiguous float32 tensor on `like`'s device, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != like.get_device():
        raise TypeError("%s must be a tensor on %s" % (name, like.device))
    if t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError("%s must be contiguous float32" % name)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    return t.data_ptr()


def _dense(t, name, shape, like):
    """Address of a dense tensor of the activations' type."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != like.get_device() or t.dtype != like.dtype \
            or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %s tensor on %s" % (name, like.dtype, like.device))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    return t.data_ptr()


def _call(fn, t, *args):
    """Enqueues fn on the current stream of t's device."""
    dev = t.get_device()
    f = getattr(_LIB or lib(), fn)
    if torch.cuda.current_device() == dev:
        rc = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(dev))
    if rc:
        raise _cfc.CfcError(fn, rc, _cfc.last_error())


def _seqs(x, cu_seqlens):
    """(n_seq, total, len, cu address) of an activation's rows."""
    if cu_seqlens is None:
        if x.dim() == 2:
            return 1, x.shape[0], x.shape[0], None
        if x.dim() == 3:
            return x.shape[0], x.shape[0] * x.shape[1], x.shape[1], None
        raise ValueError("sequences are [S, L, D], or [T, D]")
    if x.dim() != 2:
        raise ValueError("with cu_seqlens the rows are packed: [T, D]")
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.get_device() != x.get_device() or cu_seqlens.dtype != torch.int32 \
            or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 1:
        raise TypeError("cu_seqlens must be contiguous int32 [S + 1] on %s" % x.device)
    return cu_seqlens.numel() - 1, x.shape[0], 0, cu_seqlens.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _space(ws, need, like):
    """(tensor to keep, address, bytes) of a given or allocated workspace."""
    if ws is None:
        if not need:
            return None, None, 0
        ws = torch.empty((need + 3) // 4, dtype=torch.float32, device=like.device)
        return ws, ws.data_ptr(), need
    if not isinstance(ws, torch.Tensor) or ws.get_device() != like.get_device() or not ws.is_contiguous():
        raise TypeError("ws must be a contiguous tensor on %s" % like.device)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


# ---------------------------------------------------------------- layer norm

def layer_norm_fwd(x, w=None, b=None, eps=1e-5, y=None, mean=None, rstd=None):
    """(y, mean, rstd): the last axis normalised, then times w plus b; mean and
    rstd [rows] are what the backward pass reads."""
    px, ldx = _rows(x, "x")
    C, dev = x.shape[-1], x.device
    M = x.numel() // C if C else 0
    y, py, ldy = _out(y, "y", x)
    if mean is None:
        mean = torch.empty(M, dtype=torch.float32, device=dev)
    if rstd is None:
        rstd = torch.empty(M, dtype=torch.float32, device=dev)
    _call("seq_layer_norm_fwd", x, px, ldx, _f32(w, "w", (C,), x), _f32(b, "b", (C,), x), py, ldy,
          _f32(mean, "mean", (M,), x), _f32(rstd, "rstd", (M,), x), M, C, eps, _TYPES[x.dtype])
    return y, mean, rstd


def layer_norm_bwd(dy, x, w, mean, rstd, dx=None, dw=None, db=None, params=True, ws=None):
    """(dx, dw, db); with params=False dw and db are not formed (None)."""
    px, ldx = _rows(x, "x")
    pdy, lddy = _rows(dy, "dy", x)
    C, dev, t = x.shape[-1], x.device, _TYPES[x.dtype]
    M = x.numel() // C if C else 0
    dx, pdx, lddx = _out(dx, "dx", x)
    need = 0
    if params:
        if dw is None:
            dw = torch.empty(C, dtype=torch.float32, device=dev)
        if db is None:
            db = torch.empty(C, dtype=torch.float32, device=dev)
        need = lib().seq_layer_norm_bwd_workspace_bytes(M, C, t)
    elif dw is not None or db is not None:
        raise ValueError("dw and db need params=True")
    ws, pws, nws = _space(ws, need, x)
    _call("seq_layer_norm_bwd", x, pdy, lddy, px, ldx, _f32(w, "w", (C,), x), _f32(mean, "mean", (M,), x),
          _f32(rstd, "rstd", (M,), x), pdx, lddx, _f32(dw, "dw", (C,), x), _f32(db, "db", (C,), x), M, C, t, pws, nws)
    return dx, dw, db


# ---------------------------------------------------------------- dropout

def _philox_key(seed, offset):
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
        raise ValueError("seed and offset are in [0, 2^64)")
    return seed, offset


def dropout_fwd(x, p, seed, offset=0, residual=None, y=None):
    """y = residual + keep * x / (1 - p).  What is kept follows from seed, offset
    and an element's place alone; a call uses ceil(numel / 4) offsets."""
    px, ldx = _rows(x, "x")
    C = x.shape[-1]
    seed, offset = _philox_key(seed, offset)
    pr, ldr = (None, 0) if residual is None else _rows(residual, "residual", x)
    y, py, ldy = _out(y, "y", x)
    _call("seq_dropout_fwd", x, px, ldx, pr, ldr, py, ldy, x.numel() // C if C else 0, C, p, seed, offset, _TYPES[x.dtype])
    return y


def dropout_bwd(dy, p, seed, offset=0, dx=None):
    """dx = keep * dy / (1 - p) with the forward pass's p, seed and offset."""
    pdy, lddy = _rows(dy, "dy")
    C = dy.shape[-1]
    seed, offset = _philox_key(seed, offset)
    dx, pdx, lddx = _out(dx, "dx", dy)
    _call("seq_dropout_bwd", dy, pdy, lddy, pdx, lddx, dy.numel() // C if C else 0, C, p, seed, offset, _TYPES[dy.dtype])
    return dx


# ---------------------------------------------------------------- convolution

def _taps(w, b, D, like):
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w is [D, K]")
    K = w.shape[1]
    return K, _f32(w, "w", (D, K), like), _f32(b, "b", (D,), like)


def causal_conv_fwd(x, w, b=None, silu=True, state=None, cu_seqlens=None, y=None, state_out=None):
    """y_t = act(b + sum_k w[:, k] x_{t - K + 1 + k}) per channel.  `state`
    [S, K - 1, D]: the inputs before each sequence (zeros if None); `state_out`
    of that shape gets the last K - 1, which causal_conv_step carries on."""
    px, ldx = _rows(x, "x")
    D = x.shape[-1]
    K, pw, pb = _taps(w, b, D, x)
    S, total, L, cu = _seqs(x, cu_seqlens)
    y, py, ldy = _out(y, "y", x)
    _call("seq_causal_conv_fwd", x, px, ldx, pw, pb, _dense(state, "state", (S, K - 1, D), x), py, ldy,
          _dense(state_out, "state_out", (S, K - 1, D), x), cu, S, total, L, D, K, 1 if silu else 0, _TYPES[x.dtype])
    return y


def causal_conv_bwd(dy, x, w, b=None, silu=True, state=None, cu_seqlens=None, dx=None, dw=None, db=None, ws=None):
    """(dx, dw [D, K], db [D]) with the forward pass's arguments."""
    px, ldx = _rows(x, "x")
    pdy, lddy = _rows(dy, "dy", x)
    D, dev = x.shape[-1], x.device
    K, pw, pb = _taps(w, b, D, x)
    S, total, L, cu = _seqs(x, cu_seqlens)
    dx, pdx, lddx = _out(dx, "dx", x)
    if dw is None:
        dw = torch.empty((D, K), dtype=torch.float32, device=dev)
    if db is None:
        db = torch.empty((D,), dtype=torch.float32, device=dev)
    need = lib().seq_causal_conv_bwd_workspace_bytes(S, total, L, 0 if cu is None else 1, D, K)
    ws, pws, nws = _space(ws, need, x)
    _call("seq_causal_conv_bwd", x, pdy, lddy, px, ldx, pw, pb, _dense(state, "state", (S, K - 1, D), x), pdx, lddx,
          _f32(dw, "dw", (D, K), x), _f32(db, "db", (D,), x), cu, S, total, L, D, K, 1 if silu else 0, _TYPES[x.dtype],
          pws, nws)
    return dx, dw, db


def causal_conv_step(x, state, w, b=None, silu=True, y=None):
    """One token of each sequence: y [S, D] from x [S, D]; `state` [S, K - 1, D]
    is shifted by x in place."""
    px, ldx = _rows(x, "x")
    if x.dim() != 2:
        raise ValueError("x is [S, D]")
    S, D = x.shape
    K, pw, pb = _taps(w, b, D, x)
    if state is None:
        raise TypeError("state must be a tensor")
    y, py, ldy = _out(y, "y", x)
    _call("seq_causal_conv_step", x, px, ldx, _dense(state, "state", (S, K - 1, D), x), pw, pb, py, ldy, S, D, K,
          1 if silu else 0, _TYPES[x.dtype])
    return y


# ---------------------------------------------------------------- scan

@dataclass
class Scan:
    """What selective_scan_fwd gives."""
    y: torch.Tensor               # as u
    h_last: torch.Tensor          # [S, N, D] float32
    hist: Optional[torch.Tensor]  # the states the backward pass starts from (save=True)


@dataclass
class ScanGrads:
    """What selective_scan_bwd gives; None where the input was not given."""
    du: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dskip: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]
    dh0: Optional[torch.Tensor]


def _groups(t, name, u, N):
    """(address, row stride, G) of B or C: [..., G, N] or, for one group, [..., N]."""
    if not isinstance(t, torch.Tensor) or t.dtype != u.dtype or t.get_device() != u.get_device():
        raise TypeError("%s must be %s on %s" % (name, u.dtype, u.device))
    lead, shape = u.dim() - 1, t.shape
    more = len(shape) - lead
    if more not in (1, 2) or shape[:lead] != u.shape[:lead] or shape[-1] != N:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(shape), tuple(u.shape[:lead]) + ("G", N)))
    return t.data_ptr(), _row_stride(t, name, lead), shape[-2] if more == 2 else 1


def _scan_args(u, dt, A, B, C, skip, z, dt_bias, softplus, h0, cu_seqlens):
    pu, ldu = _rows(u, "u")
    pdt, lddt = _rows(dt, "dt", u)
    pz, ldz = (None, 0) if z is None else _rows(z, "z", u)
    D = u.shape[-1]
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A is [N, D]")
    N = A.shape[0]
    pB, ldb, G = _groups(B, "B", u, N)
    pC, ldc, GC = _groups(C, "C", u, N)
    if G != GC or B.dim() != C.dim():
        raise ValueError("B and C have different groups")
    S, total, L, cu = _seqs(u, cu_seqlens)
    return _Scan(pu, ldu, pdt, lddt, pz, ldz, pB, ldb, pC, ldc, _f32(A, "A", (N, D), u), _f32(skip, "skip", (D,), u),
                 _f32(dt_bias, "dt_bias", (D,), u), _f32(h0, "h0", (S, N, D), u), cu, total, L, S, D, N, G,
                 1 if softplus else 0, _TYPES[u.dtype])


def selective_scan_fwd(u, dt, A, B, C, skip=None, z=None, dt_bias=None, softplus=True, h0=None, cu_seqlens=None, save=False,
                       y=None, h_last=None, ws=None):
    """The scan over whole sequences: u, dt, z as [S, L, D] (or packed), A [N, D]
    (negative for a state that decays), B and C [..., G, N].  save=True keeps
    what selective_scan_bwd needs in `hist`."""
    a = _scan_args(u, dt, A, B, C, skip, z, dt_bias, softplus, h0, cu_seqlens)
    dev = u.device
    y, py, ldy = _out(y, "y", u)
    shape = (a.n_seq, a.N, a.D)
    if h_last is None:
        h_last = torch.empty(shape, dtype=torch.float32, device=dev)
    hist = torch.empty(lib().seq_selective_scan_hist_floats(a), dtype=torch.float32, device=dev) if save else None
    ws, pws, nws = _space(ws, lib().seq_selective_scan_fwd_workspace_bytes(a), u)
    _call("seq_selective_scan_fwd", u, a, py, ldy, _f32(h_last, "h_last", shape, u), _ptr(hist), pws, nws)
    return Scan(y, h_last, hist)


def selective_scan_bwd(dy, u, dt, A, B, C, hist, skip=None, z=None, dt_bias=None, softplus=True, h0=None, cu_seqlens=None,
                       dh_last=None, du=None, ddt=None, dz=None, ws=None):
    """Every gradient of sum(dy y) + sum(dh_last h_last), with the forward
    pass's arguments and its hist; dh0 is formed when h0 is given.  du, ddt and
    dz may be given, as halves of one buffer for instance."""
    a = _scan_args(u, dt, A, B, C, skip, z, dt_bias, softplus, h0, cu_seqlens)
    dev = u.device
    pdy, lddy = _rows(dy, "dy", u)
    if hist is None:
        raise ValueError("hist: run selective_scan_fwd with save=True")
    phist = _f32(hist, "hist", (lib().seq_selective_scan_hist_floats(a),), u)

    du, pdu, lddu = _out(du, "du", u)
    ddt, pddt, ldddt = _out(ddt, "ddt", u)
    pdz, lddz = None, 0
    if z is not None:
        dz, pdz, lddz = _out(dz, "dz", u)
    elif dz is not None:
        raise ValueError("dz without z")
    dB = torch.empty(B.shape, dtype=B.dtype, device=dev)
    dC = torch.empty(C.shape, dtype=C.dtype, device=dev)
    dA = torch.empty((a.N, a.D), dtype=torch.float32, device=dev)
    dskip = None if skip is None else torch.empty((a.D,), dtype=torch.float32, device=dev)
    ddt_bias = None if dt_bias is None else torch.empty((a.D,), dtype=torch.float32, device=dev)
    dh0 = None if h0 is None else torch.empty((a.n_seq, a.N, a.D), dtype=torch.float32, device=dev)
    g = _ScanGrads(pdu, lddu, pddt, ldddt, pdz, lddz, dB.data_ptr(), dC.data_ptr(), dA.data_ptr(), _ptr(dskip), _ptr(ddt_bias),
                   _ptr(dh0))
    ws, pws, nws = _space(ws, lib().seq_selective_scan_bwd_workspace_bytes(a), u)
    _call("seq_selective_scan_bwd", u, a, pdy, lddy, phist, _f32(dh_last, "dh_last", (a.n_seq, a.N, a.D), u), g, pws, nws)
    return ScanGrads(du, ddt, dA, dB, dC, dskip, dz, ddt_bias, dh0)


def selective_scan_step(h, u, dt, A, B, C, skip=None, z=None, dt_bias=None, softplus=True, y=None):
    """One token of each sequence: y [S, D]; the state h [S, N, D] is updated in
    place."""
    pu, ldu = _rows(u, "u")
    if u.dim() != 2:
        raise ValueError("u is [S, D]")
    S, D = u.shape
    pdt, lddt = _rows(dt, "dt", u)
    pz, ldz = (None, 0) if z is None else _rows(z, "z", u)
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A is [N, D]")
    N = A.shape[0]
    pB, ldb, G = _groups(B, "B", u, N)
    pC, ldc, GC = _groups(C, "C", u, N)
    if G != GC:
        raise ValueError("B and C have different groups")
    if h is None:
        raise TypeError("h must be a tensor")
    y, py, ldy = _out(y, "y", u)
    _call("seq_selective_scan_step", u, _f32(h, "h", (S, N, D), u), pu, ldu, pdt, lddt, _f32(A, "A", (N, D), u), pB, ldb,
          pC, ldc, _f32(skip, "skip", (D,), u), pz, ldz, _f32(dt_bias, "dt_bias", (D,), u), py, ldy, S, D, N, G,
          1 if softplus else 0, _TYPES[u.dtype])
    return y
