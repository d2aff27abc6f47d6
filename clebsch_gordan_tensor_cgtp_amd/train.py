"""The node-side operators of a training step, over the C ABI of
include/cgtp_train.h: embedding of species (token) ids and its gradient, group
normalisation with an activation over ragged segments and its gradient, the
orthogonalised update of a stack of weight matrices.

Each function checks types, devices and shapes, allocates outputs and
workspace with torch (device memory only) unless they are given, and calls the
library on the current HIP stream of the arrays' device.  Large arrays are
float32 or bfloat16; statistics, gamma, beta and their gradients float32;
indices int32.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.CGTP_F32, torch.bfloat16: L.CGTP_BF16}
_ACTS = {"none": L.CGTP_ACT_NONE, "silu": L.CGTP_ACT_SILU, "tanh": L.CGTP_ACT_TANH}


def _dtype(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return d


def _need(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name):
    """Row stride of an array of rows: [N][C], or [B][S][C] with one stride for
    all rows; the channels are contiguous."""
    shape = t.shape
    width = shape[-1]
    if t.is_contiguous():
        return width
    stride = t.stride()
    if width > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    n = t.numel() // width if width else 0
    if n <= 1:
        return width
    if len(shape) == 2:
        ld = stride[0]
    elif shape[1] > 1:
        ld = stride[1]
        if shape[0] > 1 and stride[0] != ld * shape[1]:
            raise ValueError(f"{name}: rows must be equally spaced")
    else:
        ld = stride[0]
    if ld < width:
        raise ValueError(f"{name}: rows overlap")
    return ld


def _like(t, name, dtype, shape, device):
    """An array of rows given by the caller: type, device and shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _workspace(ws, nbytes, device):
    """(address, bytes, tensor) of the workspace, allocated here if not given."""
    if ws is None:
        if nbytes == 0:
            return None, 0, None
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return ws.data_ptr(), nbytes, ws
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise TypeError("ws must be a contiguous torch.uint8 tensor")
    if ws.device != device:
        raise ValueError(f"ws is on {ws.device}, expected {device}")
    return ws.data_ptr(), ws.numel(), ws


_functions = {}  # of the library, by name


def _function(name):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(L.lib(), name)
    return f


def _call(name, device, *args):
    """The library call `name` on the device's current stream.  (These calls
    can be a few microseconds long, so the stream's handle is asked for
    directly: building a Stream object around it takes 2 us.)"""
    if device.type != "cuda":
        raise ValueError(f"{name} needs arrays on a GPU, got {device}")
    index = device.index
    if index == torch._C._cuda_getDevice():
        status = _function(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = _function(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != L.CGTP_OK:
        L.check(name, status)


@functools.lru_cache(maxsize=256)  # of sizes alone
def _bytes(name, *args):
    b = ctypes.c_size_t()
    L.check(name, _function(name)(*args, ctypes.byref(b)))
    return b.value


# ---- embedding -------------------------------------------------------------------
def embed_fwd(ids, table, scale: float = 1.0, out=None) -> torch.Tensor:
    """out[n] = scale * table[ids[n]], zeros where ids[n] is outside the table
    (padding).  ids [N] int32, table [V][C]; ``out`` [N][C] may be a view with
    a row stride, such as the l = 0 rows ``x[:, 0, :]`` of node features."""
    d = _dtype(table, "table")
    if table.dim() != 2:
        raise ValueError("table must be [V][C]")
    V, C, dev = table.shape[0], table.shape[1], table.device
    if not isinstance(ids, torch.Tensor) or ids.dim() != 1:
        raise TypeError("ids must be a torch.Tensor [N]")
    N = ids.shape[0]
    _need(ids, "ids", torch.int32, (N,), dev)
    _need(table, "table", table.dtype, (V, C), dev)
    if out is None:
        out, ldo = table.new_empty((N, C)), C
    else:
        _like(out, "out", table.dtype, (N, C), dev)
        ldo = _rows(out, "out")
    _call("cgtp_embed_fwd", dev, d, N, V, C, ids.data_ptr(), table.data_ptr(), scale, out.data_ptr(), ldo)
    return out


def embed_bwd_workspace_size(dtype, n_rows: int, table_rows: int, channels: int) -> int:
    return _bytes("cgtp_embed_bwd_workspace_size", _DTYPES[dtype], n_rows, table_rows, channels)


def embed_bwd(ids, grad_out, table_rows: int, scale: float = 1.0, grad_table=None, ws=None) -> torch.Tensor:
    """grad_table[v] = scale * sum of grad_out[n] over the n with ids[n] = v
    (zeros for rows that no id names; ids outside the table are ignored), of
    <grad_out, embed_fwd(ids, table, scale)>.  grad_out [N][C] may have a row
    stride; every row of grad_table [table_rows][C] is written."""
    d = _dtype(grad_out, "grad_out")
    if grad_out.dim() != 2:
        raise ValueError("grad_out must be [N][C]")
    N, C, dev = grad_out.shape[0], grad_out.shape[1], grad_out.device
    _need(ids, "ids", torch.int32, (N,), dev)
    ld = _rows(grad_out, "grad_out")
    nbytes = _bytes("cgtp_embed_bwd_workspace_size", d, N, table_rows, C)
    if grad_table is None:
        grad_table = grad_out.new_empty((table_rows, C))
    else:
        _need(grad_table, "grad_table", grad_out.dtype, (table_rows, C), dev)
    at, room, ws = _workspace(ws, nbytes, dev)  # (held until the call is out)
    _call("cgtp_embed_bwd", dev, d, N, table_rows, C, ids.data_ptr(), grad_out.data_ptr(), ld, scale,
          grad_table.data_ptr(), at, room)
    return grad_table


# ---- group normalisation with an activation ------------------------------------------
def _norm_shape(x, groups, seg_ptr):
    """(N, B, C) of [N][C] rows (one segment, or seg_ptr's) or [B][S][C] rows
    (B segments of S rows)."""
    shape = x.shape
    dim = len(shape)
    if dim != 2 and dim != 3:
        raise ValueError("x must be [N][C] or [B][S][C]")
    C = shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"groups = {groups} does not divide the {C} channels")
    if seg_ptr is None:
        return (shape[0], 1, C) if dim == 2 else (shape[0] * shape[1], shape[0], C)
    if dim != 2:
        raise ValueError("seg_ptr needs x as [N][C]")
    if not isinstance(seg_ptr, torch.Tensor) or seg_ptr.dim() != 1 or seg_ptr.shape[0] < 1:
        raise TypeError("seg_ptr must be a torch.Tensor [segments + 1]")
    _need(seg_ptr, "seg_ptr", torch.int32, seg_ptr.shape, x.device)
    return shape[0], seg_ptr.shape[0] - 1, C


def _act(act):
    a = _ACTS.get(act)
    if a is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return a


def _channel(t, name, C, dev):
    if t is None:
        return None
    _need(t, name, torch.float32, (C,), dev)
    return t.data_ptr()


def norm_act_workspace_size(dtype, n_rows: int, n_segments: int, channels: int, groups: int, ragged: bool,
                            backward: bool) -> int:
    return _bytes("cgtp_norm_act_workspace_size", _DTYPES[dtype], n_rows, n_segments, channels, groups, int(ragged),
                  int(backward))


def norm_act_fwd(x, gamma, beta, groups: int, seg_ptr=None, eps: float = 1e-5, act: str = "silu", out=None, ws=None):
    """(y, mean, rstd): y = act((x - mean) * rstd * gamma + beta) with the mean
    and deviation of each segment's groups of channels.

    x: [N][C] rows cut into segments by ``seg_ptr`` [B+1] int32 (the atoms of
    each structure of a batch; one segment without it), or [B][S][C] equal
    segments; rows may have a stride (``features[:, 0, :]``).  gamma, beta [C]
    float32 or None (ones, zeros).  act: "none", "silu" or "tanh".  mean and
    rstd are [B][groups] float32."""
    d = _dtype(x, "x")
    N, B, C = _norm_shape(x, groups, seg_ptr)
    dev = x.device
    ldx = _rows(x, "x")
    g, b = _channel(gamma, "gamma", C, dev), _channel(beta, "beta", C, dev)
    nbytes = _bytes("cgtp_norm_act_workspace_size", d, N, B, C, groups, int(seg_ptr is not None), 0)
    if out is None:
        out, ldo = x.new_empty(x.shape), C
    else:
        _like(out, "out", x.dtype, x.shape, dev)
        ldo = _rows(out, "out")
    stats = torch.empty((2, B, groups), dtype=torch.float32, device=dev)
    mean, rstd = stats.unbind(0)
    at, room, ws = _workspace(ws, nbytes, dev)  # (held until the call is out)
    _call("cgtp_norm_act_fwd", dev, d, _act(act), N, B, C, groups, None if seg_ptr is None else seg_ptr.data_ptr(),
          eps, x.data_ptr(), ldx, g, b, out.data_ptr(), ldo, mean.data_ptr(), rstd.data_ptr(),
          at, room)
    return out, mean, rstd


def norm_act_bwd(x, mean, rstd, gamma, beta, grad_y, groups: int, seg_ptr=None, act: str = "silu",
                 want=("x", "gamma", "beta"), ws=None, grad_x=None):
    """(grad_x, grad_gamma, grad_beta) of <grad_y, y> for norm_act_fwd's y on
    the same arguments and its mean and rstd; a gradient not in ``want`` comes
    back as None.  ``grad_x`` of x's shape may be a view with a row stride, such
    as the l = 0 rows of a gradient of node features."""
    d = _dtype(x, "x")
    N, B, C = _norm_shape(x, groups, seg_ptr)
    dev = x.device
    _like(grad_y, "grad_y", x.dtype, x.shape, dev)
    _need(mean, "mean", torch.float32, (B, groups), dev)
    _need(rstd, "rstd", torch.float32, (B, groups), dev)
    g, b = _channel(gamma, "gamma", C, dev), _channel(beta, "beta", C, dev)
    ldx, ldy = _rows(x, "x"), _rows(grad_y, "grad_y")
    nbytes = _bytes("cgtp_norm_act_workspace_size", d, N, B, C, groups, int(seg_ptr is not None), 1)
    if "x" not in want:
        gx, ldd = None, C
    elif grad_x is None:
        gx, ldd = x.new_empty(x.shape), C
    else:
        _like(grad_x, "grad_x", x.dtype, x.shape, dev)
        gx, ldd = grad_x, _rows(grad_x, "grad_x")
    gg = torch.empty(C, dtype=torch.float32, device=dev) if "gamma" in want else None
    gb = torch.empty(C, dtype=torch.float32, device=dev) if "beta" in want else None
    at, room, ws = _workspace(ws, nbytes, dev)  # (held until the call is out)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _call("cgtp_norm_act_bwd", dev, d, _act(act), N, B, C, groups, ptr(seg_ptr), x.data_ptr(), ldx, mean.data_ptr(),
          rstd.data_ptr(), g, b, grad_y.data_ptr(), ldy, ptr(gx), ldd, ptr(gg), ptr(gb), at, room)
    return gx, gg, gb


# ---- orthogonalised update -------------------------------------------------------------
def orthogonalize_workspace_size(dtype, batch: int, rows: int, cols: int) -> int:
    return _bytes("cgtp_orthogonalize_workspace_size", _DTYPES[dtype], batch, rows, cols)


def orthogonalize(grad, steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, scale: float = 1.0,
                  out=None, ws=None) -> torch.Tensor:
    """scale times ``steps`` Newton-Schulz steps of a x + b x^3 + c x^5
    (``coeffs``) on the singular values of each matrix of ``grad`` [..., rows,
    cols], taken first to grad / (Frobenius norm + eps): the update direction
    of weight matrices such as path_mix_fwd's Wmix [P][C][C_out]."""
    d = _dtype(grad, "grad")
    if grad.dim() < 2:
        raise ValueError("grad must be [..., rows, cols]")
    dev = grad.device
    _need(grad, "grad", grad.dtype, grad.shape, dev)
    m, n = grad.shape[-2:]
    if m < 1 or n < 1:
        raise ValueError(f"grad has shape {tuple(grad.shape)}: rows and cols must be at least 1")
    B = grad.numel() // (m * n)
    a, b, c = coeffs
    nbytes = _bytes("cgtp_orthogonalize_workspace_size", d, B, m, n)
    if out is None:
        out = torch.empty_like(grad)
    else:
        _need(out, "out", grad.dtype, grad.shape, dev)
    at, room, ws = _workspace(ws, nbytes, dev)  # (held until the call is out)
    _call("cgtp_orthogonalize", dev, d, B, m, n, steps, a, b, c, eps, scale, grad.data_ptr(), out.data_ptr(),
          at, room)
    return out
