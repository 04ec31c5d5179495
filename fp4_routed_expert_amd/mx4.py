"""The operators around the FP4 layer (C ABI in ``include/moe_mx4.h``).

MXFP4 quantisation and the reading back of microscaled rows, products of MXFP4
rows with MXFP4 weights (dense, and grouped by expert), the norms before and
after a block, and the layer between its norms.  As in the rest of the
package, every function marshals torch tensors and the current stream of their
device into one call of the library; outputs and workspaces may be given to
keep allocation out of the call.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _lib

_TYPES = {torch.bfloat16: _lib.MOE_TYPE_BF16, torch.float16: _lib.MOE_TYPE_FP16, torch.float32: _lib.MOE_TYPE_FP32}
_QUANT = {None: _lib.MOE_QUANT_NONE, "mxfp8": _lib.MOE_QUANT_MXFP8, "mxfp4": _lib.MOE_QUANT_MXFP4}
_NORM_DTYPES = (torch.bfloat16, torch.float32)
_U8 = (torch.uint8,)


def _need(t: torch.Tensor, name: str, dtypes, shape, dev=None):
    """Type, shape and device of a contiguous argument; its address."""
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and (t.is_cuda if dev is None else t.device == dev):
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor required")
    raise ValueError(f"{name}: on {t.device}, not on {dev if dev is not None else 'a GPU'}")


# The current device and its stream's handle without the objects around them, where torch has these.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(name: str, dev: torch.device, *args):
    """One library call on dev's current stream, dev being the current device meanwhile."""
    fn = getattr(_lib.lib(), name)
    i = dev.index
    if i == _device():
        status = fn(*args, _stream(i))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(i))
    if status:
        _lib.check(status, name)


def _workspace(ws, need, dev):
    """The given workspace, or a new one of need() bytes."""
    if ws is None:
        return torch.empty(max(need(), 256), dtype=torch.uint8, device=dev)
    if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != dev:
        raise ValueError("workspace: contiguous uint8 tensor on the inputs' device required")
    return ws


# ------------------------------------------------------------- quantisation
def quant_mxfp4(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None):
    """x [M, K] bf16, fp16 or fp32 (rows may be strided) -> (q [M, K/2] e2m1 codes, s [M, K/32] E8M0
    codes), both uint8."""
    if x.dtype not in _TYPES:
        raise TypeError(f"x: dtype {x.dtype} not in {tuple(_TYPES)}")
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x: two dimensions with neighbouring row elements required")
    M, K = x.shape
    dev = x.device
    if not x.is_cuda:
        raise ValueError("x: device tensor required")
    if q is None:
        q = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    if s is None:
        s = torch.empty((M, K // 32), dtype=torch.uint8, device=dev)
    qp, sp = _need(q, "q", _U8, (M, K // 2), dev), _need(s, "s", _U8, (M, K // 32), dev)
    _call("moe_quant_mxfp4", dev, x.data_ptr(), _TYPES[x.dtype], M, K, x.stride(0) if M > 1 else K, qp, sp)
    return q, s


def dequant_mx(q: torch.Tensor, s: torch.Tensor, format: str, dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None):
    """The values of microscaled rows: format "mxfp4" (q [M, K/2]) or "mxfp8" (q [M, K]), s [M, K/32]
    -> [M, K] of ``dtype``."""
    if format not in ("mxfp4", "mxfp8"):
        raise ValueError(f"format {format!r}")
    if s.dim() != 2:
        raise ValueError(f"s: shape {tuple(s.shape)}, not [M, K/32]")
    M, K = s.shape[0], s.shape[1] * 32
    dev = q.device
    if out is None:
        out = torch.empty((M, K), dtype=dtype, device=dev)
    qp = _need(q, "q", _U8, (M, K // 2 if format == "mxfp4" else K), None)
    sp, op = _need(s, "s", _U8, (M, K // 32), dev), _need(out, "out", _TYPES, (M, K), dev)
    _call("moe_dequant_mx", dev, qp, sp, _QUANT[format], M, K, op, _TYPES[out.dtype])
    return out


# ----------------------------------------------------------------- products
@dataclasses.dataclass
class Mxfp4Weights:
    """Prepacked weights of the MXFP4 products: the device buffer plus the plain-C descriptor."""
    buffer: torch.Tensor
    desc: _lib.MoeMxfp4Weights

    @property
    def E(self):
        return self.desc.E

    @property
    def N(self):
        return self.desc.N

    @property
    def K(self):
        return self.desc.K

    @property
    def glu(self):
        return bool(self.desc.glu)


def _prepack(wq, ws, uq, us) -> Mxfp4Weights:
    if wq.dim() not in (2, 3):
        raise ValueError(f"wq: shape {tuple(wq.shape)}, not [N, K/2] or [E, N, K/2]")
    E, N, K = (wq.shape[0] if wq.dim() == 3 else 1), wq.shape[-2], wq.shape[-1] * 2
    dev = wq.device
    sshape = wq.shape[:-1] + (K // 32,)
    ptr = [_need(wq, "wq", _U8, wq.shape, None), _need(ws, "ws", _U8, sshape, dev), None, None]
    if uq is not None:
        ptr[2:] = [_need(uq, "uq", _U8, wq.shape, dev), _need(us, "us", _U8, sshape, dev)]
    nbytes = _lib.lib().moe_mxfp4_packed_bytes(E, N, K, int(uq is not None))
    if nbytes == 0:
        raise _lib.MoeError(_lib.MOE_ERR_UNSUPPORTED, "moe_mxfp4_packed_bytes")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    desc = _lib.MoeMxfp4Weights()
    _call("moe_mxfp4_prepack", dev, *ptr, E, N, K, buf.data_ptr(), nbytes, ctypes.byref(desc))
    return Mxfp4Weights(buffer=buf, desc=desc)


def mxfp4_prepack(wq: torch.Tensor, ws: torch.Tensor) -> Mxfp4Weights:
    """Weights [N, K] or [E, N, K] as e2m1 codes [.., N, K/2] and E8M0 scales [.., N, K/32] (uint8),
    as quant_mxfp4 makes them."""
    return _prepack(wq, ws, None, None)


def mxfp4_prepack_glu(wq, ws, uq, us) -> Mxfp4Weights:
    """Gate (wq, ws) and up (uq, us) weights of one shape: the products return silu(gate) * up."""
    if uq is None or us is None:
        raise ValueError("uq, us: the up projection's weights required (mxfp4_prepack for plain ones)")
    return _prepack(wq, ws, uq, us)


def mxfp4_dense(w: Mxfp4Weights, xq: torch.Tensor, xs: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                flags: int = 0, y: torch.Tensor | None = None):
    """y [T, N] (bf16 or fp32) = MXFP4 rows (xq [T, K/2], xs [T, K/32]) times MXFP4 weights."""
    T, dev = xq.shape[0], xq.device
    if y is None:
        y = torch.empty((T, w.N), dtype=dtype, device=dev)
    xp, sp = _need(xq, "xq", _U8, (T, w.K // 2), w.buffer.device), _need(xs, "xs", _U8, (T, w.K // 32), dev)
    yp = _need(y, "y", _NORM_DTYPES, (T, w.N), dev)
    _call("moe_mxfp4_dense_forward", dev, ctypes.byref(w.desc), xp, sp, T, yp, _TYPES[y.dtype], flags)
    return y


def mxfp4_grouped_workspace_size(P: int, E: int, N: int, K: int, glu: bool = False) -> int:
    return int(_lib.lib().moe_mxfp4_grouped_workspace_size(P, E, N, K, int(glu)))


def mxfp4_grouped(w: Mxfp4Weights, xq: torch.Tensor, xs: torch.Tensor, offsets: torch.Tensor,
                  rows: torch.Tensor | None = None, row_div: int = 1, dtype: torch.dtype = torch.bfloat16,
                  flags: int = 0, y: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """y [P, N]: row s of expert e (offsets[e] <= s < offsets[e+1]) is W[e] x[r], r = rows[s] // row_div,
    or s without ``rows``.  With sort_permute's sorted_pair and row_div = k, r is the pair's token.
    Rows outside [offsets[0], offsets[E]) are left as they were.  flags: MOE_FLAG_FORCE_PREFILL is faster
    where a few experts hold most of few rows."""
    X, dev = xq.shape[0], xq.device
    P = X if rows is None else rows.shape[0]
    if y is None:
        y = torch.empty((P, w.N), dtype=dtype, device=dev)
    xp, sp = _need(xq, "xq", _U8, (X, w.K // 2), w.buffer.device), _need(xs, "xs", _U8, (X, w.K // 32), dev)
    op = _need(offsets, "offsets", (torch.int32,), (w.E + 1,), dev)
    rp = None if rows is None else _need(rows, "rows", (torch.int32,), (P,), dev)
    yp = _need(y, "y", _NORM_DTYPES, (P, w.N), dev)
    workspace = _workspace(workspace, lambda: mxfp4_grouped_workspace_size(P, w.E, w.N, w.K, w.glu), dev)
    _call("moe_mxfp4_grouped_forward", dev, ctypes.byref(w.desc), xp, sp, X, op, rp, row_div, P, yp, _TYPES[y.dtype],
          workspace.data_ptr(), workspace.numel(), flags)
    return y


# -------------------------------------------------------------------- norms
def _norm_outputs(T, H, dev, quant, z, q, s, want_z):
    if quant not in _QUANT:
        raise ValueError(f"quant {quant!r}")
    if z is None and want_z:
        z = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    ptr = [None if z is None else _need(z, "z", (torch.bfloat16,), (T, H), dev), None, None]
    if quant is None:
        if q is not None or s is not None:
            raise ValueError("q and s need quant")
    else:
        width = H // 2 if quant == "mxfp4" else H
        if q is None:
            q = torch.empty((T, width), dtype=torch.uint8, device=dev)
        if s is None:
            s = torch.empty((T, H // 32), dtype=torch.uint8, device=dev)
        ptr[1:] = [_need(q, "q", _U8, (T, width), dev), _need(s, "s", _U8, (T, H // 32), dev)]
    return z, q, s, ptr


def norm_before(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, quant: str | None = None,
                want_z: bool = True, z=None, q=None, s=None):
    """RMS norm of x [T, H] (bf16 or fp32) times weight [H]: (z [T, H] bf16, q, s), q and s the
    "mxfp8" or "mxfp4" rows of z where ``quant`` asks for them, else None."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, not [T, H]")
    T, H = x.shape
    dev = x.device
    xp = _need(x, "x", _NORM_DTYPES, (T, H), None)
    wp = _need(weight, "weight", _NORM_DTYPES, (H,), dev)
    z, q, s, out = _norm_outputs(T, H, dev, quant, z, q, s, want_z)
    _call("moe_norm_before", dev, xp, _TYPES[x.dtype], wp, _TYPES[weight.dtype], T, H, eps, *out, _QUANT[quant])
    return z, q, s


def _gate(gate, T, H, dev):
    """(address, gate_t, gate_h) of a gate [T, 1], [H], [1, H] or [T, H]."""
    if gate is None:
        return None, 0, 0
    if gate.dtype != torch.float32 or gate.device != dev:
        raise TypeError("gate: fp32 tensor on the inputs' device required")
    shape = (1,) * (2 - gate.dim()) + tuple(gate.shape)
    if len(shape) != 2 or shape[0] not in (1, T) or shape[1] not in (1, H):
        raise ValueError(f"gate: shape {tuple(gate.shape)} does not broadcast to {(T, H)}")
    stride = (0,) * (2 - gate.dim()) + gate.stride()
    gate_t, gate_h = (stride[i] if shape[i] > 1 else 0 for i in range(2))
    if gate_h not in (0, 1):
        raise ValueError("gate: neighbouring row elements required")
    return gate.data_ptr(), gate_t, gate_h


def _pair_weights(a, b, H, dev):
    """Addresses of two optional weights and their common type."""
    ptr = [None if w is None else _need(w, "weight", _NORM_DTYPES, (H,), dev) for w in (a, b)]
    if a is not None and b is not None and a.dtype != b.dtype:
        raise TypeError(f"the two norm weights have different types: {a.dtype}, {b.dtype}")
    one = a if a is not None else b
    return ptr, _lib.MOE_TYPE_FP32 if one is None else _TYPES[one.dtype]


def norm_after(y: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None = None, gate=None,
               alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6, next_weight: torch.Tensor | None = None,
               quant: str | None = None, want_z: bool = True, out=None, z=None, q=None, s=None):
    """beta residual + alpha gate branch, the branch being y [T, H] or its RMS norm times ``weight``:
    (out, z, q, s), out of residual's type (``out=residual`` for in place).  With ``next_weight`` z, q
    and s are norm_before(out, next_weight); otherwise None.  gate: fp32, one for each token ([T, 1]),
    each channel ([H]) or both ([T, H])."""
    if y.dim() != 2:
        raise ValueError(f"y: shape {tuple(y.shape)}, not [T, H]")
    T, H = y.shape
    dev = y.device
    yp, rp = _need(y, "y", _NORM_DTYPES, (T, H), None), _need(residual, "residual", _NORM_DTYPES, (T, H), dev)
    if out is None:
        out = torch.empty_like(residual)
    op = _need(out, "out", (residual.dtype,), (T, H), dev)
    (wp, np_), w_type = _pair_weights(weight, next_weight, H, dev)
    gp, gate_t, gate_h = _gate(gate, T, H, dev)
    if next_weight is None and (quant is not None or z is not None):
        raise ValueError("z and quant need next_weight")
    z, q, s, ptr = _norm_outputs(T, H, dev, quant, z, q, s, want_z and next_weight is not None)
    _call("moe_norm_after", dev, yp, _TYPES[y.dtype], rp, _TYPES[residual.dtype], wp, np_, w_type, gp, gate_t, gate_h,
          alpha, beta, eps, T, H, op, *ptr, _QUANT[quant])
    return out, z, q, s


# -------------------------------------------------- the layer between its norms
def block_workspace_size(T: int, E: int, k: int, H: int, I: int, n_shared: int = 0, flags: int = 0) -> int:
    return int(_lib.lib().moe_fp4_block_workspace_size(T, E, k, H, I, n_shared, flags))


def block_forward(pw, n_shared: int, router_w: torch.Tensor, x: torch.Tensor, k: int, pre_weight: torch.Tensor,
                  post_weight: torch.Tensor | None = None, gate=None, alpha: float = 1.0, beta: float = 1.0,
                  eps: float = 1e-6, flags: int = 0, out=None, workspace=None):
    """norm_before -> layer_forward_full -> norm_after in one call: x [T, H] (bf16 or fp32) is the
    residual stream, the result the stream behind the block (``out=x`` for in place)."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, not [T, H]")
    T, H = x.shape
    dev = x.device
    xp = _need(x, "x", _NORM_DTYPES, (T, pw.H), pw.buffer.device)
    wp = _need(router_w, "router_w", (torch.bfloat16, torch.int16, torch.uint16), (pw.E - n_shared, pw.H), dev)
    if out is None:
        out = torch.empty_like(x)
    op = _need(out, "out", (x.dtype,), (T, H), dev)
    (pre, post), w_type = _pair_weights(pre_weight, post_weight, H, dev)
    gp, gate_t, gate_h = _gate(gate, T, H, dev)
    norms = _lib.MoeBlockNorms(pre, post, w_type, gp, gate_t, gate_h, alpha, beta, eps)
    workspace = _workspace(workspace, lambda: block_workspace_size(T, pw.E, k, H, pw.I, n_shared, flags), dev)
    _call("moe_fp4_block_forward", dev, ctypes.byref(pw.desc), n_shared, wp, ctypes.byref(norms), xp, _TYPES[x.dtype], T,
          k, op, workspace.data_ptr(), workspace.numel(), flags)
    return out
