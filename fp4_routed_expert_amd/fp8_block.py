"""FP8 operators with a scale for each block of 128 (C ABI in ``include/moe_fp8_block.h``).

Rows are quantised with one fp32 scale for 128 elements, weights with one for 128 x
128.  The scales of rows [M, K] are held block by block, [K/128, M].  From a
token's row to the gradients of an expert's weights:

    xq, xs = quant_fp8_block(x)
    hq, hs, gate, up = fp8_block_glu(w13, xq, xs, offsets, rows=pair, row_div=k, save=True)
    o = fp8_block_grouped(w2, hq, hs, offsets)
    dq, ds = quant_fp8_block(do)
    gq, gs = fp8_block_glu_backward(w2_t, dq, ds, gate, up, offsets)
    dx = fp8_block_grouped(w13_t, gq, gs, offsets)
    dw2 = fp8_block_weight_grad(dq, ds, hq, hs, offsets)
    dw13 = fp8_block_weight_grad(gq, gs, xq, xs, offsets, rows=pair, row_div=k)

with w13 = fp8_block_prepack_glu(w1, s1, w3, s3), w2 = fp8_block_prepack(w2, s2) and the
same bytes transposed, w2_t = fp8_block_prepack_t(w2, s2) and w13_t =
fp8_block_prepack_t(w1, s1, w3, s3).
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _lib
from .mx4 import _NORM_DTYPES, _TYPES, _U8, _call, _need, _workspace

_F32, _BF16, _I32 = (torch.float32,), (torch.bfloat16,), (torch.int32,)
# codes: bytes, or torch's type for them
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _new(t, shape, dtype, dev):
    return torch.empty(shape, dtype=dtype, device=dev) if t is None else t


# ------------------------------------------------------------- quantisation
def quant_fp8_block(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None):
    """x [M, K] bf16, fp16 or fp32 (rows may be strided) -> (q [M, K] e4m3 codes as uint8, s [K/128, M] fp32)."""
    if x.dtype not in _TYPES:
        raise TypeError(f"x: dtype {x.dtype} not in {tuple(_TYPES)}")
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x: two dimensions with neighbouring row elements required")
    if not x.is_cuda:
        raise ValueError("x: device tensor required")
    M, K = x.shape
    dev = x.device
    q, s = _new(q, (M, K), torch.uint8, dev), _new(s, (K // 128, M), torch.float32, dev)
    qp, sp = _need(q, "q", _CODES, (M, K), dev), _need(s, "s", _F32, (K // 128, M), dev)
    _call("moe_quant_fp8_block", dev, x.data_ptr(), _TYPES[x.dtype], M, K, x.stride(0) if M > 1 else K, qp, sp)
    return q, s


def dequant_fp8_block(q: torch.Tensor, s: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                      out: torch.Tensor | None = None):
    """The values of quantised rows (q [M, K], s [K/128, M]) -> [M, K] of ``dtype``."""
    if q.dim() != 2:
        raise ValueError(f"q: shape {tuple(q.shape)}, not [M, K]")
    M, K = q.shape
    dev = q.device
    out = _new(out, (M, K), dtype, dev)
    qp, sp = _need(q, "q", _CODES, (M, K), None), _need(s, "s", _F32, (K // 128, M), dev)
    op = _need(out, "out", _TYPES, (M, K), dev)
    _call("moe_dequant_fp8_block", dev, qp, sp, M, K, op, _TYPES[out.dtype])
    return out


# ------------------------------------------------------------------ weights
@dataclasses.dataclass
class Fp8BlockWeights:
    """Prepacked weights of the products: the device buffer plus the plain-C descriptor."""
    buffer: torch.Tensor
    desc: _lib.MoeFp8BlockWeights

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


def _prepack(wq, ws, uq, us, transposed) -> Fp8BlockWeights:
    if wq.dim() not in (2, 3):
        raise ValueError(f"wq: shape {tuple(wq.shape)}, not [N, K] or [E, N, K]")
    E, rows, cols = (wq.shape[0] if wq.dim() == 3 else 1), wq.shape[-2], wq.shape[-1]
    dev = wq.device
    sshape = wq.shape[:-2] + ((rows + 127) // 128, (cols + 127) // 128)
    ptr = [_need(wq, "wq", _CODES, wq.shape, None), _need(ws, "ws", _F32, sshape, dev), None, None]
    if uq is not None:
        ptr[2:] = [_need(uq, "uq", _CODES, wq.shape, dev), _need(us, "us", _F32, sshape, dev)]
    pair = uq is not None
    if transposed:
        if rows % 128:
            raise _lib.MoeError(_lib.MOE_ERR_UNSUPPORTED, "moe_fp8_block_prepack_t")
        N, K, glu, name = cols, rows * (2 if pair else 1), 0, "moe_fp8_block_prepack_t"
    else:
        N, K, glu, name = rows, cols, int(pair), "moe_fp8_block_prepack"
    nbytes = _lib.lib().moe_fp8_block_packed_bytes(E, N, K, glu)
    if nbytes == 0:
        raise _lib.MoeError(_lib.MOE_ERR_UNSUPPORTED, "moe_fp8_block_packed_bytes")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    desc = _lib.MoeFp8BlockWeights()
    _call(name, dev, *ptr, E, N, K, buf.data_ptr(), nbytes, ctypes.byref(desc))
    return Fp8BlockWeights(buffer=buf, desc=desc)


def fp8_block_prepack(wq: torch.Tensor, ws: torch.Tensor) -> Fp8BlockWeights:
    """Weights [N, K] or [E, N, K] as e4m3 codes and fp32 scales [.., N/128 rounded up, K/128]."""
    return _prepack(wq, ws, None, None, False)


def fp8_block_prepack_glu(wq, ws, uq, us) -> Fp8BlockWeights:
    """Gate (wq, ws) and up (uq, us) weights of one shape, for fp8_block_glu."""
    if uq is None or us is None:
        raise ValueError("uq, us: the up projection's weights required (fp8_block_prepack for plain ones)")
    return _prepack(wq, ws, uq, us, False)


def fp8_block_prepack_t(wq, ws, uq=None, us=None) -> Fp8BlockWeights:
    """The same weights transposed, for the backward pass: products with W^T [K, N] of wq [N, K], both multiples
    of 128.  With uq and us: rows of 2 N elements times [wq; uq], that is dg W1 + du W3 of rows [dg, du]."""
    if (uq is None) != (us is None):
        raise ValueError("uq, us: both or neither")
    return _prepack(wq, ws, uq, us, True)


def _form(w: Fp8BlockWeights, glu: bool, name: str):
    if w.glu != glu:
        raise ValueError(f"w: {name} takes " + ("gate and up weights (fp8_block_prepack_glu)" if glu else "plain weights"))


# ----------------------------------------------------------------- products
def fp8_block_dense(w: Fp8BlockWeights, xq: torch.Tensor, xs: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                    flags: int = 0, y: torch.Tensor | None = None):
    """y [T, N] (bf16 or fp32) = rows (xq [T, K], xs [K/128, T]) times weights."""
    _form(w, False, "fp8_block_dense")
    T, dev = xq.shape[0], xq.device
    y = _new(y, (T, w.N), dtype, dev)
    xp, sp = _need(xq, "xq", _CODES, (T, w.K), w.buffer.device), _need(xs, "xs", _F32, (w.K // 128, T), dev)
    yp = _need(y, "y", _NORM_DTYPES, (T, w.N), dev)
    _call("moe_fp8_block_dense_forward", dev, ctypes.byref(w.desc), xp, sp, T, yp, _TYPES[y.dtype], flags)
    return y


def fp8_block_grouped_workspace_size(P: int, E: int, N: int, K: int) -> int:
    return int(_lib.lib().moe_fp8_block_grouped_workspace_size(P, E, N, K))


def _groups(w_E, offsets, rows, dev):
    op = None if offsets is None else _need(offsets, "offsets", _I32, (w_E + 1,), dev)
    if rows is not None and rows.dim() != 1:
        raise ValueError(f"rows: shape {tuple(rows.shape)}, not [P]")
    rp = None if rows is None else _need(rows, "rows", _I32, rows.shape, dev)
    return op, rp


def fp8_block_grouped(w: Fp8BlockWeights, xq: torch.Tensor, xs: torch.Tensor, offsets: torch.Tensor,
                      rows: torch.Tensor | None = None, row_div: int = 1, dtype: torch.dtype = torch.bfloat16,
                      flags: int = 0, y: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """y [P, N]: row s of expert e (offsets[e] <= s < offsets[e+1]) is W[e] x[r], r = rows[s] // row_div,
    or s without ``rows``.  With sort_permute's sorted_pair and row_div = k, r is the pair's token.
    Rows outside [offsets[0], offsets[E]) are left as they were.  flags: MOE_FLAG_FORCE_PREFILL is faster
    where a few experts hold most of few rows."""
    _form(w, False, "fp8_block_grouped")
    X, dev = xq.shape[0], xq.device
    P = X if rows is None else rows.shape[0]
    y = _new(y, (P, w.N), dtype, dev)
    xp, sp = _need(xq, "xq", _CODES, (X, w.K), w.buffer.device), _need(xs, "xs", _F32, (w.K // 128, X), dev)
    op, rp = _groups(w.E, offsets, rows, dev)
    yp = _need(y, "y", _NORM_DTYPES, (P, w.N), dev)
    workspace = _workspace(workspace, lambda: fp8_block_grouped_workspace_size(P, w.E, w.N, w.K), dev)
    _call("moe_fp8_block_grouped_forward", dev, ctypes.byref(w.desc), xp, sp, X, op, rp, row_div, P, yp, _TYPES[y.dtype],
          workspace.data_ptr(), workspace.numel(), flags)
    return y


# ------------------------------------------------- gated feed-forward block
def fp8_block_glu_workspace_size(P: int, E: int, N: int, K: int, flags: int = 0) -> int:
    return int(_lib.lib().moe_fp8_block_glu_workspace_size(P, E, N, K, flags))


def fp8_block_glu(w: Fp8BlockWeights, xq: torch.Tensor, xs: torch.Tensor, offsets: torch.Tensor | None = None,
                  rows: torch.Tensor | None = None, row_div: int = 1, save: bool = False, flags: int = 0,
                  q: torch.Tensor | None = None, s: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                  up: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Quantised rows of h = silu(gate) * up, gate = x W1^T and up = x W3^T: (q [P, N], s [N/128, P], gate, up).
    gate and up [P, N] bf16 are kept for the backward pass with ``save`` or where given, else None.  Rows and
    groups as for fp8_block_grouped; without ``offsets`` (and ``rows``) one group.  A workspace for the largest P
    serves every smaller one, and the backward call."""
    _form(w, True, "fp8_block_glu")
    X, dev = xq.shape[0], xq.device
    P = X if rows is None else rows.shape[0]
    q, s = _new(q, (P, w.N), torch.uint8, dev), _new(s, (w.N // 128, P), torch.float32, dev)
    if save or gate is not None or up is not None:
        gate, up = _new(gate, (P, w.N), torch.bfloat16, dev), _new(up, (P, w.N), torch.bfloat16, dev)
    xp, sp = _need(xq, "xq", _CODES, (X, w.K), w.buffer.device), _need(xs, "xs", _F32, (w.K // 128, X), dev)
    op, rp = _groups(w.E, offsets, rows, dev)
    out = [_need(q, "q", _CODES, (P, w.N), dev), _need(s, "s", _F32, (w.N // 128, P), dev), None, None]
    if gate is not None:
        out[2:] = [_need(gate, "gate", _BF16, (P, w.N), dev), _need(up, "up", _BF16, (P, w.N), dev)]
    workspace = _workspace(workspace, lambda: fp8_block_glu_workspace_size(P, w.E, w.N, w.K, flags), dev)
    _call("moe_fp8_block_glu_forward", dev, ctypes.byref(w.desc), xp, sp, X, op, rp, row_div, P, *out,
          workspace.data_ptr(), workspace.numel(), flags)
    return q, s, gate, up


def fp8_block_glu_backward(w: Fp8BlockWeights, yq: torch.Tensor, ys: torch.Tensor, gate: torch.Tensor,
                           up: torch.Tensor, offsets: torch.Tensor | None = None, rows: torch.Tensor | None = None,
                           row_div: int = 1, flags: int = 0, q: torch.Tensor | None = None,
                           s: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Quantised rows [dg, du] (q [P, 2 N], s [2 N/128, P]) of the gradients of gate and up [P, N] bf16, from the
    rows dO (yq [X, K], ys [K/128, X]) of the down projection's output; w = fp8_block_prepack_t(w2, s2)."""
    _form(w, False, "fp8_block_glu_backward")
    X, dev = yq.shape[0], yq.device
    P = X if rows is None else rows.shape[0]
    q, s = _new(q, (P, 2 * w.N), torch.uint8, dev), _new(s, (2 * w.N // 128, P), torch.float32, dev)
    yp, sp = _need(yq, "yq", _CODES, (X, w.K), w.buffer.device), _need(ys, "ys", _F32, (w.K // 128, X), dev)
    op, rp = _groups(w.E, offsets, rows, dev)
    gp, up_ = _need(gate, "gate", _BF16, (P, w.N), dev), _need(up, "up", _BF16, (P, w.N), dev)
    out = _need(q, "q", _CODES, (P, 2 * w.N), dev), _need(s, "s", _F32, (2 * w.N // 128, P), dev)
    workspace = _workspace(workspace, lambda: fp8_block_glu_workspace_size(P, w.E, w.N, w.K, flags), dev)
    _call("moe_fp8_block_glu_backward", dev, ctypes.byref(w.desc), yp, sp, X, op, rp, row_div, P, gp, up_, *out,
          workspace.data_ptr(), workspace.numel(), flags)
    return q, s


def fp8_block_weight_grad_workspace_size(P: int, E: int, N: int, K: int) -> int:
    return int(_lib.lib().moe_fp8_block_weight_grad_workspace_size(P, E, N, K))


def fp8_block_weight_grad(yq: torch.Tensor, ys: torch.Tensor, xq: torch.Tensor, xs: torch.Tensor,
                          offsets: torch.Tensor | None = None, rows: torch.Tensor | None = None, row_div: int = 1,
                          dtype: torch.dtype = torch.bfloat16, dw: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None):
    """dw [E, N, K] (bf16 or fp32): the sum over group e's rows s of dy[s]^T x[r], r as for fp8_block_grouped, from
    quantised rows (yq [P, N], ys [N/128, P]; xq [X, K], xs [K/128, X]).  Without ``offsets`` (and ``rows``) one
    group, dw [N, K] or [1, N, K].  A group without rows gets zeros."""
    if yq.dim() != 2 or xq.dim() != 2:
        raise ValueError(f"yq, xq: shapes {tuple(yq.shape)}, {tuple(xq.shape)}, not [P, N] and [X, K]")
    (P, N), (X, K) = yq.shape, xq.shape
    dev = yq.device
    if offsets is not None and offsets.dim() != 1:
        raise ValueError(f"offsets: shape {tuple(offsets.shape)}, not [E+1]")
    E = 1 if offsets is None else offsets.shape[0] - 1
    shape = (N, K) if offsets is None and (dw is None or dw.dim() == 2) else (E, N, K)
    dw = _new(dw, shape, dtype, dev)
    yp, sp = _need(yq, "yq", _CODES, (P, N), None), _need(ys, "ys", _F32, (N // 128, P), dev)
    xp, xsp = _need(xq, "xq", _CODES, (X, K), dev), _need(xs, "xs", _F32, (K // 128, X), dev)
    op, rp = _groups(E, offsets, rows, dev)
    if (P if rows is None else rows.shape[0]) != P:
        raise ValueError(f"rows: {rows.shape[0]} of them, not one for each of the {P} rows of yq")
    wp = _need(dw, "dw", _NORM_DTYPES, shape, dev)
    workspace = _workspace(workspace, lambda: fp8_block_weight_grad_workspace_size(P, E, N, K), dev)
    _call("moe_fp8_block_weight_grad", dev, yp, sp, xp, xsp, X, op, rp, row_div, P, E, N, K, wp, _TYPES[dw.dtype],
          workspace.data_ptr(), workspace.numel())
    return dw
