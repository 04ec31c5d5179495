"""The MXFP4 operators' C ABI on the host: symbols, sizes and refusals (no
device: every call below returns before it would touch the GPU), the wrappers'
argument checks, and the reference that the GPU tests compare with."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import fp4_routed_expert_amd as moe
import mx4_ref as ref
from fp4_routed_expert_amd import _lib

L = None
A = ctypes.c_void_p(1 << 20)          # aligned stand-ins, never dereferenced on error paths
MIS = ctypes.c_void_p((1 << 20) + 2)
NUL = ctypes.c_void_p(0)
INV, UNS, WSE = _lib.MOE_ERR_INVALID_ARGUMENT, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
BF, FH, FS = _lib.MOE_TYPE_BF16, _lib.MOE_TYPE_FP16, _lib.MOE_TYPE_FP32
Q0, Q8, Q4 = _lib.MOE_QUANT_NONE, _lib.MOE_QUANT_MXFP8, _lib.MOE_QUANT_MXFP4


def setup_module():
    global L
    if not os.path.exists(_lib.SO_PATH):
        from fp4_routed_expert_amd import build
        build.build()
    L = _lib.lib()


def test_header_symbols():
    text = re.sub(r"/\*.*?\*/", "", open(_lib.MX4_HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 11
    so = ctypes.CDLL(_lib.SO_PATH)
    for n in names:
        assert hasattr(so, n) and n in _lib.SIGNATURES, n


def test_quant_refusals():
    f = L.moe_quant_mxfp4
    assert f(A, BF, -1, 32, 32, A, A, NUL) == INV
    assert f(A, 3, 4, 32, 32, A, A, NUL) == INV
    assert f(A, BF, 4, 0, 32, A, A, NUL) == INV
    assert f(A, BF, 4, 64, 32, A, A, NUL) == INV        # rows overlap
    assert f(A, BF, 4, 48, 48, A, A, NUL) == UNS
    assert f(A, BF, 4, 32, 36, A, A, NUL) == INV        # unaligned rows
    assert f(A, FS, 4, 32, 34, A, A, NUL) == INV
    assert f(MIS, BF, 4, 32, 32, A, A, NUL) == INV
    assert f(NUL, BF, 4, 32, 32, A, A, NUL) == INV
    assert f(A, BF, 4, 32, 32, MIS, A, NUL) == INV
    assert f(A, FS, (1 << 31) - 1, (1 << 31) - 32, (1 << 31) - 32, A, A, NUL) == UNS
    assert f(NUL, BF, 0, 32, 32, NUL, NUL, NUL) == 0


def test_dequant_refusals():
    f = L.moe_dequant_mx
    assert f(A, A, Q0, 4, 32, A, BF, NUL) == INV
    assert f(A, A, 7, 4, 32, A, BF, NUL) == INV
    assert f(A, A, Q4, 4, 32, A, 9, NUL) == INV
    assert f(A, A, Q4, 4, 40, A, BF, NUL) == UNS
    assert f(A, NUL, Q4, 4, 32, A, BF, NUL) == INV
    assert f(ctypes.c_void_p((1 << 20) + 4), A, Q8, 4, 32, A, BF, NUL) == INV
    assert f(A, A, Q4, 4, 32, MIS, BF, NUL) == INV
    assert f(NUL, NUL, Q4, 0, 32, NUL, BF, NUL) == 0


def test_weight_sizes_and_refusals():
    p = L.moe_mxfp4_packed_bytes
    assert p(0, 32, 128, 0) == 0 and p(1, 48, 128, 0) == 0 and p(1, 32, 96, 0) == 0 and p(1025, 32, 128, 0) == 0
    assert p(1, 32, 128, 2) == 0 and p(1, 2 << 20, 128, 0) == 0
    for E, N, K, g in ((1, 32, 128, 0), (3, 96, 384, 0), (8, 64, 256, 1), (256, 7168, 2048, 0)):
        codes, scales = E * N * K // 2 << g, E * N * K // 32 << g
        # (whole pairs of K-steps of 128; the scales for whole groups of four 32-row tiles)
        even = (K + 255) // 256 * 256 / K
        assert codes + scales <= p(E, N, K, g) <= (codes + 4 * scales) * even + 256
    d = _lib.MoeMxfp4Weights()
    f, D = L.moe_mxfp4_prepack, ctypes.byref(d)
    n = p(2, 64, 128, 0)
    assert f(A, A, NUL, NUL, 2, 64, 128, A, n - 1, D, NUL) == INV
    assert f(A, A, A, NUL, 2, 64, 128, A, 2 * n, D, NUL) == INV    # half a SwiGLU pair
    assert f(A, A, NUL, A, 2, 64, 128, A, 2 * n, D, NUL) == INV
    assert f(A, A, A, A, 2, 64, 128, A, n, D, NUL) == INV          # twice the bytes
    assert f(A, NUL, NUL, NUL, 2, 64, 128, A, n, D, NUL) == INV
    assert f(A, A, NUL, NUL, 2, 64, 128, ctypes.c_void_p((1 << 20) + 16), n, D, NUL) == INV
    assert f(MIS, A, NUL, NUL, 2, 64, 128, A, n, D, NUL) == INV
    assert f(A, A, NUL, NUL, 2, 64, 128, A, n, None, NUL) == INV
    assert f(A, A, NUL, NUL, 2, 40, 128, A, n, D, NUL) == UNS


def _desc(E=1, N=64, K=256, glu=0, version=_lib.MOE_MXFP4_LAYOUT_VERSION):
    d = _lib.MoeMxfp4Weights()
    d.E, d.N, d.K, d.glu, d.layout_version, d.packed = E, N, K, glu, version, 1 << 20
    d.packed_bytes = L.moe_mxfp4_packed_bytes(E, N, K, glu)
    return d


def test_dense_refusals():
    f, R = L.moe_mxfp4_dense_forward, ctypes.byref
    d = _desc()
    assert f(None, A, A, 4, A, BF, 0, NUL) == INV
    assert f(R(_desc(version=9)), A, A, 4, A, BF, 0, NUL) == INV
    assert f(R(_desc(E=2)), A, A, 4, A, BF, 0, NUL) == INV
    bad = _desc()
    bad.packed_bytes -= 1
    assert f(R(bad), A, A, 4, A, BF, 0, NUL) == INV
    assert f(R(d), A, A, -1, A, BF, 0, NUL) == INV
    assert f(R(d), A, A, 4, A, FH, 0, NUL) == INV
    assert f(R(d), A, A, 4, A, BF, 3, NUL) == INV
    assert f(R(d), A, A, 4, A, BF, 8, NUL) == INV
    assert f(R(d), A, A, 1 << 25, A, BF, 0, NUL) == UNS            # T K / 2 = 2^32
    assert f(R(d), MIS, A, 4, A, BF, 0, NUL) == INV
    assert f(R(d), A, MIS, 4, A, BF, 0, NUL) == INV
    assert f(R(d), A, A, 4, NUL, BF, 0, NUL) == INV
    assert f(R(d), NUL, NUL, 0, NUL, BF, 0, NUL) == 0


def test_grouped_refusals():
    f, R = L.moe_mxfp4_grouped_forward, ctypes.byref
    size = L.moe_mxfp4_grouped_workspace_size
    assert size(-1, 4, 64, 256, 0) == 0 and size(4, 0, 64, 256, 0) == 0 and size(4, 4, 63, 256, 0) == 0
    d, ws = _desc(E=4), size(1000, 4, 64, 256, 0)
    # the list of row tiles: one for each 64 rows and each group, never fewer than the groups can have
    assert ws >= 16 + 16 * (1000 // 64 + 4)
    ok = (1000, A, A, 2, 1000, A, BF, A, ws, 0)

    def call(desc=d, X=1000, off=A, rows=A, div=2, P=1000, y=A, yt=BF, w=A, nb=ws, fl=0, xq=A, xs=A):
        return f(R(desc), xq, xs, X, off, rows, div, P, y, yt, w, nb, fl, NUL)

    assert len(ok) == 10
    assert call(div=0) == INV
    assert call(P=-1) == INV
    assert call(X=-1) == INV
    assert call(X=0) == INV
    assert call(X=999, rows=NUL) == INV       # fewer rows than y has
    assert call(off=NUL) == INV
    assert call(y=NUL) == INV
    assert call(yt=FH) == INV
    assert call(fl=3) == INV
    assert call(nb=ws - 1) == WSE
    assert call(w=NUL) == WSE
    assert call(w=ctypes.c_void_p((1 << 20) + 16)) == INV
    assert call(X=1 << 25) == UNS
    assert call(P=(1 << 31) - 1) == UNS and size((1 << 31) - 1, 4, 64, 256, 0) == 0   # tile ends past 32 bits
    assert call(P=0, y=NUL, off=NUL, w=NUL, nb=0) == 0


def test_norm_refusals():
    f = L.moe_norm_before

    def before(x=A, xt=BF, w=A, wt=FS, T=4, H=64, eps=1e-6, z=A, q=NUL, s=NUL, quant=Q0):
        return f(x, xt, w, wt, T, H, eps, z, q, s, quant, NUL)

    assert before(T=-1) == INV and before(H=0) == INV and before(eps=-1.0) == INV and before(eps=float("nan")) == INV
    assert before(xt=FH) == INV and before(wt=FH) == INV and before(quant=5) == INV
    assert before(H=60) == UNS and before(H=16392) == UNS and before(H=40, q=A, s=A, quant=Q4) == UNS
    assert before(z=NUL) == INV                       # nothing wanted
    assert before(q=A) == INV                         # codes without a format
    assert before(q=A, quant=Q8) == INV and before(s=A, quant=Q8) == INV
    assert before(w=NUL) == INV and before(x=MIS) == INV and before(z=MIS) == INV
    assert before(T=0, x=NUL, w=NUL, z=NUL) == 0
    g = L.moe_norm_after

    def after(y=A, yt=FS, res=A, rt=BF, wp=A, wn=NUL, wt=FS, gate=NUL, gt=0, gh=0, eps=1e-6, T=4, H=64, out=A, z=NUL,
              q=NUL, s=NUL, quant=Q0):
        return g(y, yt, res, rt, wp, wn, wt, gate, gt, gh, 1.0, 1.0, eps, T, H, out, z, q, s, quant, NUL)

    assert after(res=NUL) == INV and after(out=NUL) == INV and after(y=NUL) == INV and after(yt=FH) == INV
    assert after(z=A) == INV and after(q=A, s=A, quant=Q8) == INV      # no norm that follows
    assert after(wn=A) == INV                                           # a norm that writes nothing
    assert after(gate=A, gh=2) == INV and after(gate=A, gt=-1) == INV
    assert after(gate=MIS, gt=1) == INV
    assert after(H=48 * 1024) == UNS and after(H=20) == UNS and after(rt=FH) == INV
    assert after(T=0, y=NUL, res=NUL, out=NUL) == 0


def test_block_refusals():
    w = _lib.MoeFp4Weights()
    w.E, w.H, w.I, w.layout_version, w.packed = 8, 256, 128, 1, 1 << 20
    w.packed_bytes = L.moe_fp4_packed_weight_bytes(8, 256, 128)
    n = _lib.MoeBlockNorms(1 << 20, None, FS, None, 0, 0, 1.0, 1.0, 1e-6)
    size, f, R = L.moe_fp4_block_workspace_size, L.moe_fp4_block_forward, ctypes.byref
    assert size(16, 8, 9, 256, 128, 0, 0) == 0
    ws = size(16, 8, 2, 256, 128, 1, 0)
    assert ws >= L.moe_fp4_layer_full_workspace_size(16, 8, 2, 256, 128, 1, 0) + 16 * 256 * 6

    def call(w_=w, norms=n, ns=1, rw=A, x=A, xt=BF, T=16, k=2, out=A, mem=A, nb=ws, fl=0):
        return f(R(w_), ns, rw, None if norms is None else R(norms), x, xt, T, k, out, mem, nb, fl, NUL)

    assert call(norms=None) == INV and call(rw=NUL) == INV and call(x=NUL) == INV and call(out=NUL) == INV
    assert call(xt=FH) == INV and call(nb=ws - 1) == WSE and call(mem=NUL) == WSE and call(ns=8) == INV
    assert call(k=8) == UNS and call(fl=3) == INV and call(T=-1) == INV
    assert call(norms=_lib.MoeBlockNorms(None, None, FS, None, 0, 0, 1.0, 1.0, 1e-6)) == INV
    assert call(norms=_lib.MoeBlockNorms(1 << 20, None, FH, None, 0, 0, 1.0, 1.0, 1e-6)) == INV
    assert call(T=0, x=NUL, out=NUL, mem=NUL, nb=0) == 0


def test_wrappers_refuse_host_tensors_and_wrong_shapes():
    u8 = torch.zeros
    with pytest.raises(ValueError):
        moe.quant_mxfp4(torch.zeros(4, 64))
    with pytest.raises(TypeError):
        moe.quant_mxfp4(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        moe.dequant_mx(u8(4, 32, dtype=torch.uint8), u8(4, 2, dtype=torch.uint8), "int4")
    with pytest.raises(ValueError):
        moe.dequant_mx(u8(4, 32, dtype=torch.uint8), u8(4, 2, dtype=torch.uint8), "mxfp4")
    with pytest.raises(ValueError):
        moe.mxfp4_prepack(u8(4, dtype=torch.uint8), u8(4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.norm_before(torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64))
    with pytest.raises(TypeError):
        moe.norm_before(torch.zeros(4, 64, dtype=torch.float16), torch.ones(64))


def test_reference_codecs():
    """The reference's rounding against exhaustive neighbours, its bf16 against torch's."""
    for fmt, table in (("mxfp4", ref.E2M1), ("mxfp8", ref.E4M3)):
        top = table[-1]
        v = np.concatenate([np.linspace(-top, top, 4001), table, -table, (table[1:] + table[:-1]) / 2])
        v = v[: len(v) // 31 * 31].reshape(-1, 31)
        v = np.concatenate([v, np.full((len(v), 1), top)], 1)       # the last element fixes the scale at 2^0
        q, s = ref.quant(v, fmt)
        assert (s == 127).all()
        got = ref.values(q, s, fmt)
        gaps = np.abs(v[..., None] - np.concatenate([-table, table]))
        assert np.array_equal(np.abs(v - got), gaps.min(-1))
    r = np.random.default_rng(1).standard_normal(4000) * np.exp2(np.arange(4000) % 260 - 135)
    want = torch.from_numpy(r.astype(np.float32)).bfloat16().float().numpy()
    assert np.array_equal(ref.bf16(r.astype(np.float32)), want)
    q, s = ref.quant(np.array([[0.0] * 32, [np.nan] + [1.0] * 31, [-np.inf] + [1.0] * 31, [2.0 ** -140] * 32]), "mxfp4")
    assert s[:, 0].tolist() == [0, 255, 255, 0] and not q[:3].any() and np.isnan(ref.values(q, s)[1]).all()
