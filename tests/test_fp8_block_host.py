"""The FP8 block-scale operators' C ABI on the host: symbols, sizes and refusals (no device: every call below returns
before it would touch the GPU), the wrappers' argument checks, and the reference that the GPU tests compare with."""
import ctypes
import os
import re

import pytest
import torch

import fp4_routed_expert_amd as moe
import fp8b_ref as ref
from fp4_routed_expert_amd import _lib

L = None
A = ctypes.c_void_p(1 << 20)          # aligned stand-ins, never dereferenced on error paths
MIS = ctypes.c_void_p((1 << 20) + 2)
NUL = ctypes.c_void_p(0)
INV, UNS, WSE = _lib.MOE_ERR_INVALID_ARGUMENT, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
BF, FH, FS = _lib.MOE_TYPE_BF16, _lib.MOE_TYPE_FP16, _lib.MOE_TYPE_FP32
R = ctypes.byref


def setup_module():
    global L
    if not os.path.exists(_lib.SO_PATH):
        from fp4_routed_expert_amd import build
        build.build()
    L = _lib.lib()


def test_header_symbols():
    text = re.sub(r"/\*.*?\*/", "", open(_lib.FP8_BLOCK_HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 13
    so = ctypes.CDLL(_lib.SO_PATH)
    for n in names:
        assert hasattr(so, n) and n in _lib.SIGNATURES, n


def test_quant_refusals():
    f = L.moe_quant_fp8_block
    assert f(A, BF, -1, 128, 128, A, A, NUL) == INV
    assert f(A, 3, 4, 128, 128, A, A, NUL) == INV
    assert f(A, BF, 4, 0, 128, A, A, NUL) == INV
    assert f(A, BF, 4, 256, 128, A, A, NUL) == INV       # rows overlap
    assert f(A, BF, 4, 192, 192, A, A, NUL) == UNS
    assert f(A, BF, 4, 128, 132, A, A, NUL) == INV       # unaligned rows
    assert f(A, FS, 4, 128, 130, A, A, NUL) == INV
    assert f(MIS, BF, 4, 128, 128, A, A, NUL) == INV
    assert f(NUL, BF, 4, 128, 128, A, A, NUL) == INV
    assert f(A, BF, 4, 128, 128, MIS, A, NUL) == INV
    assert f(A, BF, 4, 128, 128, A, MIS, NUL) == INV
    assert f(A, BF, (1 << 31) - 1, 128, 128, A, A, NUL) == UNS
    assert f(A, BF, 4, 1 << 21, 1 << 21, A, A, NUL) == UNS
    assert f(NUL, BF, 0, 128, 128, NUL, NUL, NUL) == 0


def test_dequant_refusals():
    f = L.moe_dequant_fp8_block
    assert f(A, A, 4, 128, A, 9, NUL) == INV
    assert f(A, A, 4, 130, A, BF, NUL) == UNS
    assert f(A, NUL, 4, 128, A, BF, NUL) == INV
    assert f(MIS, A, 4, 128, A, BF, NUL) == INV
    assert f(A, A, 4, 128, ctypes.c_void_p((1 << 20) + 8), BF, NUL) == INV
    assert f(NUL, NUL, 0, 128, NUL, BF, NUL) == 0


def test_weight_sizes_and_refusals():
    p = L.moe_fp8_block_packed_bytes
    assert p(0, 32, 128, 0) == 0 and p(1, 48, 128, 0) == 0 and p(1, 32, 96, 0) == 0 and p(1025, 32, 128, 0) == 0
    assert p(1, 32, 128, 2) == 0 and p(1, 2 << 20, 128, 0) == 0 and p(1024, 1 << 20, 1 << 20, 0) == 0
    for E, N, K, g in ((1, 32, 128, 0), (3, 96, 384, 0), (8, 64, 256, 1), (256, 7168, 2048, 0)):
        codes, scales = E * N * K << g, E * ((N + 127) // 128) * (K // 128) * 4 << g
        assert codes + scales <= p(E, N, K, g) <= codes + scales + 256
    d = _lib.MoeFp8BlockWeights()
    D = R(d)
    n = p(2, 128, 256, 0)
    for f in (L.moe_fp8_block_prepack, L.moe_fp8_block_prepack_t):
        assert f(A, A, NUL, NUL, 2, 128, 256, A, n - 1, D, NUL) == INV
        assert f(A, A, A, NUL, 2, 128, 256, A, 2 * n, D, NUL) == INV    # half a pair
        assert f(A, A, NUL, A, 2, 128, 256, A, 2 * n, D, NUL) == INV
        assert f(A, NUL, NUL, NUL, 2, 128, 256, A, n, D, NUL) == INV
        assert f(A, MIS, NUL, NUL, 2, 128, 256, A, n, D, NUL) == INV
        assert f(MIS, A, NUL, NUL, 2, 128, 256, A, n, D, NUL) == INV
        assert f(A, A, NUL, NUL, 2, 128, 256, ctypes.c_void_p((1 << 20) + 16), n, D, NUL) == INV
        assert f(A, A, NUL, NUL, 2, 128, 256, A, n, None, NUL) == INV
        assert f(A, A, NUL, NUL, 2, 40, 256, A, n, D, NUL) == UNS
    assert L.moe_fp8_block_prepack(A, A, A, A, 2, 128, 256, A, n, D, NUL) == INV   # twice the bytes
    assert L.moe_fp8_block_prepack_t(A, A, NUL, NUL, 2, 96, 256, A, n, D, NUL) == UNS
    assert L.moe_fp8_block_prepack_t(A, A, A, A, 2, 128, 384, A, 2 * n, D, NUL) == UNS


def _desc(E=1, N=256, K=256, glu=0, version=_lib.MOE_FP8_BLOCK_LAYOUT_VERSION):
    d = _lib.MoeFp8BlockWeights()
    d.E, d.N, d.K, d.glu, d.layout_version, d.packed = E, N, K, glu, version, 1 << 20
    d.packed_bytes = L.moe_fp8_block_packed_bytes(E, N, K, glu)
    return d


def test_dense_refusals():
    f = L.moe_fp8_block_dense_forward
    d = _desc()
    assert f(None, A, A, 4, A, BF, 0, NUL) == INV
    assert f(R(_desc(version=9)), A, A, 4, A, BF, 0, NUL) == INV
    assert f(R(_desc(E=2)), A, A, 4, A, BF, 0, NUL) == INV
    assert f(R(_desc(glu=1)), A, A, 4, A, BF, 0, NUL) == INV
    bad = _desc()
    bad.packed_bytes -= 1
    assert f(R(bad), A, A, 4, A, BF, 0, NUL) == INV
    assert f(R(d), A, A, -1, A, BF, 0, NUL) == INV
    assert f(R(d), A, A, 4, A, FH, 0, NUL) == INV
    assert f(R(d), A, A, 4, A, BF, 3, NUL) == INV
    assert f(R(d), A, A, 4, A, BF, 8, NUL) == INV
    assert f(R(d), A, A, 1 << 24, A, BF, 0, NUL) == UNS            # T K = 2^32
    assert f(R(d), MIS, A, 4, A, BF, 0, NUL) == INV
    assert f(R(d), A, MIS, 4, A, BF, 0, NUL) == INV
    assert f(R(d), A, A, 4, NUL, BF, 0, NUL) == INV
    assert f(R(d), NUL, NUL, 0, NUL, BF, 0, NUL) == 0


def test_grouped_refusals():
    f, size = L.moe_fp8_block_grouped_forward, L.moe_fp8_block_grouped_workspace_size
    assert size(-1, 4, 64, 256) == 0 and size(4, 0, 64, 256) == 0 and size(4, 4, 63, 256) == 0
    d, ws = _desc(E=4), size(1000, 4, 256, 256)
    # the list of row tiles: one for each 64 rows and each group, never fewer than the groups can have
    assert ws >= 16 + 16 * (1000 // 64 + 4) + 4 * 1000

    def call(desc=d, X=1000, off=A, rows=A, div=2, P=1000, y=A, yt=BF, w=A, nb=ws, fl=0, xq=A, xs=A):
        return f(R(desc), xq, xs, X, off, rows, div, P, y, yt, w, nb, fl, NUL)

    assert call(div=0) == INV and call(P=-1) == INV and call(X=-1) == INV and call(X=0) == INV
    assert call(X=999, rows=NUL) == INV       # fewer rows than y has
    assert call(off=NUL) == INV and call(off=NUL, rows=NUL, desc=_desc()) == INV
    assert call(off=MIS) == INV and call(rows=MIS) == INV
    assert call(y=NUL) == INV and call(yt=FH) == INV and call(fl=3) == INV
    assert call(desc=_desc(E=4, glu=1)) == INV
    assert call(nb=ws - 1) == WSE and call(w=NUL) == WSE
    assert call(w=ctypes.c_void_p((1 << 20) + 16)) == INV
    assert call(X=1 << 24) == UNS
    assert call(P=(1 << 31) - 1) == UNS and size((1 << 31) - 1, 4, 64, 256) == 0   # tile ends past 32 bits
    assert call(P=0, y=NUL, off=NUL, w=NUL, nb=0) == 0


@pytest.mark.parametrize("back", [False, True])
def test_glu_refusals(back):
    size = L.moe_fp8_block_glu_workspace_size
    assert size(-1, 4, 128, 256, 0) == 0 and size(4, 4, 128, 256, 3) == 0
    d, ws = _desc(E=4, glu=int(not back)), size(1000, 4, 256, 256, 0)

    def call(desc=d, X=1000, off=A, rows=A, div=2, P=1000, q=A, s=A, gate=A, up=A, w=A, nb=ws, fl=0, xq=A, xs=A):
        if back:
            return L.moe_fp8_block_glu_backward(R(desc), xq, xs, X, off, rows, div, P, gate, up, q, s, w, nb, fl, NUL)
        return L.moe_fp8_block_glu_forward(R(desc), xq, xs, X, off, rows, div, P, q, s, gate, up, w, nb, fl, NUL)

    assert call(desc=_desc(E=4, glu=int(back))) == INV                      # the other form of weights
    assert call(desc=_desc(E=4, N=160, glu=int(not back))) == UNS           # a block of 128 columns is cut
    assert call(div=0) == INV and call(P=-1) == INV and call(X=0) == INV and call(X=999, rows=NUL) == INV
    assert call(off=NUL) == INV and call(off=NUL, rows=NUL) == INV          # E = 4 without groups
    assert call(q=NUL) == INV and call(s=NUL) == INV and call(q=MIS) == INV
    assert call(gate=NUL) == INV and call(up=NUL) == INV and call(gate=MIS) == INV
    if back:
        assert call(gate=NUL, up=NUL) == INV
    assert call(fl=3) == INV and call(nb=ws - 1) == WSE and call(w=NUL) == WSE
    assert call(w=ctypes.c_void_p((1 << 20) + 16)) == INV
    assert call(X=1 << 24) == UNS and call(P=(1 << 31) - 1) == UNS
    assert call(P=0, q=NUL, s=NUL, off=NUL, w=NUL, nb=0) == 0
    # streamed weights: the rows go through the workspace in fp32
    assert size(1000, 4, 256, 256, _lib.MOE_FLAG_FORCE_DECODE) >= 1000 * 256 * 4
    assert call(fl=_lib.MOE_FLAG_FORCE_DECODE, nb=1000 * 256 * 4 - 1) == WSE


SIZES = [(1, 128, 128), (8, 512, 512), (64, 1536, 4096), (250, 2048, 7168), (3, 640, 256), (1024, 128, 128)]


@pytest.mark.parametrize("E,N,K", SIZES)
def test_workspace_sizes_never_fall_with_more_rows(E, N, K):
    """A workspace for the largest batch serves every smaller one, whichever path either takes."""
    rows = sorted({*range(0, 400), *range(400, 40000, 97),
                   *(m * E + d for m in (6, 12) for d in (-1, 0, 1)), 1 << 20, (1 << 31) - 257} - {-1})
    kinds = [lambda P, f=f: L.moe_fp8_block_glu_workspace_size(P, E, N, K, f)
             for f in (0, _lib.MOE_FLAG_FORCE_DECODE, _lib.MOE_FLAG_FORCE_PREFILL)]
    kinds += [lambda P: L.moe_fp8_block_grouped_workspace_size(P, E, N, K),
              lambda P: L.moe_fp8_block_weight_grad_workspace_size(P, E, N, K)]
    for i, size in enumerate(kinds):
        got = [size(P) for P in rows]
        falls = [(rows[j], rows[j + 1]) for j in range(len(rows) - 1) if got[j + 1] < got[j]]
        assert not falls, (i, falls[:3])
        assert all(got[1:])


def test_weight_grad_refusals():
    f, size = L.moe_fp8_block_weight_grad, L.moe_fp8_block_weight_grad_workspace_size
    assert size(-1, 1, 128, 128) == 0 and size(10, 1, 96, 128) == 0 and size(10, 1, 128, 96) == 0
    assert 400 <= size(100, 1, 128, 128) < 128 * 128 * 4                    # one part: the rows' indices
    ws = size(4096, 1, 256, 128)
    assert ws >= 2 * 256 * 128 * 4 + 4 * 4096

    def call(yq=A, ys=A, xq=A, xs=A, X=4096, off=NUL, rows=NUL, div=1, P=4096, E=1, N=256, K=128, dw=A, t=BF, w=A, nb=ws):
        return f(yq, ys, xq, xs, X, off, rows, div, P, E, N, K, dw, t, w, nb, NUL)

    assert call(P=-1) == INV and call(X=-1) == INV and call(X=0) == INV and call(X=4095) == INV and call(div=0) == INV
    assert call(E=0) == INV and call(E=2) == INV and call(rows=A) == INV and call(off=MIS) == INV
    assert call(N=96) == UNS and call(K=96) == UNS and call(E=1025, off=A) == UNS
    assert call(N=1 << 20, K=1 << 20) == UNS and call(P=(1 << 31) - 1) == UNS
    assert call(t=FH) == INV and call(dw=NUL) == INV and call(dw=MIS) == INV
    assert call(yq=NUL) == INV and call(ys=MIS) == INV and call(xq=MIS) == INV and call(xs=NUL) == INV
    assert call(nb=ws - 1) == WSE and call(w=NUL) == WSE and call(w=ctypes.c_void_p((1 << 20) + 16)) == INV


@pytest.mark.parametrize("N,K", [(1 << 20, (1 << 19) - 128), ((1 << 19) - 128, 1 << 20)])
def test_weight_grad_refuses_as_many_tiles_as_no_launch_holds(N, K):
    """Half tiles count as whole ones: 2^23 workgroups of 512 threads are 2^32."""
    size = L.moe_fp8_block_weight_grad_workspace_size(64, 1, N, K)
    for P in (0, 64):
        assert L.moe_fp8_block_weight_grad(A, A, A, A, 64, NUL, NUL, 1, P, 1, N, K, A, BF, A, size, NUL) == UNS


def test_wrappers_refuse_host_tensors_and_wrong_shapes():
    u8, f32 = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(2, 4)
    with pytest.raises(ValueError):
        moe.quant_fp8_block(torch.zeros(4, 256))
    with pytest.raises(TypeError):
        moe.quant_fp8_block(torch.zeros(4, 256, dtype=torch.float64))
    with pytest.raises(ValueError):
        moe.dequant_fp8_block(u8, f32)
    with pytest.raises(ValueError):
        moe.dequant_fp8_block(u8[0], f32)
    with pytest.raises(ValueError):
        moe.fp8_block_prepack(u8, f32)
    with pytest.raises(ValueError):
        moe.fp8_block_prepack_glu(u8, f32, None, None)
    with pytest.raises(ValueError):
        moe.fp8_block_prepack_t(u8, f32, u8, None)
    with pytest.raises(ValueError):
        moe.fp8_block_weight_grad(u8, f32, u8, f32)
    w = moe.Fp8BlockWeights(buffer=u8, desc=_desc(glu=1))
    with pytest.raises(ValueError, match="plain"):
        moe.fp8_block_dense(w, u8, f32)
    with pytest.raises(ValueError, match="gate and up"):
        moe.fp8_block_glu(moe.Fp8BlockWeights(buffer=u8, desc=_desc()), u8, f32)


def test_reference_quantiser():
    """The reference's codes are the nearest ones, ties to even, and its scale the block's largest magnitude / 448."""
    v = torch.cat([ref.E4M3, -ref.E4M3, (ref.E4M3[1:] + ref.E4M3[:-1]) / 2])
    v = v[: len(v) // 127 * 127].view(-1, 127)
    v = torch.cat([v, torch.full((len(v), 1), 448.0)], 1)     # the last element fixes the scale at 1
    q, s = ref.quant(v)
    assert (s == 1).all()
    got = ref.rows(q, s)
    gaps = (v.double().unsqueeze(-1) - torch.cat([-ref.E4M3, ref.E4M3])).abs().amin(-1)
    assert torch.equal((got - v).abs(), gaps)
    assert torch.equal(got.float(), v.float().to(torch.float8_e4m3fn).float())
    q, s = ref.quant(torch.tensor([[0.0] * 128, [float("nan")] + [1.0] * 127, [float("-inf")] + [1.0] * 127]))
    assert s[0, 0] == 2.0 ** -110 / 448 and s[0, 1:].isnan().all() and not q.any()
