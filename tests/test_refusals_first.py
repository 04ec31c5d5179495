"""Calls of several launches refuse what a later stage would refuse before their
first launch: no HIP call is made (without a GPU a launch would answer MOE_ERR_HIP,
and the calling thread's last HIP error would change)."""
import ctypes
import os

import pytest

from fp4_routed_expert_amd import _lib

A = ctypes.c_void_p(1 << 20)          # aligned stand-in, never dereferenced on error paths
NUL = ctypes.c_void_p(0)
R = ctypes.byref
E, H, I, K = 8, 4096, 128, 2
PREFILL = _lib.MOE_FLAG_FORCE_PREFILL
T_TOO_MANY = (1 << 32) // H           # the tiled expert GEMMs address T * H < 2^32 bytes of rows
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.SO_PATH):
        from fp4_routed_expert_amd import build
        build.build()
    return _lib.lib()


def weights(lib, experts=E):
    w = _lib.MoeFp4Weights()
    w.E, w.H, w.I, w.layout_version, w.packed = experts, H, I, 1, 1 << 20
    w.packed_bytes = lib.moe_fp4_packed_weight_bytes(experts, H, I)
    return w


def block(lib, T, flags, nbytes=BIG):
    n = _lib.MoeBlockNorms(1 << 20, None, _lib.MOE_TYPE_FP32, None, 0, 0, 1.0, 1.0, 1e-6)
    return lib.moe_fp4_block_forward(R(weights(lib)), 1, A, R(n), A, _lib.MOE_TYPE_BF16, T, K, A, A, nbytes, flags, NUL)


def full(lib, T, flags, nbytes=BIG):
    return lib.moe_fp4_layer_forward_full(R(weights(lib)), 1, A, A, T, K, A, A, nbytes, flags, NUL)


def layer(lib, T, flags, nbytes=BIG):
    return lib.moe_fp4_layer_forward(R(weights(lib)), A, A, T, K, A, A, nbytes, flags, NUL)


def shared(lib, T, flags, nbytes=BIG):
    return lib.moe_fp4_shared_expert(R(weights(lib, 1)), A, A, T, A, A, nbytes, flags, NUL)


def grouped(lib, T, flags, nbytes=BIG):
    return lib.moe_fp4_grouped_forward(R(weights(lib)), A, A, A, A, A, A, T, K, A, A, nbytes, flags, NUL)


@pytest.mark.parametrize("call", [block, full, layer, shared, grouped], ids=lambda f: f.__name__)
@pytest.mark.parametrize("T,flags", [(T_TOO_MANY, 0), (T_TOO_MANY, PREFILL), (T_TOO_MANY + 4097, 0)])
def test_rows_past_32_bits(lib, call, T, flags):
    before = lib.moe_last_hip_error()
    assert call(lib, T, flags) == _lib.MOE_ERR_UNSUPPORTED
    assert lib.moe_last_hip_error() == before


@pytest.mark.parametrize("call", [block, full, layer, shared], ids=lambda f: f.__name__)
def test_workspace_comes_first(lib, call):
    """A workspace that is too small is still what such a call reports."""
    assert call(lib, T_TOO_MANY, 0, nbytes=1) == _lib.MOE_ERR_WORKSPACE
