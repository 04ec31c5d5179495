"""Index arithmetic of the MXFP4 products (csrc/mx4.h) at the ends of its range,
compiled for the host."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp4_routed_expert_amd", "csrc")
SRC = os.path.join(HERE, "native", "mx4_host.cpp")
SO = os.path.join(HERE, "native", "_build", "libmx4_host.so")
MAX_P = (1 << 31) - 257          # the largest row count that a grouped product takes
ROWS = 32                        # token rows of a pass


@pytest.fixture(scope="module")
def lib():
    newest = max(os.path.getmtime(f) for f in (SRC, os.path.join(CSRC, "mx4.h"), os.path.join(CSRC, "common.h")))
    if not os.path.exists(SO) or os.path.getmtime(SO) < newest:
        os.makedirs(os.path.dirname(SO), exist_ok=True)
        subprocess.check_call(["/opt/rocm/bin/hipcc", "-O2", "-fPIC", "-shared", "-x", "hip", "--offload-host-only", SRC,
                               "-o", SO + ".tmp"])
        os.replace(SO + ".tmp", SO)
    lib = ctypes.CDLL(SO)
    i32 = ctypes.c_int
    lib.host_walk.argtypes = [i32, i32, i32, ctypes.c_long, ctypes.POINTER(i32)]
    lib.host_walk.restype = ctypes.c_long
    return lib


@pytest.mark.parametrize("side_by_side", [1, 2, 512, 1536])      # workgroups that share a group's passes
@pytest.mark.parametrize("begin,end", [(0, 1), (0, 32), (0, 33), (5, 100000), (0, MAX_P), (7, MAX_P), (MAX_P - 1, MAX_P),
                                       (0, MAX_P - 31), (MAX_P - 49153, MAX_P)])
def test_streaming_walk_stays_in_its_group(lib, side_by_side, begin, end):
    """Workgroup z of a group takes passes z, z + n, ...: each pass once, none outside the group's rows."""
    passes = (end - begin + ROWS - 1) // ROWS
    for z in sorted({0, 1, side_by_side // 2, side_by_side - 1}):
        want = len(range(z, passes, side_by_side))
        if not want:
            continue                                              # the workgroup ends before its walk
        last = ctypes.c_int(0)
        first = begin + ROWS * z
        assert lib.host_walk(first, ROWS * side_by_side, end, want, ctypes.byref(last)) == want
        assert last.value == first + ROWS * side_by_side * (want - 1)
