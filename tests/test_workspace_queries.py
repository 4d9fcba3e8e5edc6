"""The public workspace queries answer every size: 0 for what the calls refuse, never a crash.  Callers size the
buffer before the call that would check the arguments.  (The library is called from a child process: a query that
ends its process must not end the tests.)"""
import ctypes
import subprocess
import sys

import moe_expert_gemm_mxfp4_b200 as mx
from moe_expert_gemm_mxfp4_b200 import _lib
from moe_expert_gemm_mxfp4_b200 import build as mxbuild

BIG = (1 << 62) + 64

# M, K, N, act of calls that mxfp4_linear refuses
REFUSED = [(200, 64, 1, 5), (64, 64, 1, 5), (1 << 30, 64, 1, 5), (200, 64, 511, 5), (200, 48, 512, 0), (1, 33, 8, 0),
           (8, (1 << 20) + 32, 8, 0), ((1 << 30) + 1, 64, 8, 0), (8, 64, (1 << 30) + 2, 0), (1 << 30, 32, 1 << 30, 0),
           (8, 1 << 20, (1 << 20) + 32, 0), (8, 64, 64, 6), (8, 64, 64, -1), (0, 64, 64, 0), (8, 0, 64, 0), (8, 64, 0, 0),
           (-1, 64, 64, 0), (BIG, 64, 64, 0), (8, BIG, 64, 0), (8, 64, BIG, 5), (BIG, BIG, BIG, 5)]


CHILD = """
import ctypes, sys
query = ctypes.CDLL(sys.argv[1]).mxfp4_linear_workspace_size
query.restype, query.argtypes = ctypes.c_size_t, [ctypes.c_int64] * 3 + [ctypes.c_int]
for arg in sys.argv[2:]:
    print(arg, query(*map(int, arg.split(","))), flush=True)
"""


def test_linear_query_of_refused_sizes():
    sizes = [",".join(map(str, s)) for s in REFUSED]
    r = subprocess.run([sys.executable, "-c", CHILD, mxbuild.build(), *sizes], capture_output=True, text=True, timeout=60)
    assert r.stdout.splitlines() == [s + " 0" for s in sizes], (r.returncode, r.stderr[-300:])
    assert r.returncode == 0


def test_linear_query_of_the_largest_sizes():
    """What the call takes is answered, at each limit of the sizes too."""
    mxbuild.build()
    size = mx.mxfp4_linear_workspace_size
    assert size(1 << 30, 64, 64) == 2 * 64 * 64
    assert size(1 << 30, 64, 2, mx.ACT_SWIGLU) == 256
    assert size(1 << 16, 32, 1 << 30) == 2 * 32 * (1 << 30)
    assert size(1 << 20, 1 << 20, 1 << 20) == 2 * (1 << 40)
    assert size(200, 64, 2, mx.ACT_SWIGLU) > 0


def test_scored_routing_without_its_workspace():
    """Up to 128 tokens none is needed; from 129 on one of the stated size, and less, or none, is refused."""
    mxbuild.build()
    at = ctypes.c_void_p(0x10000)      # never dereferenced: the calls are refused

    def call(T, E, ws, nbytes):
        return _lib.load().moe_mxfp4_route_scored(at, _lib.IN_F32, T, E, 1, 0, None, 1, 1, 1, 1, 1.0, at, at, at, at, at, at,
                                                  ws, nbytes, None)

    size = mx.moe_mxfp4_route_scored_workspace_size
    assert all(size(T, E, 1) == 0 for T in (1, 64, 128) for E in (1, 64, 256))
    for T in (129, 1185, 65536):
        for E in (1, 33, 64, 256):
            need = size(T, E, 1)
            # a row of E counts, in whole 16-byte vectors, for each of at most 148 chunks of at least 8 tokens
            assert 0 < need <= (min(148, -(-T // 8)) * (-(-E // 4) * 16) + 255) // 256 * 256
            assert call(T, E, at, need - 1) == _lib.ERR_WORKSPACE
            assert call(T, E, None, need) == _lib.ERR_WORKSPACE
            assert call(T, E, None, 0) == _lib.ERR_WORKSPACE
