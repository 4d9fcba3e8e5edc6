"""The CTAs that a scored routing of many tokens takes run in one round: on a device with fewer SMs (a part of one,
say) there are fewer of them, with more tokens each, and the workspace of the public query still holds their
counts."""
import ctypes
import os
import subprocess

import pytest

import moe_expert_gemm_mxfp4_b200 as mx
from moe_expert_gemm_mxfp4_b200 import build as mxbuild

CODE = """
#include "route_chunks.h"
extern "C" long long chunk(long long T, int sms) { return mx::route_chunk(T, sms); }
extern "C" long long chunks(long long T, int sms) { return mx::route_chunks(T, sms); }
"""


@pytest.fixture(scope="module")
def dealt(tmp_path_factory):
    d = tmp_path_factory.mktemp("chunks")
    (d / "chunks.cc").write_text(CODE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", mxbuild.CSRC, "-o", str(d / "chunks.so"),
                    str(d / "chunks.cc")], check=True, timeout=120)
    lib = ctypes.CDLL(os.path.join(d, "chunks.so"))
    for f in (lib.chunk, lib.chunks):
        f.restype, f.argtypes = ctypes.c_longlong, [ctypes.c_longlong, ctypes.c_int]
    return lib


@pytest.mark.parametrize("sms", [1, 2, 18, 36, 74, 132, 147, 148, 160])
def test_no_more_ctas_than_sms(dealt, sms):
    mxbuild.build()
    for T in (129, 130, 143, 145, 1000, 1184, 1185, 1192, 4737, 65536, (1 << 31) - 1):
        c, n = dealt.chunk(T, sms), dealt.chunks(T, sms)
        assert n <= min(sms, 148) and c >= 8
        assert (n - 1) * c < T <= n * c           # every token has a chunk, and no chunk is empty
        for E in (1, 64, 255, 256):
            assert n * (-(-E // 4) * 16) <= mx.moe_mxfp4_route_scored_workspace_size(T, E, 1)


def test_a_whole_gpu_is_used(dealt):
    assert [dealt.chunks(T, 148) for T in (129, 1184, 1185, 8192, 65536)] == [17, 148, 132, 147, 148]
