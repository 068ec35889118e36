"""CPU checks that the feed-forward entry points refuse outputs that share memory with another
tensor.  The addresses are never dereferenced: what is refused is refused on the host, and what
is not has no device to run on here."""
import ctypes as C

import numpy as np
import pytest
import torch

from nvfp4_bit_quantized_amax_b200 import capi

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where no launch can follow")
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from nvfp4_bit_quantized_amax_b200 import build
    build.build()
    return capi.load()


def places(names):
    """One address per name, 256 MB apart."""
    return {n: (i + 1) * 256 * MB for i, n in enumerate(names.split())}


def distances(a, b):
    """Places of a tensor of b bytes relative to one of a bytes: inside, at and beyond its ends."""
    return [0, 16, a - 16, 16 - b, a, -b]


GEMM = "A sfA B sfB sa sb bias res Z bf f32 status"
M, N, K = 200, 264, 320
SIZE = dict(A=M * K // 2, B=N * K // 2, bias=4 * N, res=2 * M * N, Z=2 * M * N, bf=2 * M * N, f32=4 * M * N, sa=4, sb=4, status=4)


def gemm(lib, at):
    e = capi.Epilogue(at["bias"], capi.ACT_SILU, at["res"], at["Z"])
    return lib.nvfp4_gemm_epilogue(at["A"], at["sfA"], at["B"], at["sfB"], at["sa"], at["sb"], 1.0, M, N, K, C.byref(e),
                                   at["bf"], at["f32"], at["status"], None)


def test_gemm_epilogue(lib):
    size = dict(SIZE, sfA=lib.nvfp4_scale_bytes(M, K), sfB=lib.nvfp4_scale_bytes(N, K))
    assert gemm(lib, places(GEMM)) == capi.ERR_CUDA  # no device: everything else was accepted
    outs = ("bf", "f32", "Z", "status")
    for a in outs:
        for b in size:
            if a == b:
                continue
            for d in distances(size[a], size[b]):
                at = places(GEMM)
                at[b] = at[a] + d
                if at[b] % 16:  # refused for another reason
                    continue
                in_place = {a, b} == {"bf", "res"} and d == 0
                meets = -size[b] < d < size[a] and not in_place
                assert gemm(lib, at) == (capi.ERR_ARG if meets else capi.ERR_CUDA), (a, b, d)
    at = places(GEMM)
    at["A"] = at["B"]  # inputs may be one tensor
    at["Z"] = at["f32"] = None
    assert gemm(lib, at) == capi.ERR_CUDA


def test_linear_fprop_epilogue(lib):
    m = n = k = 128
    signs = np.ones(16, dtype=np.int8)
    ws_bytes = capi.linear_workspace_bytes(m, k, n)

    def call(at, epilogue=True):
        e = capi.Epilogue(at["bias"], 0, at["res"], at["Z"])
        return lib.nvfp4_linear_fprop_epilogue(at["X"], at["W"], at["Y"], m, k, n, signs.ctypes.data_as(C.c_void_p), None,
                                               C.byref(e) if epilogue else None, at["ws"], ws_bytes, None)
    names = "X W Y bias res Z ws"
    assert call(places(names)) == capi.ERR_CUDA
    for a, b in (("Z", "Y"), ("Z", "res"), ("Z", "X"), ("Z", "W"), ("Z", "ws"), ("Z", "bias"), ("Y", "bias"), ("Y", "ws"),
                 ("res", "ws")):
        at = places(names)
        at[a] = at[b]
        assert call(at) == capi.ERR_ARG, (a, b)
    at = places(names)
    at["res"] = at["Y"] + 256
    assert call(at) == capi.ERR_ARG
    at["res"] = at["Y"]
    assert call(at) == capi.ERR_CUDA
    at["Y"] = at["res"] = at["X"]  # the input is in the workspace before Y is written
    assert call(at) == call(at, False) == capi.ERR_CUDA
