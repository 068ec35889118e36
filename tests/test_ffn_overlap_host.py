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


NAMES = "p grad w m v m_scale v_scale"


def adamw(lib, entries, bits, grad_f32=0):
    arr = (capi.AdamWTensor * len(entries))(*[capi.AdamWTensor(*e) for e in entries])
    o = capi.AdamWOpts(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, seed=0, state_bits=bits, grad_f32=grad_f32)
    return lib.nvfp4_adamw(arr, len(entries), C.byref(o), None)


def entry(base, n, bits):
    """One tensor whose buffers lie 64 MB apart from `base` on."""
    at = {x: base + i * 64 * MB for i, x in enumerate(NAMES.split())}
    if bits == 32:
        at["m_scale"] = at["v_scale"] = None
    return dict(at, n=n, wd=0.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("order", ["ascending", "descending"])
def test_adamw(lib, bits, order):
    """Every pair of buffers, inside a tensor and between two: what is written may not be named
    twice, gradients may."""
    n = 1000
    state, sc = (4, 0) if bits == 32 else (1, (n + 31) // 32)
    size = dict(p=4 * n, grad=2 * n, w=2 * n, m=state * n, v=state * n, m_scale=sc, v_scale=sc)
    bases = [4096 * MB, 8192 * MB, 12288 * MB]
    bases = bases if order == "ascending" else bases[::-1]
    kinds = [k for k in NAMES.split() if size[k]]

    def call(change=None):
        e = [entry(b, n, bits) for b in bases]
        e.insert(1, entry(bases[0], 0, bits))  # an empty tensor names memory, but touches none
        if change:
            (i, a), (j, b), d = change
            e[i][a] = e[j][b] + d
        return adamw(lib, [tuple(x.values()) for x in e], bits)
    assert call() == capi.ERR_CUDA  # no device: accepted
    for i, j in ((0, 0), (0, 2), (3, 2), (2, 0)):
        for a in kinds:
            for b in kinds:
                if (i, a) == (j, b):
                    continue
                for d in (0, size[b] // 16 * 16 - 16, 16 - size[a] // 16 * 16):
                    if not -size[a] < d < size[b]:
                        continue
                    want = capi.ERR_CUDA if a == b == "grad" else capi.ERR_ARG
                    assert call(((i, a), (j, b), d)) == want, (i, a, j, b, d)
                # directly behind it
                assert call(((i, a), (j, b), (size[b] + 15) // 16 * 16)) == capi.ERR_CUDA, (i, a, j, b)


def test_adamw_parts_of_one_buffer_per_kind(lib):
    """An optimizer's flat buffers: neighbouring parts, in and out of order."""
    for order in (range(50), reversed(range(50)), [(i * 7) % 50 for i in range(50)]):
        e = []
        for i in order:
            at = entry(4096 * MB, 128, 8)
            e.append(tuple(at[k] + i * s for k, s in zip(NAMES.split(), (512, 256, 256, 128, 128, 4, 4))) + (128, 0.0))
        assert adamw(lib, e, 8) == capi.ERR_CUDA
        e[31] = e[31][:3] + (e[30][3],) + e[31][4:]  # one m named twice
        assert adamw(lib, e, 8) == capi.ERR_ARG


def test_epilogue_backward(lib):
    m, n = 500, 264
    ws = capi.epilogue_backward_workspace_bytes(m, n)
    size = dict(dY=2 * m * n, Z=2 * m * n, dZ=2 * m * n, db=4 * n, ws=ws)

    def call(at, dbias=True):
        return lib.nvfp4_epilogue_backward(at["dY"], at["Z"], capi.ACT_GELU, m, n, at["dZ"], at["db"] if dbias else None,
                                           at["ws"], ws, None)
    for a in ("dZ", "db", "ws"):
        for b in size:
            if a == b:
                continue
            for d in distances(size[a], size[b]):
                at = places("dY Z dZ db ws")
                at[b] = at[a] + d
                if at[b] % 16:
                    continue
                meets = -size[b] < d < size[a] and not (a == "dZ" and b in ("dY", "Z") and d == 0)
                assert call(at) == (capi.ERR_ARG if meets else capi.ERR_CUDA), (a, b, d)
                if "ws" in (a, b):  # without sums the workspace is not touched
                    assert call(at, dbias=False) == capi.ERR_CUDA
    at = places("dY Z dZ db ws")
    at["Z"] = at["dZ"] = at["dY"]
    assert call(at) == capi.ERR_CUDA


def test_moe_layer(lib):
    t, e, topk, k, f = 7, 10, 3, 640, 384
    ws = capi.moe_layer_workspace_bytes(t, e, topk, k, f)
    r1, r2 = e * 2 * f, e * k
    size = dict(x=2 * t * k, router=2 * e * k, y=2 * t * k, bias=4 * e, idx=4 * t * topk, weight=4 * t * topk, ws=ws,
                d1=r1 * k // 2, s1=capi.scale_bytes(r1, k), g1=4 * e, d2=r2 * f // 2, s2=capi.scale_bytes(r2, f), g2=4 * e)
    names = " ".join(size)

    def call(at):
        o = capi.MoeLayerOpts(capi.ACT_SILU, 1, 0, 1, 1.0, at["bias"], at["idx"], at["weight"])
        return lib.nvfp4_moe_layer(at["x"], at["router"], C.byref(capi.Tensor(at["d1"], at["s1"], at["g1"], r1, k)),
                                   C.byref(capi.Tensor(at["d2"], at["s2"], at["g2"], r2, f)), at["y"], t, e, topk, k, f,
                                   C.byref(o), at["ws"], ws, None)
    assert call(places(names)) == capi.ERR_CUDA
    for a in ("y", "ws", "idx", "weight"):
        for b in size:
            if a == b:
                continue
            for d in distances(size[a], size[b]):
                d = d // 256 * 256 if "ws" in (a, b) else d  # the workspace's alignment
                at = places(names)
                at[b] = at[a] + d
                if at[b] % 16:
                    continue
                meets = -size[b] < d < size[a] and not ({a, b} == {"x", "y"} and d == 0)
                assert call(at) == (capi.ERR_ARG if meets else capi.ERR_CUDA), (a, b, d)
    at = places(names)
    at["y"] = at["x"]
    assert call(at) == capi.ERR_CUDA
    at["idx"] = at["x"] + 64
    assert call(at) == capi.ERR_ARG
