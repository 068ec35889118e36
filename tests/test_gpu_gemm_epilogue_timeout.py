"""Failure path of the fused GEMM's bounded waits, made to happen without a fault: with a bound
of a few clock cycles the waits run out in normal operation, the residual copies' among them.
The kernel records NVFP4_ERR_TIMEOUT, lets its own copies land and returns; the same GEMM right
after it, with the default bound, is right."""
import pytest
import torch

from gpu_util import DEV
from nvfp4_bit_quantized_amax_b200 import capi

pytestmark = pytest.mark.gpu
FORMS = {  # residual, Z kept
    "residual": (True, False),       # a box under way while the accumulator is waited for
    "residual and Z": (True, True),  # fetched after Z, then waited for
    "Z": (False, True),
    "neither": (False, False),
}


def problem(M, N, K):
    gen = torch.Generator(device=DEV).manual_seed(M)

    def operand(rows):
        return (torch.randint(0, 256, (rows, K // 2), generator=gen, device=DEV, dtype=torch.uint8),
                torch.randint(0x20, 0x48, (capi.scale_bytes(rows, K),), generator=gen, device=DEV, dtype=torch.uint8))
    (A, sA), (B, sB) = operand(M), operand(N)
    bias = torch.randn(N, generator=gen, device=DEV)
    res = torch.randn(M, N, generator=gen, device=DEV).bfloat16()
    return dict(A=A, sfA=sA, B=B, sfB=sB, alpha=0.01 / K ** 0.5, M=M, N=N, K=K, bias=bias, act=capi.ACT_SILU), res


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("M,N,K", [(128, 512, 8192), (100, 1000, 2048), (512, 512, 8192), (600, 20000, 2048)])
def test_waits_run_out_then_the_epilogue_recovers(M, N, K, form):
    kw, res = problem(M, N, K)
    use_res, use_z = FORMS[form]
    kw["residual"] = res if use_res else None

    def outputs():
        z = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV) if use_z else None
        return dict(D_bf16=torch.zeros(M, N, dtype=torch.bfloat16, device=DEV), D_f32=torch.zeros(M, N, device=DEV), Z=z,
                    status=torch.zeros(1, dtype=torch.int32, device=DEV))

    def same(a, b):
        return all(torch.equal(a[k], b[k]) for k in ("D_bf16", "D_f32", "Z") if a[k] is not None)
    want = outputs()
    capi.nvfp4_gemm_epilogue(**kw, **want)
    assert want["status"].item() == 0 and want["D_f32"].any()
    seen = set()
    # a cycle: the first wait runs out; then later ones; at last none
    for cycles in (1, 1, 200, 600, 1000, 1500, 2000, 3000, 5000, 10000, 30000, 1 << 24, 0):
        got = outputs()
        capi.nvfp4_gemm_epilogue_wait_limit(wait_cycles=cycles, **kw, **got)
        status = got["status"].item()  # the kernel returned
        assert status in (0, capi.ERR_TIMEOUT)
        if status == 0:
            assert same(got, want)
        if cycles == 1:
            assert status == capi.ERR_TIMEOUT
        if cycles in (0, 1 << 24):
            assert status == 0
        seen.add(status)
        # the next call finds the context, its barriers and its tensor memory as they should be
        again = outputs()
        capi.nvfp4_gemm_epilogue(**kw, **again)
        assert again["status"].item() == 0 and same(again, want)
    assert seen == {0, capi.ERR_TIMEOUT}


def test_a_negative_bound_is_refused():
    z = torch.zeros(64, dtype=torch.uint8, device=DEV)
    d = torch.zeros(128, 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(capi.NVFP4Error):
        capi.nvfp4_gemm_epilogue_wait_limit(z, z, z, z, 1.0, 128, 8, 64, -1, D_bf16=d)
