"""GPU tests of the fused GEMM epilogue over many tiles per CTA, where a warp's staging buffer
passes from one residual box, and one tile, to the next."""
import pytest
import torch

from ffn_ref import U
from gpu_util import DEV
from nvfp4_bit_quantized_amax_b200 import capi
from nvfp4_bit_quantized_amax_b200 import synthetic as syn

pytestmark = pytest.mark.gpu


def problem(M, N, K, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def operand(rows):
        return (torch.randint(0, 256, (rows, K // 2), generator=gen, device=DEV, dtype=torch.uint8),
                torch.randint(0x20, 0x48, (capi.scale_bytes(rows, K),), generator=gen, device=DEV, dtype=torch.uint8))
    (A, sA), (B, sB) = operand(M), operand(N)
    kw = dict(A=A, sfA=sA, B=B, sfB=sB, alpha=0.01 / K ** 0.5, M=M, N=N, K=K)
    bias = torch.randn(N, generator=gen, device=DEV)
    res = torch.randn(M, N, generator=gen, device=DEV).bfloat16()
    return kw, bias, res


@pytest.mark.parametrize("M,N,K", [(128, 512, 64), (77, 1000, 320), (33, 264, 64), (1, 8, 64), (100, 340984, 64),
                                   (300, 1032, 64), (2000, 10248, 128)])
def test_fp32_output_of_ragged_rows(M, N, K):
    """fp32 stores that only the rows inside D take, between two loads of the accumulator: the
    output alone, through both epilogues, equals the one stored beside bf16."""
    kw, bias, _ = problem(M, N, K, M + N)
    acc, d, d2 = (torch.full((M, N), float("nan"), device=DEV) for _ in range(3))
    d16 = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    plain = (kw["A"], kw["sfA"], kw["B"], kw["sfB"], kw["alpha"], M, N, K)
    capi.nvfp4_gemm(*plain, D_f32=acc, status=status)
    capi.nvfp4_gemm(*plain, D_f32=d2, D_bf16=d16, status=status)
    assert torch.equal(acc, d2) and torch.equal(acc.bfloat16(), d16) and acc.isfinite().all()
    capi.nvfp4_gemm_epilogue(**kw, D_f32=d, act=capi.ACT_RELU2, status=status)
    ref = acc.double().clamp(min=0).square()  # acc rounded once, the square once
    assert ((d.double() - ref).abs() <= 3.01 * U * ref + 1e-37).all() and status.item() == 0
    capi.nvfp4_gemm_epilogue(**kw, D_f32=d, bias=bias, act=capi.ACT_GELU, status=status)
    capi.nvfp4_gemm_epilogue(**kw, D_f32=d2, D_bf16=d16, bias=bias, act=capi.ACT_GELU, status=status)
    assert torch.equal(d, d2) and torch.equal(d.bfloat16(), d16) and status.item() == 0


# the first two: pairs of CTAs, with 8 tiles each and with ragged rows and columns; the last
# two: single CTAs (at most 128 rows), 9 tiles each
MANY_TILES = [(2048, 20480, 64), (2000, 10248, 128), (128, 340992, 64), (77, 340984, 64)]


@pytest.mark.parametrize("M,N,K", MANY_TILES)
def test_residual_with_fp32_output_alone(M, N, K):
    """D_f32 with a residual and without Z, the one form with no store between two residual
    boxes: without an activation D is nvfp4_gemm's fp32 output plus the residual."""
    kw, bias, res = problem(M, N, K, M)
    acc = torch.full((M, N), float("nan"), device=DEV)
    capi.nvfp4_gemm(kw["A"], kw["sfA"], kw["B"], kw["sfB"], kw["alpha"], M, N, K, D_f32=acc)
    d = torch.full((M, N), float("nan"), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(3):
        d.fill_(float("nan"))
        capi.nvfp4_gemm_epilogue(**kw, D_f32=d, residual=res, status=status)
        assert status.item() == 0
        ref = acc.double() + res.double()
        # acc is off by half a step of its own, D by half a step of its
        assert ((d.double() - ref).abs() <= 1.01 * U * (acc.double().abs() + ref.abs())).all()
    del acc, ref
    # with the rest of the epilogue, the bf16 output beside it goes through other copies
    d2, d16 = torch.full_like(d, float("nan")), torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    capi.nvfp4_gemm_epilogue(**kw, D_f32=d, bias=bias, act=capi.ACT_SILU, residual=res)
    capi.nvfp4_gemm_epilogue(**kw, D_f32=d2, D_bf16=d16, bias=bias, act=capi.ACT_SILU, residual=res)
    assert torch.equal(d, d2) and torch.equal(d.bfloat16(), d16)


@pytest.mark.parametrize("block_mode,dgrad_rht", [(capi.BLOCK_16X16, 0), (capi.BLOCK_1X16, 0), (capi.BLOCK_1X16, 1)])
def test_linear_fprop_in_place_and_its_options(block_mode, dgrad_rht):
    """The residual in Y's place, the input in Y's place, both at once: as with buffers of their
    own, and the workspace as nvfp4_linear_fprop_ex leaves it."""
    M, K = 192, 256
    gen = torch.Generator(device=DEV).manual_seed(6)
    X, res = (torch.randn(M, K, generator=gen, device=DEV).bfloat16() for _ in range(2))
    W = (0.05 * torch.randn(K, K, generator=gen, device=DEV)).bfloat16()
    bias = torch.randn(K, generator=gen, device=DEV)
    signs = syn.rht_signs(2)

    def call(x, y, **kw):
        ws = torch.zeros(capi.linear_workspace_bytes(M, K, K), dtype=torch.uint8, device=DEV)
        capi.nvfp4_linear_fprop_epilogue(x, W, y, signs, ws, act=capi.ACT_SILU, weight_block_mode=block_mode,
                                         dgrad_rht=dgrad_rht, **kw)
        assert capi.nvfp4_read_status(ws) == 0
        return y, ws
    want, ws = call(X, torch.empty_like(X), bias=bias, residual=res)
    plain = torch.zeros_like(ws)
    capi.nvfp4_linear_fprop_ex(X, W, torch.empty_like(X), signs, plain, weight_block_mode=block_mode, dgrad_rht=dgrad_rht)
    assert torch.equal(ws, plain)
    r = res.clone()
    assert torch.equal(call(X, r, bias=bias, residual=r)[0], want)
    x = X.clone()
    assert torch.equal(call(x, x, bias=bias, residual=res)[0], want)
    alone = call(X, torch.empty_like(X), residual=X)[0]
    x = X.clone()
    assert torch.equal(call(x, x, residual=x)[0], alone)
