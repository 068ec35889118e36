"""GPU tests of the epilogue's backward where the last columns part a warp: every N % 32 that
N % 8 == 0 allows, with one and with several clusters per strip of columns."""
import pytest
import torch

from ffn_ref import U
from gpu_util import DEV
from nvfp4_bit_quantized_amax_b200 import capi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [8, 16, 24, 32, 40, 232, 248, 256, 264, 1000, 2056])
@pytest.mark.parametrize("M", [1, 200, 300, 2600])
def test_column_sums_at_every_end(M, N):
    """Without an activation dZ is dY and dbias its column sums: at most M roundings in any
    order.  The columns behind N keep what they held."""
    gen = torch.Generator(device=DEV).manual_seed(M + N)
    dY = torch.randn(M, N, generator=gen, device=DEV).bfloat16()
    dZ = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    db = torch.full((N + 64,), 7.0, device=DEV)
    ws = torch.empty(max(16, capi.epilogue_backward_workspace_bytes(M, N)), dtype=torch.uint8, device=DEV)
    capi.nvfp4_epilogue_backward(dY, dY, dZ, dbias=db[:N], workspace=ws)
    y = dY.double()
    assert torch.equal(dZ, dY) and (db[N:] == 7).all()
    assert ((db[:N].double() - y.sum(0)).abs() <= M * U * y.abs().sum(0)).all()
