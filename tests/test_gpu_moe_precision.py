"""GPU test of what the expert layer keeps of the rows between its projections.

The first projection (no activation) gives every even row of h the value x0 + x1 and every
odd row x0; the second takes their difference, so y is x1 in exact arithmetic.  With x0 = 1
and x1 a bf16 number in [2^-16, 2^-1), x0 + x1 has at most 24 bits: all sums are exact in fp32,
and any rounding of h to fewer than 24 bits shows in y in full.  A row is kept to at least
2^-22 of each value (two fp16 parts, 11 bits each); here the parts hold it exactly: the first
ends at 2^-10, what is left has the 8 bits of x1 at most, and y must equal x1."""
import pytest
import torch

from gpu_util import DEV
from nvfp4_bit_quantized_amax_b200 import capi

pytestmark = pytest.mark.gpu
ONE, MINUS_ONE, SCALE_ONE = 2, 10, 0x38  # E2M1 codes of 1 and -1, E4M3 code of 1


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


@pytest.mark.parametrize("T,E,K,F", [
    (1, 2, 128, 128),
    (3, 1, 128, 256),
    (4, 1, 256, 128),     # a whole tile of the second projection
    (5, 1, 256, 384),     # one token more
    (9, 2, 128, 640),
    (23, 1, 128, 128),    # several passes over the weights
    (128, 3, 256, 128),
    (6, 1, 128, 12288),   # long rows: few tokens at a time
    (3, 1, 128, 16384),
    (64, 16, 1024, 512),
])
def test_rows_between_the_projections_keep_22_bits(T, E, K, F):
    gen = torch.Generator(device=DEV).manual_seed(T + F)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    x1 = torch.exp2(-16 + 15 * torch.rand(T, generator=gen, device=DEV)).bfloat16()
    x1 *= torch.where(torch.arange(T, device=DEV) % 2 == 0, 1, -1)
    x[:, 1] = x1
    router = torch.randn(E, K, generator=gen, device=DEV).bfloat16()
    c1 = torch.zeros(E * F, K, dtype=torch.uint8, device=DEV)
    c1[:, 0] = ONE
    c1[0::2, 1] = ONE
    c2 = torch.zeros(E * K, F, dtype=torch.uint8, device=DEV)
    rows = torch.arange(E * K, device=DEV)
    pair = 2 * torch.randint(0, F // 2, (E * K,), generator=gen, device=DEV)
    c2[rows, pair] = ONE
    c2[rows, pair + 1] = MINUS_ONE
    one = torch.ones(E, device=DEV)
    sf = lambda r, c: torch.full((capi.scale_bytes(r, c),), SCALE_ONE, dtype=torch.uint8, device=DEV)  # noqa: E731
    y = torch.full_like(x, float("nan"))
    ws = torch.empty(capi.moe_layer_workspace_bytes(T, E, 1, K, F), dtype=torch.uint8, device=DEV)
    capi.nvfp4_moe_layer(x, router, (pack(c1), sf(E * F, K), one), (pack(c2), sf(E * K, F), one), y, F, 1, ws,
                         act=capi.ACT_NONE, gated=False)
    assert torch.equal(y, x1[:, None].expand(T, K))
