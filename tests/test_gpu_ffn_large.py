"""GPU tests of the feed-forward operators on tensors of more than 2^31 elements or bytes: the
places at the ends are checked against 64 bits, and against the same rows in a small call."""
import pytest
import torch

from ffn_ref import U, moe64, random_experts, slope64
from gpu_util import DEV
from nvfp4_bit_quantized_amax_b200 import capi

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def test_epilogue_backward_past_32_bits():
    M, N = 139264, 16384  # 2^31.09 elements
    gen = torch.Generator(device=DEV).manual_seed(0)
    row = torch.randn(512, N, generator=gen, device=DEV).bfloat16()
    Z = row.repeat(M // 512, 1)
    dY = torch.zeros_like(Z)
    dY[:64] = 1
    dY[-512:] = row.flip(0)
    dZ = torch.full_like(Z, float("nan"))
    db = torch.empty(N, device=DEV)
    ws = torch.empty(capi.epilogue_backward_workspace_bytes(M, N), dtype=torch.uint8, device=DEV)
    capi.nvfp4_epilogue_backward(dY, Z, dZ, act=capi.ACT_SILU, dbias=db, workspace=ws)
    small = torch.empty_like(row)
    capi.nvfp4_epilogue_backward(dY[-512:], Z[-512:], small, act=capi.ACT_SILU)
    assert torch.equal(dZ[-512:], small)
    capi.nvfp4_epilogue_backward(dY[:512], Z[:512], small, act=capi.ACT_SILU)
    assert torch.equal(dZ[:512], small)
    assert not dZ[512:-512].any()
    s = slope64(row.double(), capi.ACT_SILU)
    ref = s[:64].sum(0) + (row.flip(0).double() * s).sum(0)
    mag = s[:64].abs().sum(0) + (row.flip(0).double() * s).abs().sum(0)
    # 576 terms that are not zero, each off by 2^-18 (the slope's bound for |z| < 6), summed in fp32
    assert ((db.double() - ref).abs() <= (2.0 ** -18 + 576 * U) * mag).all()


def test_gemm_epilogue_past_32_bits():
    M, N, K = 66048, 32768, 64  # 2^31.01 elements
    gen = torch.Generator(device=DEV).manual_seed(1)

    def operand(rows):
        return (torch.randint(0, 256, (rows, K // 2), generator=gen, device=DEV, dtype=torch.uint8),
                torch.full((capi.scale_bytes(rows, K),), 0x30, device=DEV, dtype=torch.uint8))
    (A, sA), (B, sB) = operand(M), operand(N)
    bias = torch.randn(N, generator=gen, device=DEV)
    res = torch.randn(512, N, generator=gen, device=DEV).bfloat16().repeat(M // 512, 1)
    kw = dict(alpha=0.05, N=N, K=K, bias=bias, act=capi.ACT_GELU)
    top = M - 256
    want = [torch.empty(256, N, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    capi.nvfp4_gemm_epilogue(A[top:], sA[top * K // 16:], B, sB, M=256, D_bf16=want[0], residual=res[top:], Z=want[1], **kw)
    d32 = torch.full((M, N), float("nan"), device=DEV)
    Z = torch.zeros_like(res)
    capi.nvfp4_gemm_epilogue(A, sA, B, sB, M=M, D_bf16=res, D_f32=d32, residual=res, Z=Z, **kw)  # in place
    assert torch.equal(res[top:], want[0]) and torch.equal(Z[top:], want[1])
    for at in range(0, M, 8256):
        d = d32[at:at + 8256]
        assert d.isfinite().all() and torch.equal(d.bfloat16(), res[at:at + 8256])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_32_bits(bits):
    n = (1 << 31) + 5000
    gen = torch.Generator(device=DEV).manual_seed(2)
    tail = 3 << 20
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g[-tail:] = (1e-3 * torch.randn(tail, generator=gen, device=DEV)).bfloat16()
    p = torch.ones(n, device=DEV)
    w = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    dt = torch.float32 if bits == 32 else torch.uint8
    m, v = (torch.zeros(n, dtype=dt, device=DEV) for _ in range(2))
    ms, vs = (torch.zeros((n + 31) // 32, dtype=torch.uint8, device=DEV) for _ in range(2))
    extra = {} if bits == 32 else dict(m_scale=[ms], v_scale=[vs])
    capi.nvfp4_adamw(capi.adamw_plan([p], [g], [m], [v], w=[w], **extra), lr=1e-2, step=1, seed=3)
    gd = g[-tail:].double()
    want = 1 - 1e-2 * gd / (gd.abs() + 1e-8)  # the first step: m / (1 - b1) = g, v / (1 - b2) = g^2
    assert ((p[-tail:].double() - want).abs() <= 2 * U + 32 * U * 1e-2).all()
    assert torch.equal(w[-tail:], p[-tail:].bfloat16())
    for at in range(0, n - tail, 1 << 28):
        part = slice(at, min(at + (1 << 28), n - tail))
        assert (p[part] == 1).all() and (w[part] == 1).all()
    if bits == 32:
        assert ((m[-tail:].double() - 0.1 * gd).abs() <= 4 * U * gd.abs()).all() and not m[:1 << 30].any()
    else:
        assert (v[-tail:] != 0)[gd != 0].all() and not v[:1 << 30].any() and not ms[:1 << 25].any()


def test_expert_layer_past_32_bits():
    """First weights of 4.3 GB: the tokens take the first, middle and last experts."""
    E, K, F, T, topk = 256, 4096, 4096, 6, 3
    gen = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(T, K, generator=gen, device=DEV).bfloat16()
    router = (0.5 / K ** 0.5 * torch.randn(E, K, generator=gen, device=DEV)).bfloat16()
    bias = torch.zeros(E, device=DEV)
    bias[[0, 1, E // 2, E // 2 + 1, E - 2, E - 1]] = 1.0
    w1, w2 = random_experts(gen, E, 2 * F, K, DEV), random_experts(gen, E, K, F, DEV)
    assert w1[0].numel() > 1 << 31 and w2[0].numel() >= 1 << 31
    y = torch.empty_like(x)
    idx = torch.empty(T, topk, dtype=torch.int32, device=DEV)
    ws = torch.empty(capi.moe_layer_workspace_bytes(T, E, topk, K, F), dtype=torch.uint8, device=DEV)
    capi.nvfp4_moe_layer(x, router, w1, w2, y, F, topk, ws, select_bias=bias, topk_idx=idx)
    assert set(idx.unique().tolist()) <= set(bias.nonzero().flatten().tolist()) and (idx == E - 1).any()
    # ffn_ref.decode spreads a whole operand's bytes: the taken experts alone, under new numbers
    taken = idx.unique()
    part = lambda t, k: t.view(E, -1)[taken.long()].reshape(-1) if k < 2 else t[taken.long()]  # noqa: E731
    few = [tuple(part(t, k) for k, t in enumerate(w)) for w in (w1, w2)]
    score = torch.softmax(x.double() @ router.double().t(), -1)
    # the same scores up to their total, which renormalizing takes out
    ref, tol, ridx, _ = moe64(x, router[taken.long()], *few, F, topk, capi.ACT_SILU, True, capi.SCORE_SOFTMAX,
                              torch.full((len(taken),), 0.0, device=DEV), True, 1.0)
    best = (score + bias.double()).topk(topk, -1)[1]
    assert torch.equal(idx.long(), best) and torch.equal(taken.long()[ridx], best)
    assert ((y.double() - ref).abs() <= tol).all()
