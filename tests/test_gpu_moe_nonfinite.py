"""GPU tests of the expert layer's router where logits are infinite or NaN."""
import pytest
import torch

from ffn_ref import random_experts
from gpu_util import DEV
from nvfp4_bit_quantized_amax_b200 import capi

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def route(logits, topk, **kw):
    """The choice for tokens with these logits [T][E]: token t has a one in column t and the
    router's column t holds its logits.  E from 2 up, K and F 128."""
    T, E = logits.shape
    gen = torch.Generator(device=DEV).manual_seed(E)
    x = torch.zeros(T, 128, dtype=torch.bfloat16, device=DEV)
    x[torch.arange(T), torch.arange(T)] = 1
    # an infinite or NaN entry spoils the other tokens' sums (0 times it): one token at a time
    w1, w2 = random_experts(gen, E, 128, 128, DEV), random_experts(gen, E, 128, 128, DEV)
    ws = torch.empty(capi.moe_layer_workspace_bytes(1, E, topk, 128, 128), dtype=torch.uint8, device=DEV)
    idx = torch.full((T, topk), -1, dtype=torch.int32, device=DEV)
    weight = torch.full((T, topk), -1.0, device=DEV)
    y = torch.empty_like(x)
    for t in range(T):
        router = torch.zeros(E, 128, dtype=torch.bfloat16, device=DEV)
        router[:, t] = logits[t].to(DEV).bfloat16()
        capi.nvfp4_moe_layer(x[t:t + 1], router, w1, w2, y[t:t + 1], 128, topk, ws, gated=False, topk_idx=idx[t:t + 1],
                             topk_weight=weight[t:t + 1], **kw)
    return idx.cpu(), weight.cpu()


def order(keys, topk):
    """Descending, equal ones by index, NaN behind -infinity."""
    rank = sorted(range(len(keys)), key=lambda e: (keys[e] != keys[e], -keys[e] if keys[e] == keys[e] else 0.0, e))
    return rank[:topk]


ROWS = [
    [1.0, NAN, -INF, 2.0, NAN, -INF],
    [NAN, -INF, NAN, -INF, NAN, -INF],
    [NAN, NAN, NAN, NAN, NAN, NAN],
    [-INF, NAN, 0.0, -0.0, NAN, -3.0],
    [-INF, -INF, -INF, -INF, -INF, -INF],
    [3.0, -INF, NAN, 3.0, NAN, 3.0],
]


@pytest.mark.parametrize("scoring", [capi.SCORE_SOFTMAX, capi.SCORE_SIGMOID])
@pytest.mark.parametrize("topk", [1, 3, 6])
def test_nan_comes_behind_minus_infinity(topk, scoring):
    logits = torch.tensor(ROWS)
    idx, _ = route(logits, topk, scoring=scoring)
    for t, row in enumerate(ROWS):
        assert idx[t].tolist() == order(row, topk), t


def test_nan_comes_behind_minus_infinity_with_a_bias():
    """A bias of -infinity keeps an expert from being chosen before any finite score; a NaN
    score comes after it all the same."""
    bias = torch.tensor([0.0, -INF, 0.25, -INF, NAN, 0.0], device=DEV)
    logits = torch.tensor([[1.0, 5.0, 0.0, 4.0, 9.0, NAN]])
    s = torch.sigmoid(logits.double())[0] + bias.cpu().double()
    for topk in (1, 4, 6):
        idx, _ = route(logits, topk, scoring=capi.SCORE_SIGMOID, select_bias=bias)
        assert idx[0].tolist() == order(s.tolist(), topk)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_one_nan_spoils_a_softmax(bias, renormalize):
    """softmax has no value where one logit has none, whichever experts are taken; logistic
    scores stand each for itself."""
    logits = torch.tensor([[1.0, 3.0, NAN, 2.0], [0.5, NAN, -INF, 0.25], [1.0, 3.0, -INF, 2.0]])
    sel = torch.zeros(4, device=DEV) if bias else None
    idx, w = route(logits, 2, scoring=capi.SCORE_SOFTMAX, select_bias=sel, renormalize=renormalize)
    assert w[:2].isnan().all() and w[2].isfinite().all()
    assert idx[2].tolist() == [1, 3] and (bias or idx[:2].tolist() == [[1, 3], [0, 3]])
    idx, w = route(logits, 2, scoring=capi.SCORE_SIGMOID, select_bias=sel, renormalize=renormalize)
    assert w.isfinite().all() and idx.tolist() == [[1, 3], [0, 3], [1, 3]]
    s = torch.sigmoid(logits.double()).gather(1, idx.long())
    s = s / s.sum(1, keepdim=True) if renormalize else s
    assert ((w.double() - s).abs() <= 2.0 ** -18 * s).all()
