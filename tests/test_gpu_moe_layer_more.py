"""GPU tests of the expert layer where a warp's lanes part: rows whose length is an odd
multiple of 128 (half a warp has one load fewer), warps without an expert, clusters with
fewer tokens than they hold."""
import pytest
import torch

from ffn_ref import moe64, random_experts
from gpu_util import DEV
from nvfp4_bit_quantized_amax_b200 import capi

pytestmark = pytest.mark.gpu


def layer(T, E, topk, K, F, act=capi.ACT_SILU, gated=True, scoring=capi.SCORE_SOFTMAX, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, K, generator=gen, device=DEV).bfloat16()
    router = (1.5 / K ** 0.5 * torch.randn(E, K, generator=gen, device=DEV)).bfloat16()
    w1 = random_experts(gen, E, F * (2 if gated else 1), K, DEV)
    w2 = random_experts(gen, E, K, F, DEV)
    return dict(x=x, router=router, w1=w1, w2=w2, F=F, topk=topk, act=act, gated=gated, scoring=scoring, sel_bias=None,
                renormalize=True, route_scale=1.0)


def call(c):
    T, K = c["x"].shape
    E = c["router"].shape[0]
    ws = torch.full((capi.moe_layer_workspace_bytes(T, E, c["topk"], K, c["F"]),), 0xFF, dtype=torch.uint8, device=DEV)
    y = torch.full((T, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    idx = torch.full((T, c["topk"]), -1, dtype=torch.int32, device=DEV)
    weight = torch.full((T, c["topk"]), float("nan"), device=DEV)
    capi.nvfp4_moe_layer(c["x"], c["router"], c["w1"], c["w2"], y, c["F"], c["topk"], ws, act=c["act"], gated=c["gated"],
                         scoring=c["scoring"], select_bias=c["sel_bias"], renormalize=c["renormalize"],
                         route_scale=c["route_scale"], topk_idx=idx, topk_weight=weight)
    return y, idx, weight


@pytest.mark.parametrize("K", [128, 384])
@pytest.mark.parametrize("E", [1, 9, 65])
@pytest.mark.parametrize("T", [1, 19, 38, 75, 127])  # clusters of 1, 2, 4, 8 and 8 tokens, the last one not full
def test_router_with_parted_lanes(T, E, K):
    c = layer(T, E, min(E, 3), K, 128, seed=T + E)
    y, idx, weight = call(c)
    ref, tol, ridx, rw = moe64(**c)
    assert torch.equal(idx.long(), ridx)
    assert ((weight.double() - rw).abs() <= 2.0 ** -18 * rw + 1e-37).all()
    assert ((y.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("T,E,topk,K,F", [
    (128, 2, 2, 16384, 128),   # every token on both experts, four or two tokens a pass
    (128, 2, 1, 128, 16384),
    (127, 3, 3, 4096, 4096),
    (128, 16, 16, 640, 640),   # every token on every expert
    (65, 1024, 16, 256, 128),
    (2, 2, 1, 16384, 16384),
])
@pytest.mark.parametrize("gated", [False, True])
def test_many_passes_and_the_largest_sizes(T, E, topk, K, F, gated):
    c = layer(T, E, topk, K, F, gated=gated, seed=T + K)
    y, idx, _ = call(c)
    ref, tol, ridx, _ = moe64(**c)
    assert torch.equal(idx.long(), ridx)
    assert ((y.double() - ref).abs() <= tol).all()
    assert torch.equal(call(c)[0], y)
