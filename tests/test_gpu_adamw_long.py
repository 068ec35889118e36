"""GPU tests of the AdamW step over lists long enough for several passes per CTA (8-bit
moments): bit for bit what the same tensors give in short lists, and spans of it against the
definition."""
import numpy as np
import pytest
import torch

from ffn_ref import encode8
from gpu_util import DEV
from nvfp4_bit_quantized_amax_b200 import capi

pytestmark = pytest.mark.gpu
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, seed=(9 << 33) + 77)
PASS, CHUNK = 2048, 4 * 2048  # elements of a pass and of a CTA's four
f32 = np.float32


def tensors(sizes, grad_f32):
    gen = torch.Generator(device=DEV).manual_seed(len(sizes))
    z8 = lambda n: torch.zeros(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    out = []
    for n in sizes:
        g = 1e-3 * torch.randn(n, generator=gen, device=DEV)
        out.append(dict(p=0.02 * torch.randn(n, generator=gen, device=DEV), g=g if grad_f32 else g.bfloat16(),
                        w=torch.zeros(n, dtype=torch.bfloat16, device=DEV), m=z8(n), v=z8(n), ms=z8((n + 31) // 32),
                        vs=z8((n + 31) // 32)))
    return out


def plan(ts, decay):
    pick = lambda k: [t[k] for t in ts]  # noqa: E731
    return capi.adamw_plan(pick("p"), pick("g"), pick("m"), pick("v"), w=pick("w"), m_scale=pick("ms"), v_scale=pick("vs"),
                           weight_decay=decay)


@pytest.mark.parametrize("grad_f32", [False, True])
def test_8_bit_states_over_several_passes(ora, grad_f32):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    several = PASS * 4 * 16 * sms  # parameters from which a CTA takes four passes
    big = several // 2 // CHUNK * CHUNK
    # ends in the first, second, third and last pass of a chunk, whole chunks, empty and tiny ones
    sizes = [big + 3, 0, 5, 3 * CHUNK + PASS + 17, 31, CHUNK + 2 * PASS + 1, 5 * CHUNK, 2 * CHUNK + 3 * PASS + 2047, 0,
             big + CHUNK + 33, PASS - 1]
    assert sum(sizes) >= several > max(sizes)
    decay = [0.1 * (i % 3) for i in range(len(sizes))]
    a, b = tensors(sizes, grad_f32), tensors(sizes, grad_f32)
    first = [t["g"].float().cpu().numpy() for t in a]
    whole = plan(a, decay)
    none = tensors([0], grad_f32)[0]
    alone = [plan([none] * i + [t], [0.0] * i + [d]) for i, (t, d) in enumerate(zip(b, decay))]
    for step in (1, 2):
        capi.nvfp4_adamw(whole, step=step, **HYPER)
        for one in alone:  # the tensor's number in its list is part of its draws
            capi.nvfp4_adamw(one, step=step, **HYPER)
        for i, (x, y) in enumerate(zip(a, b)):
            for k in x:
                assert torch.equal(x[k], y[k]), (i, k, step)
        if step == 1:  # from zero states: m = 0.1 g, r = sqrt(0.05 g^2), each operation rounded
            for i, n in enumerate(sizes):
                ends = [0, PASS, CHUNK - 64, CHUNK + 2 * PASS - 32, n // CHUNK * CHUNK, (n - 1) // 32 * 32 - 64]
                for at in {e for e in ends if 0 <= e < n}:
                    g = first[i][at:at + 160]
                    m = g * f32(1 - 0.9) + f32(0)
                    r = np.sqrt(g * g * f32(1 - 0.95) + f32(0))
                    s = HYPER["seed"]
                    d = [ora.philox4x32_10((q & 0xFFFFFFFF, q >> 32, i, step), (s & 0xFFFFFFFF, s >> 32))
                         for q in range(at // 4, (at + len(g) + 3) // 4)]
                    d = np.array(d, dtype=np.uint32).reshape(-1)[:len(g)].astype(np.int64)
                    for k, ref in zip(("m", "ms", "v", "vs"), encode8(m, d & 0xFFFF, False) + encode8(r, d >> 16, True)):
                        got = a[i][k][at:at + 160] if len(k) == 1 else a[i][k][at // 32:(at + 160 + 31) // 32]
                        assert np.array_equal(got.cpu().numpy(), ref), (i, at, k)
