"""silu of fdllm_linear with an fp32 result, over its whole range: W = I, so that
the argument is x itself."""
import pytest
import torch

import kv_cache_attention_flash_b200 as fd

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("rows", [1, 40, 700])
@pytest.mark.parametrize("gate", [False, True])
def test_silu_keeps_fp32(rows, gate):
    """Relative to the value: exp(-|x| / 2) 2 steps of 2^-23, squared 2 x 2 + 1/2;
    x t t 2 x 2 + 2 x 1/2; 1 + e half a step and at most half of e's error; the
    quotient 2: under 11 steps, 2^-19.5. Below 2^-126 three roundings to the
    spacing of 2^-149. The product by an up of 1 is exact."""
    n = rows * 64
    x = torch.cat([torch.linspace(-110, 110, n // 2), torch.linspace(-92, -80, n // 4),
                   torch.linspace(-3, 3, n - n // 2 - n // 4)]).cuda().to(BF).view(rows, 64)
    eye = torch.eye(64, device="cuda").to(BF)
    if gate:
        up = torch.zeros(64, 64, device="cuda").to(BF)
        one = torch.ones(64, dtype=torch.float32, device="cuda")
        y = fd.fdllm_linear(x, up, bias=one, act="silu", w_gate=eye, out_dtype=torch.float32)
    else:
        y = fd.fdllm_linear(x, eye, act="silu", out_dtype=torch.float32)
    d = x.double()
    want = d / (1 + torch.exp(-d))
    off = (y.double() - want).abs()
    assert bool((off <= 2.0 ** -19.5 * want.abs() + 2.0 ** -147).all()), float((off / want.abs()).nan_to_num(0).max())
    assert bool(((x.float() < -88.8) & (x.float() > -100)).any())


def test_silu_of_what_is_not_finite():
    x = torch.tensor([[float("inf"), 0.0], [float("nan"), 0.0], [0.0, 0.0]], device="cuda")
    x = torch.nn.functional.pad(x, (0, 6)).to(BF)
    w = torch.zeros(8, 8, device="cuda").to(BF)
    w[0, 0] = 1
    y = fd.fdllm_linear(x, w, act="silu", out_dtype=torch.float32)
    assert float(y[0, 0]) == float("inf") and bool(y[1, 0].isnan()) and bool((y[2] == 0).all())
