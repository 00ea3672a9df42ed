"""The 8-bit layer for a few tokens with scales at the lower end of fp32's range beside large rows of h:
the block's sum takes the scale before the gate, so that no product of two small factors is formed."""
import pytest
import torch

from _fp8 import dequantize
from test_gpu_few import _case, _check, _run

pytestmark = pytest.mark.gpu


def _scaled(c, which, scale):
    """The case with scales `scale` of weight `which` (0 gate, 1 up, 2 down)."""
    q, s = c["w"][which]
    s = scale.expand_as(s).contiguous()
    c["w"][which] = (q, s)
    c["exact"][which] = torch.stack([dequantize(q[e], s[e], 128) for e in range(c["E"])])


# h of about 2^105: up's scales are 2^98 of what they would be, down's 2 to 9 units of 2^-149, or 2^-126
@pytest.mark.parametrize("down", [2, 3, 5, 7, 9, 1 << 23])
@pytest.mark.parametrize("T,E,k,d,F", [(3, 6, 3, 256, 384), (8, 5, 2, 128, 1024), (16, 8, 4, 384, 256)])
def test_smallest_fp32_scales_of_down(T, E, k, d, F, down):
    c = _case(T, E, k, d, F, "e4m3-f32", seed=T + down % 100)
    _scaled(c, 1, torch.tensor(2.0 ** 98, dtype=torch.float32) * c["w"][1][1])
    _scaled(c, 2, torch.tensor(down * 2.0 ** -149, dtype=torch.float32))
    out, ints = _run(c)
    assert bool(out.isfinite().all()) and bool((out != 0).any())
    _check(c, out, ints)


@pytest.mark.parametrize("down", [0, 1, 2])
@pytest.mark.parametrize("T", [2, 13])
def test_smallest_e8m0_scales_of_down(T, down):
    c = _case(T, 6, 3, 256, 384, "e4m3-e8m0", seed=T + down)
    _scaled(c, 1, (c["w"][1][1].int() + 98).to(torch.uint8))
    _scaled(c, 2, torch.tensor(down, dtype=torch.uint8))
    out, ints = _run(c)
    assert bool(out.isfinite().all()) and bool((out != 0).any())
    _check(c, out, ints)


def test_smallest_scales_of_gate_and_up():
    """Their sums take the scale alone: x of 2^100 and up's scales of 2^-140."""
    c = _case(4, 4, 2, 256, 256, "e4m3-f32", seed=9)
    c["x"] = (c["x"].float() * 2.0 ** 100).to(torch.bfloat16)
    c["w_router"] = (c["w_router"].float() * 2.0 ** -100).to(torch.bfloat16)
    _scaled(c, 0, c["w"][0][1] * 2.0 ** -100)
    _scaled(c, 1, torch.tensor(3 * 2.0 ** -149, dtype=torch.float32))
    _scaled(c, 2, c["w"][2][1] * 2.0 ** 40)
    out, ints = _run(c)
    assert bool((out != 0).any())
    _check(c, out, ints)
