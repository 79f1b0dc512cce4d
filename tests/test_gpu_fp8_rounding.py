"""What the block quantisation does next to the middle of two e4m3 values: it
multiplies by the scale's reciprocal, rounded to fp32, as the header says. The
quotient by the scale would go to the other neighbour for these values."""

import pytest
import torch

from causal_convolution_gb300 import api
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn

# (largest |v| of the block, v, e4m3 of v * (1 / s), e4m3 of v / s)
NEAR_TIES = [(6.125, -3.171875, -240.0, -224.0), (6.125, -0.79296875, -60.0, -56.0), (8.625, -0.404296875, -22.0, -20.0),
             (8.625, 0.80859375, 44.0, 40.0), (4.75, -0.013916015625, -1.375, -1.25), (4.75, 0.111328125, 11.0, 10.0)]


def test_the_listed_values_tell_the_two_apart():
    for top, v, by_reciprocal, by_quotient in NEAR_TIES:
        s = torch.tensor(top) / torch.tensor(448.0)
        assert float((torch.tensor(v) * (1 / s)).to(F8)) == by_reciprocal
        assert float((torch.tensor(v) / s).to(F8)) == by_quotient


@pytest.mark.parametrize("at", [0, 5, 127])
def test_values_are_multiplied_by_the_rounded_reciprocal(at):
    ensure_built()
    n = len(NEAR_TIES)
    x = torch.zeros((n, 256), dtype=BF16, device=DEV)
    for i, (top, v, _, _) in enumerate(NEAR_TIES):
        x[i, 128 + at], x[i, 128 + (at + 9) % 128] = v, top
    want = torch.tensor([t[2] for t in NEAR_TIES], device=DEV)
    y, s = torch.empty((n, 256), dtype=F8, device=DEV), torch.empty((n, 2), device=DEV)
    api.cc_fp8_quantize(x, y, s)
    assert torch.equal(y[:, 128 + at].float(), want)
    for i in range(n):  # the same block as weights
        wq, sw = torch.empty((1, 256), dtype=F8, device=DEV), torch.empty((1, 2), device=DEV)
        api.cc_gemm_fp8_prepare(x[i:i + 1].contiguous(), wq, sw)
        assert float(wq[0, 128 + at].float()) == float(want[i]) and torch.equal(sw, s[i:i + 1])
    api.cc_check_device()
