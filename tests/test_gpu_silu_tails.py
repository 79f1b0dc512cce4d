"""SiLU far from zero: what is left of it below -87, and large values."""

import pytest
import torch

import norm_fp8_ref as ref
from causal_convolution_gb300 import api
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def values():
    steps = torch.arange(-130.0, 130.0, 0.5, device=DEV).to(BF16)
    far = torch.tensor([-3e38, -1e30, -1e5, 1e5, 1e30, 3e38, 0.0, -0.0], dtype=BF16, device=DEV)
    return torch.cat([steps, far])


@pytest.mark.parametrize("norm", ["rms", "group"])
def test_silu_of_values_far_from_zero(norm):
    # the norms' results are gamma or beta: rows of ones, or a constant instance
    ensure_built()
    v = values()
    c = v.numel()
    assert c % 8 == 0
    x = torch.ones((3, c), dtype=BF16, device=DEV)
    y = torch.empty_like(x)
    if norm == "rms":
        api.cc_rms_norm_act(x, v, y, eps=1e-12)  # 1 + 1e-12 is 1 in fp32
    else:
        ws = torch.empty(api.cc_group_norm_workspace_bytes(1, 3, c, 1), dtype=torch.uint8, device=DEV)
        api.cc_group_norm_act(x[None], None, v, y[None], 1, ws)
    api.cc_check_device()
    vd = v.double()
    want = (vd / (1 + torch.exp(-vd))).nan_to_num(nan=0.0)  # -3e38 / inf
    # two fast operations of 2^-21 each; the exponent v log2 e is rounded (2^-24 of it, and its constant less), which
    # the exponential passes on as |v| 2^-23 at most while it is not small beside 1; the flushed tail
    rel = 2.0 ** -19 + vd.clamp(max=0).abs() * 2.0 ** -23
    ref.assert_bf16(y, want.expand(3, c), (rel * want.abs() + 2.0 ** -119).expand(3, c), "silu")
    tail = (vd < -88) & (vd > -130)
    assert bool((y[:, tail] == 0).all()) and bool(torch.isfinite(y.float()).all())
