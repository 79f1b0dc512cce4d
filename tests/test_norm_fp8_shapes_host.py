"""Shapes that the binding of the norms and the 8-bit product refuses, on the
host: tensors that hold the right number of elements under other sizes, and sizes
that a C int does not hold."""

import pytest
import torch

from causal_convolution_gb300 import _lib, api

BF16, F8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


class OnDevice(torch.Tensor):
    """A CPU tensor that says it lives on cuda:0."""

    is_cuda = True
    device = torch.device("cuda:0")

    def get_device(self):
        return 0


def t(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=F32).to(dtype).as_subclass(OnDevice)


class Calls:
    """Stands in for the library and takes down what it is called with."""

    def __init__(self):
        self.seen = []

    def __getattr__(self, name):
        def call(*args):
            self.seen.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    calls = Calls()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(api, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(_lib, "load", lambda: calls)
    return calls


def gemm(a, sa, out, res=None, n=16, k=256):
    api.cc_gemm_fp8(a, sa, t(n, k, dtype=F8), t((n + 127) // 128, (k + 127) // 128, dtype=F32), None, res, out)


def test_the_product_takes_rows_of_any_dimensions(calls):
    gemm(t(6, 256, dtype=F8), t(6, 2, dtype=F32), t(6, 16))
    gemm(t(2, 3, 256, dtype=F8), t(2, 3, 2, dtype=F32), t(2, 3, 16), t(2, 3, 16))
    gemm(t(256, dtype=F8), t(2, dtype=F32), t(16))
    gemm(t(0, 3, 256, dtype=F8), t(0, 3, 2, dtype=F32), t(0, 3, 16))
    assert [args[7:10] for _, args in calls.seen] == [(6, 16, 256), (6, 16, 256), (1, 16, 256), (0, 16, 256)]


@pytest.mark.parametrize("a,sa,out", [
    ((2, 3, 256), (2, 3, 2), (3, 2, 16)),   # rows in another order
    ((2, 3, 256), (3, 2, 2), (2, 3, 16)),   # their scales
    ((2, 3, 256), (2, 3, 2), (1, 6, 16)),
    ((6, 256), (6, 2), (2, 3, 16)),
    ((6, 256), (2, 3, 2), (6, 16)),
    ((6, 256), (6, 1), (6, 16)),
    ((6, 256), (5, 2), (6, 16)),
    ((5, 256), (5, 2), (6, 16)),
    ((3, 512), (3, 2), (6, 16)),            # as many elements, other rows
    ((0, 3, 256), (3, 0, 2), (0, 3, 16)),
    ((), (1,), (16,)),
])
def test_the_product_refuses_other_leading_sizes(calls, a, sa, out):
    with pytest.raises(ValueError, match="gemm_fp8"):
        gemm(t(*a, dtype=F8), t(*sa, dtype=F32), t(*out))
    assert not calls.seen


@pytest.mark.parametrize("x,scales", [
    ((2, 3, 256), (3, 2, 2)), ((2, 3, 256), (6, 2)), ((2, 3, 256), (1, 2, 3, 2)), ((2, 3, 256), (2, 3, 3)),
    ((2, 3, 256), (2, 2, 3)),
])
def test_scales_share_the_leading_sizes(calls, x, scales):
    x, y, s = t(*x), t(*x, dtype=F8), t(*scales, dtype=F32)
    with pytest.raises(ValueError, match="scales"):
        api.cc_fp8_quantize(x, y, s)
    with pytest.raises(ValueError, match="scales"):
        api.cc_rms_norm_act_fp8(x, None, y, s)
    with pytest.raises(ValueError, match="scales"):
        api.cc_group_norm_act_fp8(x, None, None, y, s, 8, None)
    assert not calls.seen


def test_scales_of_the_right_sizes_pass(calls):
    for shape in ((6, 200), (2, 3, 128), (2, 1, 1, 3, 136), (2, 0, 64)):
        x, y, s = t(*shape), t(*shape, dtype=F8), t(*shape[:-1], (shape[-1] + 127) // 128, dtype=F32)
        api.cc_fp8_quantize(x, y, s)
        api.cc_rms_norm_act_fp8(x, None, y, s)
        api.cc_group_norm_act_fp8(x, None, None, y, s, 8, None)
    assert len(calls.seen) == 12


INT = api.INT_MAX
BIG = (1 << 32) + 5  # as a C int: 5


def wide(rows, c, dtype=BF16):
    """A [rows, c] view of one row or one element: sizes only."""
    return t(1, 1, dtype=dtype).expand(rows, c) if c > INT else t(1, c, dtype=dtype).expand(rows, c)


@pytest.mark.parametrize("rows", [INT + 1, BIG])
def test_rows_beyond_an_int_are_refused(calls, rows):
    x, y8, s = wide(rows, 8), wide(rows, 8, F8), wide(rows, 1, F32)
    many = f"at most {INT}"
    with pytest.raises(ValueError, match=many):
        api.cc_rms_norm_act(x, None, x)
    with pytest.raises(ValueError, match=many):
        api.cc_rms_norm_act_fp8(x, None, y8, s)
    with pytest.raises(ValueError, match=many):
        api.cc_fp8_quantize(x, y8, s)
    with pytest.raises(ValueError, match=many):
        api.cc_gemm_fp8(wide(rows, 16, F8), s, t(8, 16, dtype=F8), t(1, 1, dtype=F32), None, None, x)
    with pytest.raises(ValueError, match=many):  # as instances and as positions
        api.cc_group_norm_act(x.unsqueeze(1), None, None, x.unsqueeze(1), 1, None)
    with pytest.raises(ValueError, match=many):
        api.cc_group_norm_act_fp8(x.unsqueeze(0), None, None, y8.unsqueeze(0), s.unsqueeze(0), 1, None)
    assert not calls.seen
    assert api.cc_group_norm_workspace_bytes(rows, 1, 8, 1) == api.cc_group_norm_workspace_bytes(1, rows, 8, 1) == 0
    assert api.cc_group_norm_workspace_bytes(1, 30000, 8, (1 << 32) + 1) == 0
    assert not calls.seen


def test_positions_are_counted_before_they_are_refused(calls):
    x = t(1, 1, 1, 8).expand(1, 1 << 16, 1 << 16, 8)  # 2^32 positions
    with pytest.raises(ValueError, match=f"at most {INT}"):
        api.cc_group_norm_act(x, None, None, x, 1, None)
    assert not calls.seen


def test_other_sizes_beyond_an_int_are_refused(calls):
    many = f"at most {INT}"
    x = t(2, 3, 8)
    for groups in ((1 << 32) + 8, -(1 << 32) + 8):
        with pytest.raises(ValueError, match=many):
            api.cc_group_norm_act(x, None, None, x, groups, None)
    for n, k in ((BIG + 11, 16), (16, BIG + 11)):
        w = wide(n, k)
        sw = t(1, 1, dtype=F32).expand((n + 127) // 128, (k + 127) // 128)
        with pytest.raises(ValueError, match=many):
            api.cc_gemm_fp8_prepare(w, w, sw)
    with pytest.raises(ValueError, match=many):
        api.cc_gemm_fp8(wide(1, k, F8), t(1, 1, dtype=F32).expand(1, (k + 127) // 128), wide(n, k, F8), sw, None, None,
                        t(1, n))
    assert not calls.seen
