"""What the norm and 8-bit product entry points refuse, on the host: nothing
here reaches a device."""

import ctypes
import os

import pytest
import torch

from causal_convolution_gb300 import _lib, api

F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from causal_convolution_gb300 import build
        build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(1 << 12)
    p.keep = buf
    return (ctypes.addressof(buf) + 15) // 16 * 16


def test_group_norm_refusals(lib, p):
    gn, gn8 = lib.cc_group_norm_act, lib.cc_group_norm_act_fp8
    e = F(1e-6)
    big = 1 << 40
    assert gn(None, p, p, p, 1, 4, 64, 8, e, 0, p, big, None) == 1 and b"null" in lib.cc_last_error()
    assert gn(p, p, p, None, 1, 4, 64, 8, e, 0, p, big, None) == 1
    assert gn8(p, p, p, p, None, 1, 4, 64, 8, e, 0, p, big, None) == 1
    assert gn(p, p + 2, p, p, 1, 4, 64, 8, e, 0, p, big, None) == 1 and b"aligned" in lib.cc_last_error()
    assert gn8(p, p, p, p, p + 4, 1, 4, 64, 8, e, 0, p, big, None) == 1
    assert gn(p, p, p, p, 1, 4, 64, 7, e, 0, p, big, None) == 1 and b"divide" in lib.cc_last_error()
    assert gn(p, p, p, p, 1, 4, 64, 0, e, 0, p, big, None) == 1
    assert gn(p, p, p, p, 1, 4, 0, 1, e, 0, p, big, None) == 1
    assert gn(p, p, p, p, 1, 4, 12, 4, e, 0, p, big, None) == 2 and b"multiple of 8" in lib.cc_last_error()
    assert gn(p, p, p, p, 1, 4, 4104, 1, e, 0, p, big, None) == 2 and b"4096" in lib.cc_last_error()
    assert gn(p, p, p, p, 65536, 1, 64, 1, e, 0, p, big, None) == 2
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert gn(p, p, p, p, 1, 4, 64, 8, F(eps), 0, p, big, None) == 1 and b"eps" in lib.cc_last_error()
    assert gn(p, p, p, p, 1, 4, 64, 8, e, 2, p, big, None) == 1 and b"activation" in lib.cc_last_error()
    assert gn(p, p, p, p, 1, -4, 64, 8, e, 0, p, big, None) == 1 and b"negative" in lib.cc_last_error()


def test_group_norm_workspace(lib, p):
    need = lib.cc_group_norm_workspace_bytes(16, 219648, 256, 32)
    assert need > 0
    assert lib.cc_group_norm_act(p, p, p, p, 16, 219648, 256, 32, F(1e-6), 0, p, need - 1, None) == 1
    assert b"workspace" in lib.cc_last_error()
    assert lib.cc_group_norm_act(p, p, p, p, 16, 219648, 256, 32, F(1e-6), 0, None, need, None) == 1
    assert lib.cc_group_norm_workspace_bytes(0, 5, 64, 8) == 0
    assert lib.cc_group_norm_workspace_bytes(2, 0, 64, 8) == 0
    assert lib.cc_group_norm_workspace_bytes(-1, 5, 64, 8) == 0
    # clusters of CTAs keep the slabs, and need none ...
    for shape in ((2, 96, 64, 32), (4, 3432, 1024, 32), (5, 2000, 64, 2), (1, 2000, 64, 2)):
        assert lib.cc_group_norm_workspace_bytes(*shape) == 0, shape
    # ... and two readings take slabs that are too large, or few and long
    for shape in ((2, 30001, 64, 4), (16, 9000, 64, 2), (1, 5700, 64, 2), (1, 353, 792, 1)):
        assert lib.cc_group_norm_workspace_bytes(*shape) > 0, shape


def test_row_refusals(lib, p):
    e = F(1e-6)
    rms, rms8, quant = lib.cc_rms_norm_act, lib.cc_rms_norm_act_fp8, lib.cc_fp8_quantize
    assert rms(None, p, p, 4, 64, 64, e, 0, None) == 1 and rms(p, p, None, 4, 64, 64, e, 0, None) == 1
    assert rms8(p, p, p, None, 4, 64, 64, e, 0, None) == 1 and quant(p, p, None, 4, 64, 64, None) == 1
    assert rms(p, p + 8, p, 4, 64, 64, e, 0, None) == 1 and b"aligned" in lib.cc_last_error()
    assert rms(p, p, p, 4, 60, 64, e, 0, None) == 2 and b"multiple of 8" in lib.cc_last_error()
    assert rms(p, p, p, 4, 16392, 16392, e, 0, None) == 2 and quant(p, p, p, 4, 16392, 16392, None) == 2
    assert rms(p, p, p, 4, 64, 56, e, 0, None) == 1 and quant(p, p, p, 4, 64, 68, None) == 1
    assert rms(p, p, p, 4, 64, 64, F(0.0), 0, None) == 1 and rms(p, p, p, 4, 64, 64, e, -1, None) == 1
    assert rms(p, p, p, -1, 64, 64, e, 0, None) == 1 and quant(p, p, p, 4, 0, 64, None) == 1


def test_gemm_refusals(lib, p):
    g = lib.cc_gemm_fp8
    for i in (0, 1, 2, 3, 6):
        ptrs = [p, p, p, p, p, p, p]
        ptrs[i] = None
        assert g(*ptrs, 4, 64, 128, 64, 64, None) == 1 and b"null" in lib.cc_last_error()
    for i in range(7):
        ptrs = [p, p, p, p, p, p, p]
        ptrs[i] = p + 4
        assert g(*ptrs, 4, 64, 128, 64, 64, None) == 1 and b"aligned" in lib.cc_last_error()
    assert g(p, p, p, p, p, p, p, 4, 64, 120, 64, 64, None) == 2 and b"multiple of 16" in lib.cc_last_error()
    assert g(p, p, p, p, p, p, p, 4, 60, 128, 64, 64, None) == 2 and b"multiple of 8" in lib.cc_last_error()
    assert g(p, p, p, p, p, p, p, 4, 64, 128, 64, 56, None) == 1 and g(p, p, p, p, p, p, p, 4, 64, 128, 60, 64, None) == 1
    assert g(p, p, p, p, p, p, p, 4, 0, 128, 64, 64, None) == 1 and g(p, p, p, p, p, p, p, 4, 64, 0, 64, 64, None) == 1
    assert g(p, p, p, p, p, p, p, -4, 64, 128, 64, 64, None) == 1
    prep = lib.cc_gemm_fp8_prepare
    assert prep(None, p, p, 64, 64, None) == 1 and prep(p, p, p, 0, 64, None) == 1
    assert prep(p, p, p + 4, 64, 64, None) == 1 and prep(p, p, p, 64, 72, None) == 2


def test_sizes_beyond_the_kernels_indexes(lib, p):
    g, prep = lib.cc_gemm_fp8, lib.cc_gemm_fp8_prepare
    big = (1 << 24) + 16
    assert g(p, p, p, p, p, p, p, (1 << 31) - 1, 64, 128, 64, 64, None) == 2 and b"too many" in lib.cc_last_error()
    assert g(p, p, p, p, p, p, p, 4, big, 128, big, big, None) == 2
    assert g(p, p, p, p, p, p, p, 4, 64, big, 64, 64, None) == 2
    assert prep(p, p, p, 8388481, 64, None) == 2 and prep(p, p, p, 64, big, None) == 2
    assert lib.cc_group_norm_act(p, p, p, p, 1, (1 << 30) + 1, 64, 8, F(1e-6), 0, p, 1 << 60, None) == 2
    assert lib.cc_group_norm_workspace_bytes(65536, 5, 64, 8) == 0


def test_empty_requests(lib):
    e = F(1e-6)
    assert lib.cc_group_norm_act(None, None, None, None, 0, 4, 64, 8, e, 0, None, 0, None) == 0
    assert lib.cc_group_norm_act(None, None, None, None, 3, 0, 64, 8, e, 0, None, 0, None) == 0
    assert lib.cc_group_norm_act_fp8(None, None, None, None, None, 0, 4, 64, 8, e, 0, None, 0, None) == 0
    assert lib.cc_rms_norm_act(None, None, None, 0, 64, 64, e, 0, None) == 0
    assert lib.cc_rms_norm_act_fp8(None, None, None, None, 0, 64, 64, e, 0, None) == 0
    assert lib.cc_fp8_quantize(None, None, None, 0, 64, 64, None) == 0
    assert lib.cc_gemm_fp8(None, None, None, None, None, None, None, 0, 64, 128, 64, 64, None) == 0


def test_the_binding_refuses_what_it_cannot_pass_on(lib, monkeypatch):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    f8 = torch.zeros(4, 64).to(torch.float8_e4m3fn)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(api, "_raw_stream", lambda stream, dev: 0)
    with pytest.raises(ValueError, match="CUDA"):
        api.cc_rms_norm_act(x, None, torch.empty_like(x))
    with pytest.raises(ValueError, match="CUDA"):
        api.cc_group_norm_act(x, None, None, torch.empty_like(x), 8, None)
    with pytest.raises(ValueError, match="share"):
        api.cc_group_norm_act(x, None, None, x[:2], 8, None)
    with pytest.raises(ValueError, match="C elements"):
        api.cc_group_norm_act(x, x[0, :8], None, x, 8, None)
    with pytest.raises(ValueError, match="sw"):
        api.cc_gemm_fp8_prepare(x, f8, torch.zeros(2, 1))
    with pytest.raises(ValueError, match="act"):
        api._act("relu")


def test_rows_at_one_stride():
    t = torch.zeros(2, 5, 48, dtype=torch.bfloat16)

    def layout(v):
        return api._row_layout(v, "t")

    assert layout(t) == (10, 48, 48)
    assert layout(t[..., 16:32]) == (10, 16, 48)
    assert layout(t[:1, 2:4, :8]) == (2, 8, 48)
    assert layout(t[0, 0]) == (1, 48, 48)
    assert layout(t[:0]) == (0, 48, 48)
    with pytest.raises(ValueError, match="one stride"):
        layout(t[:, :3, :8])
    with pytest.raises(ValueError, match="contiguous"):
        layout(t.transpose(1, 2))


def test_tensors_on_another_device_are_refused():
    class Elsewhere(torch.Tensor):  # a CPU tensor that says it lives on cuda:1
        is_cuda = True
        device = torch.device("cuda:1")

        def get_device(self):
            return 1

    t = torch.zeros(4, 64, dtype=torch.bfloat16).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        api._arg(t, torch.bfloat16, "x", 0)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        api._last_rows(t, torch.bfloat16, "x", 0)
    assert api._arg(t, torch.bfloat16, "x", 1) == t.data_ptr()
