"""Norms and 8-bit products one after the other on a stream, with the buffers
between them rewritten with other values every time: each kernel may start
before the previous one ends, and must still read what that one wrote."""

import os
import re

import pytest
import torch

import norm_fp8_ref as ref
from causal_convolution_gb300 import api
from gpu_util import ensure_built

DEV = "cuda"
BF16, F8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_convolution_gb300", "csrc")


def test_kernels_that_start_early_read_with_ordinary_loads():
    # non-coherent loads are for data that nobody writes while the kernel lives
    for name in ("gemm_fp8.cu", "group_norm.cu", "rows.cu", "cc_rows.cuh"):
        code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        assert "__ldg" not in code and "ld.global.nc" not in code and ".nc." not in code, name


def rnd(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF16)


def chain(steps, out, between=None):
    """Each step: an input, a function of it."""
    for i, step in enumerate(steps):
        step(out[i])
        if between:
            between()


def compare(steps, shape):
    """The steps' outputs back to back, and from a graph, against one step at a time."""
    want, got = [[torch.zeros(shape, dtype=BF16, device=DEV) for _ in steps] for _ in range(2)]
    chain(steps, want, torch.cuda.synchronize)
    assert not any(torch.equal(want[0], w) for w in want[1:])
    for _ in range(5):
        for g in got:
            g.zero_()
        chain(steps, got)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(steps, got)
    for _ in range(5):
        for g in got:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    api.cc_check_device()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1, 512, 4096), (17, 1024, 2048), (64, 256, 1040), (100, 256, 4112), (300, 1024, 512),
                                   (2300, 520, 272)])
@pytest.mark.parametrize("norm", [False, True])
def test_products_behind_their_quantisation(m, n, k, norm):
    # one pair of buffers for the 8-bit rows and their scales, which change by powers of two from step to step
    ensure_built()
    wq, sw = torch.empty((n, k), dtype=F8, device=DEV), torch.empty((ref.blocks(n), ref.blocks(k)), device=DEV)
    api.cc_gemm_fp8_prepare(rnd((n, k), 1, k ** -0.5), wq, sw)
    y, s = torch.empty((m, k), dtype=F8, device=DEV), torch.empty((m, ref.blocks(k)), device=DEV)

    def step(i):
        x, gamma = rnd((m, k), 10 + i, 2.0 ** (i % 5 - 2)), rnd((k,), 40 + i)

        def run(out):
            if norm:
                api.cc_rms_norm_act_fp8(x, gamma, y, s)
            else:
                api.cc_fp8_quantize(x, y, s)
            api.cc_gemm_fp8(y, s, wq, sw, None, None, out)
        return run

    compare([step(i) for i in range(12)], (m, n))


@pytest.mark.gpu
@pytest.mark.parametrize("n,p,c,groups", [(1, 6000, 64, 2), (2, 705, 424, 8), (1, 40000, 128, 16), (2, 96, 64, 32)])
def test_group_norms_behind_a_product(n, p, c, groups):
    # the product writes what the norm reads, and its bias and the norm's gamma and beta are rewritten too
    ensure_built()
    k = 128
    wq, sw = torch.empty((c, k), dtype=F8, device=DEV), torch.empty((ref.blocks(c), 1), device=DEV)
    api.cc_gemm_fp8_prepare(rnd((c, k), 2, k ** -0.5), wq, sw)
    h = torch.empty((n, p, c), dtype=BF16, device=DEV)
    params = torch.empty((3, c), dtype=BF16, device=DEV)
    ws = torch.empty(api.cc_group_norm_workspace_bytes(n, p, c, groups), dtype=torch.uint8, device=DEV)

    def step(i):
        q, s = torch.empty((n, p, k), dtype=F8, device=DEV), torch.empty((n, p, 1), device=DEV)
        api.cc_fp8_quantize(rnd((n, p, k), 60 + i, 2.0 ** (i % 5 - 2)), q, s)
        of = rnd((3, c), 90 + i)

        def run(out):
            api.cc_rms_norm_act(of, None, params, act="none")
            api.cc_gemm_fp8(q, s, wq, sw, params[0], None, h)
            api.cc_group_norm_act(h, params[1], params[2], out, groups, ws)
        return run

    compare([step(i) for i in range(8)], (n, p, c))
