"""Norms with an activation, block quantisation and the 8-bit product against
plain 64-bit forms: small and odd sizes, rows at a stride, offsets, NaN and
infinity, guard bands, and a run of them together as they are used around the
attention."""

import pytest
import torch

import norm_fp8_ref as ref
from causal_convolution_gb300 import api
from gpu_util import ensure_built
from test_gpu_guard_bands import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    # a tensor: torch divides by a Python number with its rounded reciprocal, one step away from the quotient
    globals()["E4M3_MAX"] = torch.tensor(448.0, device=DEV)
    return ensure_built()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rnd(shape, seed, scale=1.0, offset=0.0):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * scale + offset).to(BF16)


def rnd_f8(shape, seed):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * 100).clamp(-448, 448).to(F8)


def rnd_scales(shape, seed):
    return torch.rand(shape, generator=gen(seed), device=DEV) * 0.02 + 0.001


class GuardedF8:
    """Guarded, for e4m3 (a byte tensor seen as e4m3)."""

    def __init__(self, shape):
        self.g = Guarded(shape, torch.uint8)
        self.t = self.g.t.view(F8)

    def bands_intact(self):
        return self.g.bands_intact()


def group_norm(x, gamma, beta, groups, act, fp8, eps=1e-6):
    """One guarded call; (y,) or (y, scales)."""
    n, c = x.shape[0], x.shape[-1]
    p = x.numel() // max(1, n * c)
    ws = Guarded((api.cc_group_norm_workspace_bytes(n, p, c, groups),), torch.uint8)
    before = x.clone()
    if fp8:
        y, s = GuardedF8(x.shape), Guarded((*x.shape[:-1], ref.blocks(c)), F32)
        api.cc_group_norm_act_fp8(x, gamma, beta, y.t, s.t, groups, ws.t, eps=eps, act=act)
    else:
        y, s = Guarded(x.shape), None
        api.cc_group_norm_act(x, gamma, beta, y.t, groups, ws.t, eps=eps, act=act)
    api.cc_check_device()
    assert torch.equal(x.view(torch.int16), before.view(torch.int16))
    for g in (ws, y, s):
        assert g is None or g.bands_intact()
    return (y.t, s.t) if fp8 else (y.t,)


def check_group_norm(x, gamma, beta, groups, act, fp8, what):
    want, bound = ref.group_norm(x, gamma, beta, groups, 1e-6, act)
    got = group_norm(x, gamma, beta, groups, act, fp8)
    (ref.assert_fp8 if fp8 else ref.assert_bf16)(*got, want, bound, what)


GN_SHAPES = [  # n, p, c, groups
    (1, 1, 8, 1), (1, 1, 8, 8), (1, 1, 64, 8), (2, 96, 64, 32), (3, 17, 480, 32), (2, 33, 120, 8), (1, 5, 4096, 1),
    (2, 3, 4088, 7), (1, 3432, 1024, 32), (2, 700, 256, 256), (1, 2, 136, 17), (5, 64, 128, 4), (3, 1, 2048, 16),
    (1, 4001, 96, 32), (4, 130, 512, 32), (7, 11, 1032, 1), (1, 13728, 128, 32), (2, 20011, 64, 2), (1, 9000, 640, 1),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("n,p,c,groups", GN_SHAPES)
def test_group_norm_matches_64_bits(n, p, c, groups, act, fp8):
    x = rnd((n, p, c), 1 + p, 1.5, 0.25) * rnd((c,), 2).abs()
    check_group_norm(x, 1 + rnd((c,), 3, 0.3), rnd((c,), 4, 0.3), groups, act, fp8, f"{(n, p, c, groups)}")


@pytest.mark.parametrize("fp8", [False, True])
def test_group_norm_large_instances(fp8):
    # instances beyond what one cluster of CTAs keeps on chip, and several of them
    x = rnd((3, 60011, 256), 5, 1.0, 0.5)
    check_group_norm(x, rnd((256,), 6), rnd((256,), 7), 32, "silu", fp8, "large")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,p,c,groups", [(2, 60001, 136, 17), (1, 70000, 200, 100), (1, 33000, 1000, 8)])
def test_group_norm_large_instances_with_uneven_slabs(n, p, c, groups, fp8):
    x = rnd((n, p, c), 24, 1.0, 0.5)
    check_group_norm(x, rnd((c,), 25), rnd((c,), 26), groups, "silu", fp8, f"{(n, p, c, groups)}")


@pytest.mark.parametrize("n,p,c,groups,fp8", [
    (2, 219648, 64, 8, False),   # 32 channels to a slab on all SMs
    (1, 120000, 192, 3, True),   # two readings: 128 channels are too many for the SMs
    (2, 60007, 264, 1, False),   # two readings, one group of everything
    (1, 100003, 72, 9, True),    # a slab of 72 channels, padded to 128
    (3, 40009, 328, 41, False),  # the last slab is narrower
    (1, 600000, 64, 32, False),  # a frame beyond the SMs' shared memory
    (1, 3001, 4096, 1, True), (1, 70001, 8, 2, False), (1, 300000, 8, 8, False),
])
def test_group_norm_of_large_frames(n, p, c, groups, fp8):
    x = rnd((n, p, c), 27, 1.0, -0.5)
    check_group_norm(x, rnd((c,), 28), rnd((c,), 29), groups, "silu", fp8, f"{(n, p, c, groups)}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,p,c,groups", [
    (1, 3840, 64, 2), (1, 5700, 64, 2), (4, 5800, 64, 2), (5, 5800, 64, 2),  # few slabs: clusters or all SMs
    (2, 1600, 208, 1), (2, 705, 424, 8), (1, 353, 792, 1), (1, 50, 4096, 1), (3, 21, 4096, 2),
    (15, 9000, 64, 2), (16, 9000, 64, 2), (16, 6500, 64, 2),                 # many: clusters of one or two CTAs to an SM
    (1, 17253, 112, 2), (2, 29001, 64, 4), (2, 30001, 64, 4),                # about as much as eight SMs hold
])
def test_group_norm_on_both_sides_of_the_choice_of_kernel(n, p, c, groups, fp8):
    x = rnd((n, p, c), 90 + p, 1.0, 0.5)
    check_group_norm(x, 1 + rnd((c,), 91, 0.3), rnd((c,), 92, 0.3), groups, "silu", fp8, f"{(n, p, c, groups)}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,p,c,groups", [  # clusters of four to eight CTAs, some with a short or an empty last share
    (12, 1001, 128, 4), (16, 1500, 128, 32), (20, 1001, 64, 2), (24, 997, 120, 8), (28, 700, 64, 2), (34, 501, 120, 8),
    (40, 1300, 64, 4), (16, 13, 4096, 1), (17, 16, 4096, 1), (29, 9, 4096, 1), (3, 911, 1000, 25), (2, 1717, 1024, 32),
    (80, 1501, 64, 2), (150, 601, 64, 8), (60, 1499, 128, 4), (75, 1497, 120, 8), (120, 401, 64, 8), (300, 400, 64, 2),
])
def test_group_norm_by_many_clusters(n, p, c, groups, fp8):
    x = rnd((n, p, c), 190 + n, 1.0, -0.5)
    check_group_norm(x, 1 + rnd((c,), 191, 0.3), rnd((c,), 192, 0.3), groups, "silu", fp8, f"{(n, p, c, groups)}")


def test_group_norm_of_large_frames_replays_from_a_graph():
    for n, p, c, groups in ((3, 60000, 128, 16), (1, 200000, 256, 1)):
        x, y = rnd((n, p, c), 30), torch.empty((n, p, c), dtype=BF16, device=DEV)
        ws = torch.empty(api.cc_group_norm_workspace_bytes(n, p, c, groups), dtype=torch.uint8, device=DEV)
        api.cc_group_norm_act(x, None, None, y, groups, ws)
        torch.cuda.synchronize()
        eager = y.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(2):
                api.cc_group_norm_act(x, None, None, y, groups, ws)
        for _ in range(3):
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, eager)
        api.cc_check_device()


def test_large_group_norms_on_two_streams_at_once():
    # both want every SM: the second waits for the first, neither for parts of the other
    x = [rnd((4, 60000, 128), 31 + i) for i in range(2)]
    ws = [torch.empty(api.cc_group_norm_workspace_bytes(4, 60000, 128, 16), dtype=torch.uint8, device=DEV)
          for _ in range(2)]
    y = [torch.empty_like(v) for v in x]
    for i in range(2):
        api.cc_group_norm_act(x[i], None, None, y[i], 16, ws[i])
    torch.cuda.synchronize()
    want = [v.clone() for v in y]
    for v in y:
        v.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            api.cc_group_norm_act(x[i], None, None, y[i], 16, ws[i], stream=streams[i])
    torch.cuda.synchronize()
    api.cc_check_device()
    assert all(torch.equal(v, w) for v, w in zip(y, want))


def test_group_norm_without_gamma_and_beta():
    x = rnd((2, 50, 64), 8)
    check_group_norm(x, None, None, 4, "none", False, "plain")
    check_group_norm(x, rnd((64,), 9), None, 4, "silu", True, "gamma only")
    check_group_norm(x, None, rnd((64,), 10), 4, "silu", False, "beta only")


def test_group_norm_of_a_constant_is_beta():
    x = torch.full((2, 40, 64), 3.25, dtype=BF16, device=DEV)
    beta = rnd((64,), 11)
    (y,) = group_norm(x, rnd((64,), 12), beta, 8, "none", False)
    assert torch.equal(y, beta.expand(2, 40, 64))


@pytest.mark.parametrize("offset", [64.0, -1000.0])
def test_group_norm_with_a_mean_far_from_zero(offset):
    # sum(x^2) - n mean^2 in fp32 would keep few digits of the variance here
    x = rnd((2, 3000, 128), 13, 1.0, offset)
    check_group_norm(x, rnd((128,), 14), rnd((128,), 15), 8, "none", False, f"offset {offset}")


def test_group_norm_with_an_outlier_in_front():
    x = rnd((1, 5000, 64), 16)
    x[0, 0] = 1000.0
    check_group_norm(x, rnd((64,), 17), rnd((64,), 18), 4, "none", False, "outlier")


def test_group_norm_keeps_nan_and_infinity_inside_their_group():
    x = rnd((2, 100, 64), 19)
    x[0, 7, 3] = float("nan")      # group 0 of instance 0
    x[1, 99, 17] = float("inf")    # group 1 of instance 1 (cpg 16)
    (y,) = group_norm(x, None, None, 4, "silu", False)
    bad = torch.zeros(2, 100, 64, dtype=torch.bool, device=DEV)
    bad[0, :, :16] = True
    bad[1, :, 16:32] = True
    assert bool(torch.isnan(y[bad]).all()) and bool(torch.isfinite(y[~bad]).all())
    x0 = torch.where(bad, torch.zeros_like(x), x)
    want, bound = ref.group_norm(x0, None, None, 4, 1e-6, "silu")
    ref.assert_bf16(y[~bad], want[~bad], bound[~bad], "the other groups")
    _, s = group_norm(x, None, None, 4, "none", True)
    assert bool(torch.isnan(s[0]).all()) and bool(torch.isnan(s[1]).all())  # one block of 128 covers all 64 channels


def test_group_norm_is_the_same_every_time():
    x, g, b = rnd((2, 60000, 256), 20), rnd((256,), 21), rnd((256,), 22)
    first = group_norm(x, g, b, 32, "silu", False)[0].clone()
    for _ in range(5):
        assert torch.equal(group_norm(x, g, b, 32, "silu", False)[0], first)


def test_group_norm_of_many_small_instances():
    x = rnd((3001, 5, 72), 24, 2.0, 1.0)
    check_group_norm(x, rnd((72,), 25), rnd((72,), 26), 9, "silu", False, "3001 instances")
    check_group_norm(x, rnd((72,), 25), rnd((72,), 26), 3, "none", True, "3001 instances, e4m3")


def test_group_norm_one_value_to_a_group():
    # the variance of one value is 0: everything is beta
    x, beta = rnd((4, 1, 64), 27), rnd((64,), 28)
    (y,) = group_norm(x, rnd((64,), 29), beta, 64, "none", False)
    assert torch.equal(y, beta.expand(4, 1, 64))


def test_empty_tensors():
    e = torch.empty
    api.cc_group_norm_act(e((0, 5, 64), dtype=BF16, device=DEV), None, None, e((0, 5, 64), dtype=BF16, device=DEV), 8,
                          None)
    api.cc_group_norm_act_fp8(e((2, 0, 64), dtype=BF16, device=DEV), None, None, e((2, 0, 64), dtype=F8, device=DEV),
                              e((2, 0, 1), device=DEV), 8, None)
    api.cc_rms_norm_act(e((0, 64), dtype=BF16, device=DEV), None, e((0, 64), dtype=BF16, device=DEV))
    api.cc_fp8_quantize(e((0, 3, 64), dtype=BF16, device=DEV), e((0, 3, 64), dtype=F8, device=DEV),
                        e((0, 3, 1), device=DEV))
    api.cc_gemm_fp8(e((0, 64), dtype=F8, device=DEV), e((0, 1), device=DEV), rnd_f8((128, 64), 30),
                    rnd_scales((1, 1), 31), None, None, e((0, 128), dtype=BF16, device=DEV))
    api.cc_check_device()


def test_group_norm_of_video_frames():
    # [N, D, H, W, C] normalised per frame
    x = rnd((2, 3, 6, 7, 64), 23)
    y = torch.empty_like(x)
    ws = torch.empty(api.cc_group_norm_workspace_bytes(6, 42, 64, 32), dtype=torch.uint8, device=DEV)
    api.cc_group_norm_act(x.view(6, 6, 7, 64), None, None, y.view(6, 6, 7, 64), 32, ws)
    for i in range(2):
        for d in range(3):
            want, bound = ref.group_norm(x[i, d][None], None, None, 32, 1e-6, "silu")
            ref.assert_bf16(y[i, d][None], want, bound, f"frame {i} {d}")


# ---------------------------------------------------------------------- rows --

ROW_SHAPES = [(1, 8), (1, 128), (3, 136), (17, 2048), (1000, 512), (5, 1000), (2, 16384), (33, 64), (257, 1024),
              (4, 4104), (70000, 16), (129, 256), (9, 6000)]


def strided_rows(rows, c, seed, pad):
    """rows x c, `pad` unused channels behind each row"""
    return rnd((rows, c + pad), seed, 1.5)[:, :c]


@pytest.mark.parametrize("pad", [0, 24])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("rows,c", ROW_SHAPES)
def test_rms_norm_matches_64_bits(rows, c, act, fp8, pad):
    x, gamma = strided_rows(rows, c, rows, pad), rnd((c,), 31, 0.5, 1.0)
    want, bound = ref.rms_norm(x, gamma, 1e-6, act)
    if fp8:
        y, s = GuardedF8((rows, c)), Guarded((rows, ref.blocks(c)), F32)
        api.cc_rms_norm_act_fp8(x, gamma, y.t, s.t, act=act)
        api.cc_check_device()
        assert s.bands_intact()
        ref.assert_fp8(y.t, s.t, want, bound, f"{rows}x{c}")
    else:
        y = Guarded((rows, c))
        api.cc_rms_norm_act(x, gamma, y.t, act=act)
        api.cc_check_device()
        ref.assert_bf16(y.t, want, bound, f"{rows}x{c}")
    assert y.bands_intact()


def test_rms_norm_of_zeros_and_without_gamma():
    x = torch.zeros((4, 64), dtype=BF16, device=DEV)
    x[2] = rnd((64,), 32)
    y = torch.empty_like(x)
    api.cc_rms_norm_act(x, None, y, eps=1e-12, act="none")
    assert bool((y[[0, 1, 3]] == 0).all())
    ref.assert_bf16(y, *ref.rms_norm(x, None, 1e-12, "none"), "row 2")
    x[1, 5], x[3, 0] = float("nan"), float("inf")
    api.cc_rms_norm_act(x, None, y, act="none")
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[3, 0])) and bool((y[3, 1:] == 0).all())
    assert bool((y[0] == 0).all()) and bool(torch.isfinite(y[2].float()).all())


@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("rows,c", ROW_SHAPES)
def test_quantize_matches_its_definition_bit_by_bit(rows, c, pad):
    x = strided_rows(rows, c, 40 + rows, pad) * torch.logspace(-3, 3, rows, device=DEV).to(BF16)[:, None]
    y, s = GuardedF8((rows, c)), Guarded((rows, ref.blocks(c)), F32)
    api.cc_fp8_quantize(x, y.t, s.t)
    api.cc_check_device()
    assert y.bands_intact() and s.bands_intact()
    xf = torch.cat([x.float(), torch.zeros(rows, ref.blocks(c) * 128 - c, device=DEV)], 1).view(rows, -1, 128)
    scale = (xf.abs().amax(-1) / E4M3_MAX).clamp(min=2.0 ** -126)
    want = (xf * (1 / scale)[..., None]).view(rows, -1)[:, :c].to(F8)
    assert torch.equal(s.t, scale)
    assert torch.equal(y.t.view(torch.uint8), want.contiguous().view(torch.uint8))


# four vectors to a lane, rows cut into pieces, a row to a CTA, and more rows than are taken at once
MORE_ROW_SHAPES = [(4001, 616), (7, 520), (3001, 1160), (2600, 1536), (5, 1288), (1, 2056), (6001, 1032), (700, 5128)]


@pytest.mark.parametrize("rows,c", MORE_ROW_SHAPES)
def test_quantize_of_wide_rows(rows, c):
    test_quantize_matches_its_definition_bit_by_bit(rows, c, 8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,c", MORE_ROW_SHAPES)
def test_rms_norm_of_wide_rows(rows, c, fp8):
    test_rms_norm_matches_64_bits(rows, c, "silu", fp8, 8)


def test_quantize_of_zeros_tiny_values_nan_and_infinity():
    x = torch.zeros((5, 256), dtype=BF16, device=DEV)
    x[1, :128] = 1e-38
    x[2, 0], x[3, 200] = float("nan"), float("inf")
    x[3, 201] = 5.0
    x[4] = 3.0e38
    y = torch.empty((5, 256), dtype=F8, device=DEV)
    s = torch.empty((5, 2), device=DEV)
    api.cc_fp8_quantize(x, y, s)
    yf = y.float()
    assert bool((s[0] == 2.0 ** -126).all()) and bool((yf[0] == 0).all())
    assert bool((yf[1, :128] == 0.875).all()) and float(s[1, 0]) == 2.0 ** -126  # 1e-38 in bf16 / 2^-126, rounded
    assert bool(torch.isnan(s[2, 0])) and bool(torch.isnan(yf[2, :128]).all()) and bool((yf[2, 128:] == 0).all())
    assert float(s[3, 1]) == float("inf") and bool(torch.isnan(yf[3, 200])) and float(yf[3, 201]) == 0
    assert bool((yf[4] == 448).all())


@pytest.mark.parametrize("n,k", [(1, 16), (128, 128), (130, 144), (8, 1040), (1000, 64), (256, 4096)])
def test_prepared_weights(n, k):
    w = rnd((n, k), 50 + n, 0.05) * torch.logspace(-2, 2, n, device=DEV).to(BF16)[:, None]
    wq, sw = GuardedF8((n, k)), Guarded((ref.blocks(n), ref.blocks(k)), F32)
    api.cc_gemm_fp8_prepare(w, wq.t, sw.t)
    api.cc_check_device()
    assert wq.bands_intact() and sw.bands_intact()
    for i in range(ref.blocks(n)):
        for j in range(ref.blocks(k)):
            part = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
            scale = (w[part].float().abs().max() / E4M3_MAX).clamp(min=2.0 ** -126)
            assert float(sw.t[i, j]) == float(scale)
            want = (w[part].float() * (1 / scale)).to(F8)
            assert torch.equal(wq.t[part].float(), want.float())


# ------------------------------------------------------------------- product --

def gemm(a, sa, wq, sw, bias, res, ld_pad=0):
    m, n = a.shape[0], wq.shape[0]
    out = Guarded((m, n + ld_pad))
    api.cc_gemm_fp8(a, sa, wq, sw, bias, res, out.t[:, :n])
    api.cc_check_device()
    assert out.bands_intact()
    if ld_pad:
        assert out.untouched(out.t[:, n:])
    return out.t[:, :n]


def check_gemm(got, a, sa, wq, sw, bias, res, what):
    """One rounding to bf16; fp32 sums of exact products: each of the K / 32 steps of the tensor core, the scale's
    multiplication and the sum over blocks rounds (or truncates: a whole 2^-23) relative to the magnitudes so far."""
    want, size = ref.gemm(a, sa, wq, sw, bias, res)
    ref.assert_bf16(got, want, (a.shape[1] / 32 + 8) * 2.0 ** -23 * size, what)


GEMM_SHAPES = [  # m, n, k
    (1, 8, 16), (1, 4096, 4096), (7, 1024, 2048), (16, 256, 128), (17, 264, 144), (33, 136, 400), (64, 512, 512),
    (65, 1000, 784), (128, 128, 128), (129, 130 * 8, 272), (200, 1024, 1024), (257, 264, 1040), (300, 8, 64),
    (1000, 256, 512), (3432, 1024, 1024), (5000, 520, 256), (2, 2048, 16), (100, 4096, 4096), (777, 776, 784),
]


@pytest.mark.parametrize("extras", ["none", "bias", "both"])
@pytest.mark.parametrize("m,n,k", GEMM_SHAPES)
def test_gemm_matches_64_bits(m, n, k, extras):
    a, sa = rnd_f8((m, k), 60 + m), rnd_scales((m, ref.blocks(k)), 61)
    wq, sw = rnd_f8((n, k), 62 + n), rnd_scales((ref.blocks(n), ref.blocks(k)), 63)
    bias = rnd((n,), 64, 20.0) if extras != "none" else None
    res = rnd((m, n), 65, 20.0) if extras == "both" else None
    check_gemm(gemm(a, sa, wq, sw, bias, res), a, sa, wq, sw, bias, res, f"{m}x{n}x{k} {extras}")


@pytest.mark.parametrize("m,n,k", [
    (20001, 520, 272),   # several tiles to a CTA pair, an odd number of blocks of K
    (19999, 264, 1280),  # ten blocks: fours and a rest
    (30000, 136, 16),    # one block, half of every tile empty
    (3, 128, 16384),     # few rows, more blocks of K than stages
    (40, 136, 66000),    # few rows, too many scales to stage: the pairs' kernel
    (64, 1000, 16), (33, 8, 5008),
])
def test_gemm_walks_many_tiles_and_blocks(m, n, k):
    a, sa = rnd_f8((m, k), 160 + m), rnd_scales((m, ref.blocks(k)), 161)
    wq, sw = rnd_f8((n, k), 162 + n), rnd_scales((ref.blocks(n), ref.blocks(k)), 163)
    bias, res = rnd((n,), 164, 20.0), rnd((m, n), 165, 20.0)
    first = gemm(a, sa, wq, sw, bias, res).clone()
    check_gemm(first, a, sa, wq, sw, bias, res, f"{m}x{n}x{k}")
    for _ in range(3):
        assert torch.equal(gemm(a, sa, wq, sw, bias, res), first)  # the sums' order is fixed


@pytest.mark.parametrize("m,n,k", [
    (2300, 1800, 656), (2200, 1800, 1040), (40000, 504, 400),  # tiles of 256 columns
    (4097, 1096, 144), (2310, 2040, 1040), (66, 136, 4096), (300, 200, 272),  # of 128
    (700, 1000, 2064), (20000, 72, 144), (65, 8, 16),
    (64, 12296, 272), (33, 8200, 1040), (50, 4104, 2064), (64, 1032, 4112), (17, 4096, 4112), (3, 4104, 1040),  # splits of K
])
def test_gemm_on_both_sides_of_the_choice_of_tiles(m, n, k):
    test_gemm_matches_64_bits(m, n, k, "both")
    test_gemm_matches_64_bits(m, n, k, "none")


# few tiles and long K, whose blocks are divided among pairs of CTAs: evenly, with a short or an empty last share
SPLIT_SHAPES = [(66, 136, 4096), (100, 1000, 5136), (400, 1656, 4112), (129, 8, 9232), (65, 264, 3088),
                (200, 128, 2704), (1039, 120, 1584), (128, 4096, 4096), (513, 72, 16384)]


@pytest.mark.parametrize("m,n,k", SPLIT_SHAPES)
def test_gemm_with_divided_sums(m, n, k):
    for extras in ("none", "bias", "both"):
        test_gemm_matches_64_bits(m, n, k, extras)
    a, sa = rnd_f8((m, k), 170 + m), rnd_scales((m, ref.blocks(k)), 171)
    wq, sw = rnd_f8((n, k), 172 + n), rnd_scales((ref.blocks(n), ref.blocks(k)), 173)
    res = rnd((m, n + 40), 174, 20.0)[:, 8:8 + n]
    first = gemm(a, sa, wq, sw, None, res, ld_pad=24).clone()
    check_gemm(first, a, sa, wq, sw, None, res, f"strided {m}x{n}x{k}")
    io = res.contiguous()
    for _ in range(3):  # in place, and the same every time
        io.copy_(res)
        api.cc_gemm_fp8(a, sa, wq, sw, None, io, io)
        assert torch.equal(io, first)
    api.cc_check_device()


@pytest.mark.parametrize("m", [1, 40, 300])
def test_gemm_with_strided_rows(m):
    # out and res as column slices of wider rows (packed q, k, v)
    n, k = 136, 256
    a, sa = rnd_f8((m, k), 70), rnd_scales((m, 2), 71)
    wq, sw = rnd_f8((n, k), 72), rnd_scales((2, 2), 73)
    res = rnd((m, n + 40), 74, 20.0)[:, 8:8 + n]
    check_gemm(gemm(a, sa, wq, sw, None, res, ld_pad=24), a, sa, wq, sw, None, res, f"strided {m}")


@pytest.mark.parametrize("m", [3, 150, 1000])
def test_gemm_into_its_own_residual(m):
    n, k = 264, 400
    a, sa = rnd_f8((m, k), 75), rnd_scales((m, 4), 76)
    wq, sw = rnd_f8((n, k), 77), rnd_scales((3, 4), 78)
    res = rnd((m, n), 79, 20.0)
    io = res.clone()
    api.cc_gemm_fp8(a, sa, wq, sw, None, io, io)
    api.cc_check_device()
    check_gemm(io, a, sa, wq, sw, None, res, f"in place {m}")


@pytest.mark.parametrize("m,n,k", [(1, 128, 512), (50, 264, 384), (700, 520, 2048)])
def test_gemm_of_small_integers_is_exact(m, n, k):
    # every product and partial sum is an integer below 2^24 and every scale a power of two: fp32 loses nothing
    a = torch.randint(-8, 9, (m, k), generator=gen(80), device=DEV).float().to(F8)
    wq = torch.randint(-8, 9, (n, k), generator=gen(81), device=DEV).float().to(F8)
    sa = torch.exp2(torch.randint(0, 3, (m, ref.blocks(k)), generator=gen(82), device=DEV).float())
    sw = torch.exp2(torch.randint(0, 3, (ref.blocks(n), ref.blocks(k)), generator=gen(83), device=DEV).float())
    want, _ = ref.gemm(a, sa, wq, sw, None, None)
    assert torch.equal(gemm(a, sa, wq, sw, None, None), want.float().to(BF16))


@pytest.mark.parametrize("m", [4, 500])
def test_gemm_keeps_nan_and_infinity_in_their_rows(m):
    n, k = 256, 384
    a, sa = rnd_f8((m, k), 84), rnd_scales((m, 3), 85)
    wq, sw = rnd_f8((n, k), 86), rnd_scales((2, 3), 87)
    clean = gemm(a, sa, wq, sw, None, None).clone()
    a.view(torch.uint8)[1, 200] = 0x7F  # NaN
    sa[3, 1] = float("inf")
    out = gemm(a, sa, wq, sw, None, None)
    assert bool(torch.isnan(out[1]).all()) and not bool(torch.isfinite(out[3].float()).any())
    keep = [i for i in range(m) if i not in (1, 3)]
    assert torch.equal(out[keep], clean[keep])


# ------------------------------------------------------------------ together --

def attention_block(t, hw, c, seed):
    """The mid block's attention as a decoder runs it: norm -> e4m3 -> q, k, v -> attention -> e4m3 -> projection
    plus the residual."""
    x = rnd((t, hw, c), seed)
    gamma, beta = rnd((c,), seed + 1, 0.2, 1.0), rnd((c,), seed + 2, 0.2)
    w = [rnd((c, c), seed + 3 + i, c ** -0.5) for i in range(4)]
    b = [rnd((c,), seed + 10 + i, 0.1) for i in range(4)]
    nb = ref.blocks(c)
    wq, sw = [torch.empty((c, c), dtype=F8, device=DEV) for _ in w], [torch.empty((nb, nb), device=DEV) for _ in w]
    for i in range(4):
        api.cc_gemm_fp8_prepare(w[i], wq[i], sw[i])
    q8, s8 = torch.empty((t, hw, c), dtype=F8, device=DEV), torch.empty((t, hw, nb), device=DEV)
    ws = torch.empty(api.cc_group_norm_workspace_bytes(t, hw, c, 32), dtype=torch.uint8, device=DEV)
    wsa = torch.empty(api.cc_attn_exp_workspace_bytes(t, hw), dtype=torch.uint8, device=DEV)
    qkv = torch.empty((t, hw, 3 * c), dtype=BF16, device=DEV)
    o, out = torch.empty((t, hw, c), dtype=BF16, device=DEV), torch.empty((t, hw, c), dtype=BF16, device=DEV)

    def step():
        api.cc_group_norm_act_fp8(x, gamma, beta, q8, s8, 32, ws, act="none")
        parts = [qkv[..., i * c:(i + 1) * c] for i in range(3)]
        for i in range(3):
            api.cc_gemm_fp8(q8, s8, wq[i], sw[i], b[i], None, parts[i])
        api.cc_attn_frame_exp(*parts, o, wsa)
        api.cc_fp8_quantize(o, q8, s8)
        api.cc_gemm_fp8(q8, s8, wq[3], sw[3], b[3], x, out)

    return step, x, gamma, beta, w, b, out


def test_attention_block_runs_together():
    t, hw, c = 2, 300, 256
    step, x, gamma, beta, w, b, out = attention_block(t, hw, c, 90)
    step()
    api.cc_check_device()
    h, _ = ref.group_norm(x, gamma, beta, 32, 1e-6, "none")
    q, k, v = (h @ w[i].double().T + b[i].double() for i in range(3))
    o = torch.softmax(q @ k.transpose(1, 2) / c ** 0.5, -1) @ v
    add = o @ w[3].double().T + b[3].double()
    # what the block adds to x, from operands rounded to e4m3 (2^-4 at most, about 0.025 rms each) on both sides of
    # two products in a row: 4 * 0.025, and bf16's roundings; the softmax passes the scores' error on, of the same size
    got = out.double() - x.double()
    assert float((got - add).norm() / add.norm()) < 0.2
    assert float((out.double() - x.double() - add).norm() / (x.double() + add).norm()) < 0.1


def test_attention_block_replays_from_a_graph_bit_by_bit():
    step, x, *_, out = attention_block(2, 300, 256, 120)
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    eager = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    x.copy_(rnd(x.shape, 140))
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    step()
    api.cc_check_device()
    assert torch.equal(out, replayed) and not torch.equal(out, eager)


def test_graphs_with_one_workspace_one_after_the_other():
    # the workspace needs no preparation and keeps nothing: two graphs may share it while they do not overlap
    x = [rnd((1, 200000, 128), 190), rnd((2, 90000, 256), 191)]
    y = [torch.empty_like(v) for v in x]
    need = max(api.cc_group_norm_workspace_bytes(v.shape[0], v.shape[1], v.shape[2], 8) for v in x)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    want, graphs = [], []
    for v, o in zip(x, y):
        api.cc_group_norm_act(v, None, None, o, 8, ws)
        torch.cuda.synchronize()
        want.append(o.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.cc_group_norm_act(v, None, None, o, 8, ws)
        graphs.append(g)
    for _ in range(3):
        ws.fill_(0xFF)
        for o in y:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(y, want))
    api.cc_check_device()


def test_packed_rows_of_a_chunk():
    # q, k and v normalised and quantised out of, and projected into, packed rows
    t, hw, c = 2, 77, 128
    qkv = rnd((t, hw, 3 * c), 192)
    q8, s8 = torch.empty((t, hw, c), dtype=F8, device=DEV), torch.empty((t, hw, 1), device=DEV)
    out = torch.zeros((t, hw, 3 * c), dtype=BF16, device=DEV)
    wq, sw = rnd_f8((c, c), 193), rnd_scales((1, 1), 194)
    for i in range(3):
        part = qkv[..., i * c:(i + 1) * c]
        api.cc_rms_norm_act_fp8(part, None, q8, s8, act="none")
        want, bound = ref.rms_norm(part, None, 1e-6, "none")
        ref.assert_fp8(q8, s8, want, bound, f"part {i}")
        api.cc_gemm_fp8(q8, s8, wq, sw, None, part, out[..., i * c:(i + 1) * c])
        check_gemm(out[..., i * c:(i + 1) * c].reshape(t * hw, c), q8.view(t * hw, c), s8.view(t * hw, 1), wq, sw,
                   None, part.reshape(t * hw, c), f"part {i}")
    api.cc_check_device()


def test_calls_on_two_streams_at_once():
    x = [rnd((2, 5000, 256), 150 + i) for i in range(2)]
    a, sa = [rnd_f8((600, 512), 160 + i) for i in range(2)], [rnd_scales((600, 4), 170 + i) for i in range(2)]
    wq, sw = rnd_f8((256, 512), 180), rnd_scales((2, 4), 181)
    ws = [torch.empty(api.cc_group_norm_workspace_bytes(2, 5000, 256, 32), dtype=torch.uint8, device=DEV)
          for _ in range(2)]
    y = [torch.empty_like(v) for v in x]
    o = [torch.empty((600, 256), dtype=BF16, device=DEV) for _ in range(2)]

    def one(i, stream=None):
        api.cc_group_norm_act(x[i], None, None, y[i], 32, ws[i], stream=stream)
        api.cc_gemm_fp8(a[i], sa[i], wq, sw, None, None, o[i], stream=stream)

    for i in range(2):
        one(i)
    torch.cuda.synchronize()
    want = [t.clone() for t in y + o]
    for t in y + o:
        t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            one(i, streams[i])
    torch.cuda.synchronize()
    api.cc_check_device()
    assert all(torch.equal(t, w) for t, w in zip(y + o, want))


def test_every_kind_of_product_on_two_streams_and_from_graphs():
    # few rows, divided sums, narrow and wide tiles, between norms: no kernel of one stream may hold up the other's
    shapes = [(3, 1024, 4096), (60, 2048, 1040), (100, 256, 4112), (300, 1024, 1040), (2300, 1800, 656), (20000, 136, 144)]
    sets = []
    for i, (m, n, k) in enumerate(shapes):
        wq, sw = rnd_f8((n, k), 300 + i), rnd_scales((ref.blocks(n), ref.blocks(k)), 310 + i)
        sets.append((rnd((m, k), 320 + i), wq, sw, rnd((n,), 330 + i)))

    def run(out, stream=None):
        for (x, wq, sw, bias), (y, s, o) in zip(sets, out):
            api.cc_rms_norm_act_fp8(x, None, y, s, act="silu", stream=stream)
            api.cc_gemm_fp8(y, s, wq, sw, bias, None, o, stream=stream)

    def outputs():
        return [(torch.zeros((m, k), dtype=torch.uint8, device=DEV).view(F8), torch.zeros((m, ref.blocks(k)), device=DEV),
                 torch.zeros((m, n), dtype=BF16, device=DEV)) for m, n, k in shapes]

    want, outs = outputs(), [outputs() for _ in range(4)]
    run(want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(8):
        for i in range(2):
            run(outs[i], streams[i])
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(outs[2 + i])
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    api.cc_check_device()
    for out in outs:
        for got, w in zip(out, want):
            assert torch.equal(got[2], w[2]) and torch.equal(got[1], w[1])
