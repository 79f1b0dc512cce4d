"""Plain 64-bit forms of the norms, the block quantisation and the 8-bit
product, with the error bounds the GPU tests hold the kernels to."""

import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2       # 2^-8: half a step, relative
E4M3_HALF = torch.finfo(torch.float8_e4m3fn).eps / 2  # 2^-4
E4M3_HALF_SUBNORMAL = 2.0 ** -10                      # half of the smallest step, in units of the scale
F32 = 2.0 ** -24


def blocks(c):
    return -(-c // 128)


def spread(scales, c):
    """A scale per block -> a scale per channel."""
    return scales.repeat_interleave(128, -1)[..., :c]


def activation(v, act):
    return v * torch.sigmoid(v) if act == "silu" else v


def group_norm(x, gamma, beta, groups, eps, act):
    """(y, bound) in fp64; bound: what fp32 arithmetic may be off by before the output's rounding.

    The kernels compute (x - mean) * a + beta with a = gamma * r. Each of r, a, the difference and the fused
    multiply-add is rounded once or twice; r and the mean carry the error of sums in fp32, at most 128 terms one after
    the other in a thread and a tree above them: below (128 + 64) * 2^-24 relative to the summed magnitudes. 256 * 2^-24
    of |x a| + |mean a| + |b|, and of |(x - mean) a| for r's error, covers them. silu has a slope below 1.1 and two
    fast operations of 2^-21 each: 2^-19 of the result."""
    n, c = x.shape[0], x.shape[-1]
    xd = x.double().reshape(n, -1, groups, c // groups)
    mean = xd.mean((1, 3), keepdim=True)
    var = (xd - mean).square().mean((1, 3), keepdim=True)
    r = (var + eps).rsqrt()
    g = torch.ones(c, dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    b = torch.zeros(c, dtype=torch.float64, device=x.device) if beta is None else beta.double()
    g, b = g.view(groups, -1), b.view(groups, -1)
    v = (xd - mean) * r * g + b
    size = (xd.abs() + mean.abs()) * r * g.abs() + b.abs()
    # the mean's own error is relative to the mean of |x|, which may exceed |mean|
    size = size + xd.abs().mean((1, 3), keepdim=True) * r * g.abs()
    y = activation(v, act)
    bound = 1.1 * 256 * F32 * size + 2.0 ** -19 * y.abs()
    return y.reshape(x.shape), bound.reshape(x.shape)


def rms_norm(x, gamma, eps, act):
    """(y, bound) in fp64; the sum over at most 16384 squares has at most 64 terms in a row and a tree above them."""
    xd = x.double()
    g = 1.0 if gamma is None else gamma.double()
    v = xd / (xd.square().mean(-1, keepdim=True) + eps).sqrt() * g
    y = activation(v, act)
    return y, 1.1 * 128 * F32 * v.abs() + 2.0 ** -19 * y.abs()


def block_scales(v):
    """max(max |v| / 448, 2^-126) of each block of 128 channels, in fp64."""
    c = v.shape[-1]
    pad = torch.zeros(*v.shape[:-1], blocks(c) * 128 - c, dtype=v.dtype, device=v.device)
    top = torch.cat([v, pad], -1).reshape(*v.shape[:-1], blocks(c), 128).abs().amax(-1)
    return (top / 448).clamp(min=2.0 ** -126)


def gemm(a, sa, wq, sw, bias, res):
    """(out, sum of the products' magnitudes) in fp64."""
    k, n = a.shape[-1], wq.shape[0]
    ad = a.double() * spread(sa.double(), k)
    wd = wq.double() * spread(sw.double(), k).repeat_interleave(128, 0)[:n]
    out, size = ad @ wd.T, ad.abs() @ wd.abs().T
    for extra in (bias, res):
        if extra is not None:
            out, size = out + extra.double(), size + extra.double().abs()
    return out, size


def assert_bf16(y, ref, bound, what):
    """Off by one rounding to bf16 and the bound in front of it."""
    err = (y.double() - ref).abs()
    room = BF16_HALF * (ref.abs() + bound) + bound + 2.0 ** -133
    bad = ~(err <= room)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / room).max()):.3g}x"


def assert_fp8(q, scales, ref, bound, what):
    """The scales to fp32 of the block's largest value, each value within half an e4m3 step of its own."""
    c = ref.shape[-1]
    want = block_scales(ref)
    slack = block_scales(bound.abs()) + 4 * F32 * want
    assert bool(((scales.double() - want).abs() <= slack).all()), f"{what}: scales"
    s = spread(scales.double(), c)
    err = (q.double() * s - ref).abs()
    room = E4M3_HALF * (ref.abs() + bound) + E4M3_HALF_SUBNORMAL * s + bound + 8 * F32 * ref.abs()
    bad = ~(err <= room)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / room).max()):.3g}x"
