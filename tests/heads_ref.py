"""Plain 64-bit forms of the operators with heads, each with a bound on what a kernel with fp32 sums may be off.

A rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by 2^-24."""

import torch

STEP = 2.0 ** -8    # half a step of bf16, relative
FP32 = 2.0 ** -24   # the same of fp32


def assert_close(got, want, bound, what):
    got = got.double()
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, the worst by "
                                 f"{float((off / bound.clamp(min=1e-300)).nan_to_num(1e9)[bad].max()):.3g} bounds")


def rotated(x, gamma, rot, pos, eps, style):
    """x [rows, heads, D]; rot [positions, rd/2, 2] or None; pos: a list or tensor of positions."""
    x = x.double()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    if gamma is not None:
        y = y * gamma.double()
    size = y.abs()
    rd = 0 if rot is None else 2 * rot.shape[1]
    if rd:
        t = rot.double()[torch.as_tensor(pos, device=x.device).long()][:, None]
        c, s = t[..., 0], t[..., 1]
        if style == "pairs":
            ia, ib = torch.arange(0, rd, 2), torch.arange(1, rd, 2)
        else:
            ia, ib = torch.arange(rd // 2), torch.arange(rd // 2, rd)
        a, b = y[..., ia].clone(), y[..., ib].clone()
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        size[..., ia], size[..., ib] = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    # sum of squares (a tree of at most 8 + 5 additions), mean, root and quotient, gamma, two products and their sum:
    # fewer than 2^5 roundings of fp32 in a row
    return y, STEP * y.abs() + 2 ** 5 * FP32 * size + 1e-37


def attend(q, k, v, limit, scale):
    """q [n, H, D], k, v [L, Hk, D]; query i sees the first limit[i] keys. Rows that see none are zeros."""
    n, heads, d = q.shape
    length, kv_heads, _ = k.shape
    q, k, v = q.double(), k.double(), v.double()
    group = heads // kv_heads
    want = torch.zeros(n, heads, d, dtype=torch.float64, device=q.device)
    bound = torch.full_like(want, 1e-37)
    if length == 0 or n == 0:
        return want, bound
    sees = torch.arange(length, device=q.device) < limit[:, None]
    empty = ~sees.any(-1)
    for h in range(heads):
        kh, vh = k[:, h // group], v[:, h // group]
        scores = (q[:, h] @ kh.T * scale).masked_fill(~sees, float("-inf"))
        scores[empty] = 0.0
        p = torch.softmax(scores, -1)
        p[empty] = 0.0
        want[:, h] = p @ vh
        size = p @ vh.abs()
        # a score: D products summed in fp32 and scaled; a weight is off by twice the scores' error (its own and the
        # sum's), by the exponential's (2^-22), and by its rounding to bf16; length terms are summed in fp32 twice,
        # by adders that may drop bits down to 2^-22 of a term. The exponent's own rounding: |exponent| 2^-24.
        # What is divided by is the sum of the rounded weights: sum p (1 + e_i) v / sum p (1 + e_i) with |e_i| <= 2^-8 has a
        # numerator off by 2^-8 sum p |v| and a denominator off by 2^-8 of itself, which is 2^-8 of the result; the
        # result's own rounding is another.
        top = (scores.masked_fill(~sees, 0.0).abs().amax(-1, keepdim=True)) * 1.5
        err = (d + 4) * 4 * FP32 * scale * (q[:, h].abs() @ kh.abs().T).amax(-1, keepdim=True) + 4 * FP32 * top
        bound[:, h] = STEP * want[:, h].abs() * (2 + 2 ** -6) + size * (
            STEP + 2 * err + 2.0 ** -20 + 2 * length * 2.0 ** -22)
    return want, bound + 1e-37


def limits(n, length, block, device):
    i = torch.arange(n, device=device)
    if block == 0:
        return torch.full((n,), length, device=device)
    return length - n + ((i // block + 1) * block).clamp(max=n)
