"""What attention over a long cache comes to when every key can be told from its neighbours' run.

A sum over tens of thousands of random values is small beside the sum of their sizes, and so is what a lost key changes of
it. Here SHARE keys in a row have one score and a channel of their own in v, which is 1 for them and 0 for all others, so
that a channel's result is their share of the weights alone: n p / sum p. With one key lost, counted twice or given
another one's value it is off by 1 / SHARE or more, and with a piece of the sum on a wrong scale by a factor of two. A
call has room for d channels, so calls are made until all keys had their turn.

What a right kernel may be off, relative to the result: SHARE keys have the same weight, whose rounding to bf16 (2^-8) is
the same for all of them; the sum that is divided by is off by 2^-8 of itself in the same way, and the result's own
rounding is another 2^-8. Everything in fp32 is small beside that: a weight by its exponent's rounding (60 x 2^-24) and the
exponential's (2^-22), the sum by fewer than 2^11 additions in a row (2^-13), the channel by SHARE additions, as adding
zeros and multiplying by powers of two is exact."""

import torch

SHARE = 32
PATTERNS = 4          # sets of scores; a query head picks one
STEP = 2.0 ** -8      # half a step of bf16, relative
BOUND = (1 + STEP) ** 2 / (1 - STEP) - 1 + 2.0 ** -12


def runs_of(length):
    return -(-length // SHARE)


def scores(length, spread, seed):
    """[PATTERNS, runs]: multiples of 1/4 up to `spread` <= 32 in size, which bf16 and fp32 products hold exactly."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-4 * spread, 4 * spread + 1, (PATTERNS, runs_of(length)), generator=g).double() / 4


def keys(s, length, d):
    """[length, d], the patterns' scores in the first channels. (A query is 1 in the channel of its pattern.)"""
    k = torch.zeros(length, d, dtype=torch.float64)
    k[:, :PATTERNS] = s.repeat_interleave(SHARE, 1)[:, :length].T
    return k


def calls_of(length, d):
    return -(-runs_of(length) // d)


def values(length, d, call):
    """[length, d] of call number `call`: the runs call * d .. call * d + d - 1 have a channel each."""
    run = torch.arange(length) // SHARE - call * d
    return (run[:, None] == torch.arange(d)).double()


def shares(s, pattern, limits):
    """[rows, runs]: each run's share of a row's weights. Row i has the scores s[pattern[i]] and sees limits[i] keys."""
    seen = (limits[:, None] - SHARE * torch.arange(s.shape[1])).clamp(0, SHARE).double()
    p = torch.exp(s[pattern] - s[pattern].amax(-1, keepdim=True))
    total = (p * seen).sum(-1, keepdim=True)
    return torch.where(total > 0, p * seen / total, 0.0)


def result_of(share, d, call):
    """[rows, d] of a call."""
    part = share[:, call * d:call * d + d]
    return torch.nn.functional.pad(part, (0, d - part.shape[1]))


def off(got, want):
    """How many values are off by more than a right kernel's."""
    return int((~((got.double() - want).abs() <= BOUND * want)).sum())
