"""That the check of attention over a long cache sees what it is for: mistakes planted in the oracle, on the host."""

import pytest
import torch

import long_cache_ref as ref

CASES = [(40000, 128), (61001, 128), (61001, 16), (99999, 64)]


def attention(k, v, counts, scale_off=None):
    """Rows of one query to a pattern over k [L, d], with each key counted counts[j] times; bf16 as a kernel rounds."""
    p = torch.exp(k[:, :ref.PATTERNS].T - k[:, :ref.PATTERNS].amax())
    p = p.to(torch.bfloat16).double() * counts
    if scale_off is not None:
        p[:, scale_off] *= 2
    return (p @ v / p.sum(-1, keepdim=True)).to(torch.bfloat16)


@pytest.mark.parametrize("length,d", CASES)
@pytest.mark.parametrize("spread", [0, 16])
def test_planted_mistakes_are_seen(length, d, spread):
    s = ref.scores(length, spread, 1)
    k, one = ref.keys(s, length, d), torch.ones(length, dtype=torch.float64)
    share = ref.shares(s, torch.arange(ref.PATTERNS), torch.full((ref.PATTERNS,), length))
    assert torch.allclose(share.sum(-1), torch.ones(ref.PATTERNS, dtype=torch.float64))

    def seen(at, counts=one, value_of=None, scale_off=None):
        """Whether a mistake at key `at` is seen by the call in which it has its turn, for every pattern."""
        call = at // ref.SHARE // d
        v = ref.values(length, d, call)
        v = v if value_of is None else v[value_of]
        got, want = attention(k, v, counts, scale_off), ref.result_of(share, d, call)
        return all(ref.off(got[i], want[i]) for i in range(ref.PATTERNS))

    last = (length - 1) // ref.SHARE * ref.SHARE
    for at in (0, 63, 64, 255, 256, 12345, length // 2, last, length - 1):
        assert not seen(at)  # nothing planted
        for size in (1, 64, 256, length // 20):  # a key, a tile, a piece, a twentieth of the cache
            lo = min(at, length - size)
            for times in (0.0, 2.0):
                counts = one.clone()
                counts[lo:lo + size] = times
                assert seen(lo, counts), (at, size, times)
        where = torch.arange(length)  # a key has another run's value
        where[at] = (at + ref.SHARE) % length
        assert seen(at, value_of=where)
        assert seen(at, scale_off=slice(at, at + 64))


def test_the_last_run_and_rows_that_see_a_part():
    length, d = 1000, 16
    s = ref.scores(length, 16, 2)
    limits = torch.tensor([0, 1, 31, 32, 33, 500, 999, 1000])
    share = ref.shares(s, torch.zeros(8, dtype=torch.int64), limits)
    p = torch.exp(ref.keys(s, length, d)[:, 0])
    for i, limit in enumerate(limits.tolist()):
        for run in range(ref.runs_of(length)):
            lo, hi = run * ref.SHARE, min(limit, run * ref.SHARE + ref.SHARE)
            want = float(p[lo:hi].sum() / p[:limit].sum()) if limit > lo else 0.0
            assert abs(float(share[i, run]) - want) <= 1e-12 * want
    assert ref.calls_of(length, d) == 2
    assert torch.equal(ref.result_of(share, d, 1)[:, :16], share[:, 16:])
