"""Attention over long caches and long encoder's states, in which every key is looked for (long_cache_ref.py): items cut
over the whole grid, several cut ones in a call, both kernels."""

import pytest
import torch

import long_cache_ref as ref
from causal_convolution_gb300 import api
from gpu_util import ensure_built
from test_gpu_heads import BF16, DEV, Cache, ints, paged, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return ensure_built()


def queries(rows, heads, d):
    """(q [rows, heads, d], pattern of each): row i's head h is 1 in channel (i + h) % PATTERNS."""
    pattern = (torch.arange(rows)[:, None] + torch.arange(heads)) % ref.PATTERNS
    return torch.nn.functional.one_hot(pattern, d).to(BF16).to(DEV), pattern


def expected(s, pattern, limits):
    """Shares [rows, heads, runs] of rows whose head h has the scores s[h // group] of one key head."""
    group = pattern.shape[1] // len(s)
    return torch.stack([ref.shares(s[h // group], pattern[:, h], limits) for h in range(pattern.shape[1])], 1).to(DEV)


def result_of(share, d, call):
    return ref.result_of(share.flatten(0, 1), d, call).view(*share.shape[:2], d)


@pytest.mark.parametrize("spread", [0, 16])
@pytest.mark.parametrize("lens,page,heads,kv_heads,d", [
    ([(1, 40000)], 128, 16, 2, 128),
    ([(1, 61001)], 16, 1, 1, 128), ([(1, 61001)], 16, 8, 1, 64), ([(8, 61001)], 16, 1, 1, 96),  # few rows
    ([(1, 61001)], 16, 16, 1, 128), ([(16, 61001)], 16, 16, 1, 128), ([(130, 61001)], 16, 2, 1, 64),
    ([(3, 61001)], 16, 7, 1, 16), ([(600, 30000)], 64, 2, 2, 80),
    ([(1, 30000), (1, 100), (1, 50001), (1, 1)], 48, 8, 2, 128), ([(300, 9000), (0, 70), (1, 30000), (40, 5000)], 32, 6, 2, 112),
])
def test_every_key_of_a_long_cache_counts_once(lens, page, heads, kv_heads, d, spread):
    c = Cache(lens, page, kv_heads, d, seed=240)
    q, pattern = queries(c.rows, heads, d)
    c.k.fill_(float("nan")), c.v.fill_(float("nan"))  # behind the sequences' ends
    at = [c.slots(b, 0, kv) for b, (_, kv) in enumerate(lens)]
    share = []
    for b, (new, kv) in enumerate(lens):
        s = [ref.scores(kv, spread, 10 * b + h) for h in range(kv_heads)]
        c.k[at[b]] = torch.stack([ref.keys(x, kv, d) for x in s], 1).to(BF16).to(DEV)
        first = c.offsets_host[b]
        share.append(expected(s, pattern[first:first + new], torch.arange(kv - new + 1, kv + 1)))
    for call in range(max(ref.calls_of(kv, d) for _, kv in lens)):
        for b, (_, kv) in enumerate(lens):
            c.v[at[b]] = ref.values(kv, d, call).to(BF16).to(DEV)[:, None]
        o = paged(c, q, 1.0, 1)
        for b, (new, _) in enumerate(lens):
            got = o[c.offsets_host[b]:c.offsets_host[b] + new]
            assert ref.off(got, result_of(share[b], d, call)) == 0, (call, b)


@pytest.mark.parametrize("spread", [0, 16])
@pytest.mark.parametrize("n,lq,lk,heads,kv_heads,d,lens", [
    (1, 1, 100000, 1, 1, 128, [99999]), (1, 500, 20000, 1, 1, 96, [19999]), (2, 40, 9000, 4, 2, 80, [8999, 5000]),
    (3, 1, 30000, 8, 1, 64, None),
])
def test_every_key_of_long_states_counts_once(n, lq, lk, heads, kv_heads, d, lens, spread):
    q, pattern = queries(n * lq, heads, d)
    k, v = (torch.full((n, lk, kv_heads, d), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    o, ws = torch.empty((n, lq, heads, d), dtype=BF16, device=DEV), workspace(
        api.cc_attn_cross_workspace_bytes(n, lq, lk, heads, kv_heads, d))
    share = []
    for b in range(n):
        length = lens[b] if lens else lk
        s = [ref.scores(length, spread, 10 * b + h) for h in range(kv_heads)]
        k[b, :length] = torch.stack([ref.keys(x, length, d) for x in s], 1).to(BF16).to(DEV)
        share.append(expected(s, pattern[b * lq:(b + 1) * lq], torch.full((lq,), length)))
    for call in range(ref.calls_of(lk, d)):
        for b in range(n):
            length = lens[b] if lens else lk
            v[b, :length] = ref.values(length, d, call).to(BF16).to(DEV)[:, None]
        api.cc_attn_cross(q.view(n, lq, heads, d), k, v, o, ints(lens) if lens else None, ws.t, scale=1.0)
        api.cc_check_device()
        for b in range(n):
            assert ref.off(o[b], result_of(share[b], d, call)) == 0, (call, b)
