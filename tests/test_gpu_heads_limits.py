"""The operators with heads at the limits of what they take: the most sequences, strides that do not count."""

import pytest
import torch

from causal_convolution_gb300 import api
from gpu_util import ensure_built
from test_gpu_heads import BF16, DEV, I32, Cache, paged, rnd, same_bits

pytestmark = pytest.mark.gpu
MOST = 1 << 20  # sequences


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return ensure_built()


def test_the_most_instances():
    # one key to an instance: its value is the result
    q, k, v = (rnd((MOST, 1, 1, 16), 200 + i) for i in range(3))
    o = torch.empty_like(q)
    api.cc_attn_cross(q, k, v, o, None, None)
    api.cc_check_device()
    assert same_bits(o, v)


def test_the_most_sequences_nearly_all_without_new_tokens():
    k, v = rnd((2, 16, 1, 16), 210), rnd((2, 16, 1, 16), 211)
    q, o = rnd((2, 1, 16), 212), torch.empty((2, 1, 16), dtype=BF16, device=DEV)
    offsets = torch.ones(MOST + 1, dtype=I32, device=DEV)
    offsets[0], offsets[-1] = 0, 2
    lens, table = torch.ones(MOST, dtype=I32, device=DEV), torch.zeros((MOST, 1), dtype=I32, device=DEV)
    table[-1] = 1
    api.cc_attn_paged(q, k, v, o, offsets, lens, table, None)
    api.cc_check_device()
    assert same_bits(o, v[:, 0])


def test_the_most_sequences_half_of_them_of_two_items():
    # 8 query heads to a key head: an item of the variant for few rows is one token. Token 0 sees itself alone, token 1
    # two keys that are the same.
    k, v = rnd((1, 16, 1, 16), 220), rnd((1, 16, 1, 16), 221)
    k[0, 1], v[0, 1] = k[0, 0], v[0, 0]
    q, o = rnd((MOST, 8, 16), 222), torch.empty((MOST, 8, 16), dtype=BF16, device=DEV)
    offsets = (torch.arange(MOST + 1, device=DEV) // 2 * 2).to(I32)
    lens, table = torch.full((MOST,), 2, dtype=I32, device=DEV), torch.zeros((MOST, 1), dtype=I32, device=DEV)
    ws = torch.empty(api.cc_attn_paged_workspace_bytes(MOST, MOST, 8, 1, 16), dtype=torch.uint8, device=DEV)
    api.cc_attn_paged(q, k, v, o, offsets, lens, table, ws)
    api.cc_check_device()
    assert same_bits(o, v[0, 0].expand(MOST, 8, 16))


@pytest.mark.parametrize("lens,heads,kv_heads,d,spare", [
    ([(1, 300)], 4, 1, 64, 0), ([(40, 300), (3, 90)], 4, 1, 80, 2), ([(1, 40)], 6, 3, 128, 0), ([(100, 176)], 2, 1, 32, 0),
])
def test_strides_of_a_single_head_or_page_do_not_count(lens, heads, kv_heads, d, spare):
    c = Cache(lens, 176, kv_heads, d, seed=230, spare=spare)
    if len(lens) == 1 and lens[0][1] <= 176:
        assert c.k.shape[0] == 1
    q = rnd((c.rows, heads, d), 231, 2.0)
    x = rnd((c.rows, heads + 2 * kv_heads, d), 232)

    def append(k, v):
        qo = torch.empty_like(q)
        api.cc_qk_norm_rope_append(x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], None, None, None,
                                   None, qo, k, v, *c.plan)
        api.cc_check_device()

    def strided(t, stride):
        # the same memory with another stride where there is one page or head
        return t.as_strided(t.shape, (stride if t.shape[0] == 1 else t.stride(0), t.stride(1),
                                      stride if t.shape[2] == 1 else t.stride(2), 1))

    append(c.k, c.v)
    want, k, v = paged(c, q, None, 1), c.k, c.v
    want_k, want_v = k.clone(), v.clone()
    for stride in (0, 3, 1 << 40):
        for b, (new, kv) in enumerate(lens):
            at = c.slots(b, kv - new, kv)
            k[at], v[at] = 0, 0
        c.k, c.v = strided(k, stride), strided(v, stride)
        append(c.k, c.v)
        assert same_bits(k, want_k) and same_bits(v, want_v)
        assert same_bits(paged(c, q, None, 1), want)
