"""Head norms with rotation, the paged cache and the attentions over it and over an encoder's states, against plain
64-bit forms: from one token to long caches, odd sizes, strides and layouts, rows that see nothing, NaN behind a
sequence's end, bad plans, guard bands, graphs and streams, and a run of them together as a decoder's block uses them."""

import pytest
import torch

import heads_ref as ref
from causal_convolution_gb300 import api
from gpu_util import ensure_built
from test_gpu_guard_bands import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return ensure_built()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rnd(shape, seed, scale=1.0, offset=0.0):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * scale + offset).to(BF16)


def ints(values):
    return torch.tensor(values, dtype=I32, device=DEV)


def rot_table(positions, rd):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rd // 2) / (rd // 2))
    return torch.stack([angle.cos(), angle.sin()], -1).float().to(DEV)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


# ------------------------------------------------------------------------------------------------ norm, rotation --

@pytest.mark.parametrize("style", ["pairs", "halves"])
@pytest.mark.parametrize("rows,heads,kv_heads,d,rd", [
    (1, 1, 1, 16, 16), (2, 8, 8, 64, 64), (5, 3, 1, 32, 16), (7, 14, 2, 80, 80), (33, 10, 10, 96, 64),
    (100, 32, 8, 128, 128), (3, 1, 5, 144, 48), (9, 2, 3, 256, 256), (17, 5, 4, 240, 0), (3000, 7, 1, 112, 112),
])
def test_norm_and_rotation_match_64_bits(rows, heads, kv_heads, d, rd, style):
    packed = rnd((rows, heads + kv_heads, d), 1 + rows, 1.7, 0.2)
    q, k = packed[:, :heads], packed[:, heads:]
    gq, gk = rnd((d,), 2, 0.3, 1.0), rnd((d,), 3, 0.3, 1.0)
    rot = rot_table(rows + 3, rd) if rd else None
    pos = torch.randint(0, rows + 3, (rows,), generator=gen(4), device=DEV).to(I32)
    qo, ko = Guarded((rows, heads, d)), Guarded((rows, kv_heads, d))
    before = packed.clone()
    api.cc_qk_norm_rope(q, k, gq, gk, rot, pos, qo.t, ko.t, style=style)
    api.cc_check_device()
    assert qo.bands_intact() and ko.bands_intact() and same_bits(packed, before)
    ref.assert_close(qo.t, *ref.rotated(q, gq, rot, pos, 1e-6, style), "q")
    ref.assert_close(ko.t, *ref.rotated(k, gk, rot, pos, 1e-6, style), "k")
    # in place, without positions and gammas
    api.cc_qk_norm_rope(q, k, None, None, rot, None, q, k, eps=0.01, style=style)
    api.cc_check_device()
    rows_at = torch.arange(rows, device=DEV)
    ref.assert_close(q, *ref.rotated(before[:, :heads], None, rot, rows_at, 0.01, style), "q in place")
    ref.assert_close(k, *ref.rotated(before[:, heads:], None, rot, rows_at, 0.01, style), "k in place")


def test_norm_of_one_side_and_of_more_dimensions():
    x, g = rnd((2, 3, 4, 64), 5), rnd((64,), 6, 0.3, 1.0)
    want = ref.rotated(x.view(6, 4, 64), g, None, None, 1e-6, "pairs")
    for args in ((x, None, g, None), (None, x, None, g)):
        y = torch.empty_like(x)
        outs = (y, None) if args[0] is not None else (None, y)
        api.cc_qk_norm_rope(*args, None, None, *outs)
        api.cc_check_device()
        ref.assert_close(y.view(6, 4, 64), *want, "one side")


def test_norm_keeps_zeros_nan_and_far_positions():
    q = rnd((4, 2, 64), 7)
    q[0], q[1, 0, 5], q[2] = 0, float("nan"), q[2] * 1e-18
    rot = rot_table(200001, 64)
    pos = ints([200000, 1, 0, 199999])
    out = torch.empty_like(q)
    api.cc_qk_norm_rope(q, None, None, None, rot, pos, out, None, style="halves")
    api.cc_check_device()
    assert not bool(out[0].any()) and bool(out[1, 0].isnan().all()) and not bool(out[1, 1].isnan().any())
    rows = torch.tensor([0, 2, 3], device=DEV)
    want, bound = ref.rotated(q[rows], None, rot, pos[rows], 1e-6, "halves")
    ref.assert_close(out[rows], want, bound, "far")


def test_norm_reports_positions_outside_of_the_table():
    q, rot, out = rnd((6, 3, 32), 8), rot_table(5, 32), Guarded((6, 3, 32))
    api.cc_qk_norm_rope(q, None, None, None, rot, ints([0, 5, 4, -1, 2, 2147483647]), out.t, None)
    with pytest.raises(api.CCError) as e:
        api.cc_check_device()
    assert e.value.status == 5 and out.bands_intact()
    api.cc_check_device()
    good = torch.tensor([0, 2, 4], device=DEV)
    ref.assert_close(out.t[good], *ref.rotated(q[good], None, rot, [0, 4, 2], 1e-6, "pairs"), "the others")


# ------------------------------------------------------------------------------------------------------ the cache --

class Cache:
    """A paged cache of random content with a plan: lens [(new, tokens with them)]."""

    def __init__(self, lens, page, kv_heads, d, layout="plain", seed=10, spare=2, lead=0, tail=0):
        self.lens, self.page = lens, page
        used = [-(-kv // page) for _, kv in lens]
        pages = sum(used) + spare
        if layout == "plain":
            self.k, self.v = rnd((pages, page, kv_heads, d), seed), rnd((pages, page, kv_heads, d), seed + 1)
        elif layout == "joint":  # a page holds its keys and values
            both = rnd((pages, 2, page, kv_heads, d), seed)
            self.k, self.v = both[:, 0], both[:, 1]
        elif layout == "heads":  # a page holds a head's tokens side by side
            both = rnd((pages, kv_heads, page, d), seed), rnd((pages, kv_heads, page, d), seed + 1)
            self.k, self.v = both[0].transpose(1, 2), both[1].transpose(1, 2)
        else:  # channels of wider rows
            both = rnd((pages, page, kv_heads, 2 * d + 8), seed)
            self.k, self.v = both[..., :d], both[..., d + 8:]
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        most = max(max(used, default=0), 1) + 1
        self.table_host = []
        for u in used:
            self.table_host.append(order[:u] + [-7] * (most - u))  # what lies behind the last page is not read
            order = order[u:]
        self.spare = order
        self.table = ints(self.table_host)
        offsets = [lead]
        for new, _ in lens:
            offsets.append(offsets[-1] + new)
        self.offsets_host, self.rows = offsets, offsets[-1] + tail
        self.offsets, self.kv_lens = ints(offsets), ints([kv for _, kv in lens])

    @property
    def plan(self):
        return self.offsets, self.kv_lens, self.table

    def slots(self, b, lo, hi):
        at = torch.arange(lo, hi)
        pages = torch.tensor(self.table_host[b])[at // self.page]
        return pages.to(DEV), (at % self.page).to(DEV)

    def seq(self, b):
        return [c[self.slots(b, 0, self.lens[b][1])] for c in (self.k, self.v)]


@pytest.mark.parametrize("style", ["pairs", "halves"])
@pytest.mark.parametrize("lens,page,heads,kv_heads,d,rd,layout", [
    ([(1, 1)], 16, 1, 1, 16, 16, "plain"),
    ([(1, 700), (1, 1), (1, 64), (1, 65)], 64, 8, 2, 128, 128, "joint"),
    ([(77, 80), (0, 50), (300, 300), (5, 4000)], 48, 10, 10, 96, 64, "plain"),
    ([(0, 0), (130, 131), (0, 7)], 16, 3, 3, 80, 80, "heads"),
    ([(1, 100 + b) for b in range(50)], 32, 4, 1, 32, 0, "wide"),
    ([(1 + b % 3, 900 + b) for b in range(700)], 128, 2, 2, 64, 32, "joint"),
])
def test_append_matches_64_bits(lens, page, heads, kv_heads, d, rd, layout, style):
    c = Cache(lens, page, kv_heads, d, layout, lead=2, tail=3)
    packed = rnd((c.rows, heads + 2 * kv_heads, d), 11, 1.5)
    q, k, v = packed[:, :heads], packed[:, heads:heads + kv_heads], packed[:, heads + kv_heads:]
    gq, gk = rnd((d,), 12, 0.3, 1.0), rnd((d,), 13, 0.3, 1.0)
    rot = rot_table(max(kv for _, kv in lens), rd) if rd else None
    qo = Guarded((c.rows, heads, d))
    qo.t.fill_(7.0)
    k_before, v_before = c.k.clone(), c.v.clone()
    api.cc_qk_norm_rope_append(q, k, v, gq, gk, rot, None, qo.t, c.k, c.v, *c.plan, style=style)
    api.cc_check_device()
    assert qo.bands_intact()
    outside = torch.ones(c.rows, dtype=torch.bool)
    for b, (new, kv) in enumerate(lens):
        first = c.offsets_host[b]
        rows, pos = slice(first, first + new), torch.arange(kv - new, kv)
        outside[rows] = False
        at = c.slots(b, kv - new, kv)
        ref.assert_close(qo.t[rows], *ref.rotated(q[rows], gq, rot, pos, 1e-6, style), f"q of {b}")
        ref.assert_close(c.k[at], *ref.rotated(k[rows], gk, rot, pos, 1e-6, style), f"k of {b}")
        assert same_bits(c.v[at], v[rows])
        k_before[at], v_before[at] = c.k[at], c.v[at]
    # nothing else was written
    assert same_bits(c.k, k_before) and same_bits(c.v, v_before)
    assert bool((qo.t[outside.to(DEV)] == 7.0).all())


def test_append_reports_bad_plans_and_keeps_to_the_cache():
    heads, kv_heads, d, page = 2, 1, 32, 16
    cases = {
        "page": lambda c: c.table[1].fill_(c.k.shape[0]), "negative page": lambda c: c.table[1].fill_(-1),
        "too long": lambda c: c.kv_lens[1:2].fill_(5000), "too short": lambda c: c.kv_lens[1:2].fill_(3),
        "negative": lambda c: c.kv_lens[1:2].fill_(-2147483648),
    }
    for what, spoil in cases.items():
        c = Cache([(4, 20), (5, 30), (3, 3)], page, kv_heads, d)
        spoil(c)
        packed = rnd((c.rows, heads + 2, d), 14)
        guard_k, guard_v = Guarded(tuple(c.k.shape)), Guarded(tuple(c.v.shape))
        guard_k.t.copy_(c.k), guard_v.t.copy_(c.v)
        qo = Guarded((c.rows, heads, d))
        api.cc_qk_norm_rope_append(packed[:, :2], packed[:, 2:3], packed[:, 3:], None, None, None, None, qo.t,
                                   guard_k.t, guard_v.t, *c.plan)
        with pytest.raises(api.CCError) as e:
            api.cc_check_device()
        assert e.value.status == 5, what
        assert qo.bands_intact() and guard_k.bands_intact() and guard_v.bands_intact(), what
        for b in (0, 2):  # the good sequences
            new, kv = c.lens[b]
            rows = slice(c.offsets_host[b], c.offsets_host[b] + new)
            ref.assert_close(guard_k.t[c.slots(b, kv - new, kv)], *ref.rotated(packed[rows, 2:3], None, None, None, 1e-6,
                                                                               "pairs"), what)


# -------------------------------------------------------------------------------------------------- the attentions --

def workspace(need):
    ws = Guarded((need,), torch.uint8)
    ws.t.fill_(0xFF)  # its contents need no preparation
    return ws


def paged(c, q, scale, block):
    o, ws = Guarded(tuple(q.shape)), workspace(api.cc_attn_paged_workspace_bytes(
        c.rows, len(c.lens), q.shape[1], c.k.shape[2], q.shape[2]))
    o.t.fill_(7.0)
    api.cc_attn_paged(q, c.k, c.v, o.t, *c.plan, ws.t, scale=scale, causal_block=block)
    api.cc_check_device()
    assert o.bands_intact() and ws.bands_intact()
    return o.t


def check_paged(c, q, o, scale, block, what):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    outside = torch.ones(c.rows, dtype=torch.bool)
    for b, (new, kv) in enumerate(c.lens):
        rows = slice(c.offsets_host[b], c.offsets_host[b] + new)
        outside[rows] = False
        k, v = c.seq(b)
        ref.assert_close(o[rows], *ref.attend(q[rows], k, v, ref.limits(new, kv, block, DEV), scale), f"{what} {b}")
    assert bool((o[outside.to(DEV)] == 7.0).all())


PAGED = [  # lens, page, heads, kv_heads, d, block, layout
    ([(1, 1)], 16, 1, 1, 16, 1, "plain"),
    ([(1, 2000)], 16, 8, 8, 64, 1, "plain"),
    ([(1, 1), (1, 127), (1, 128), (1, 129), (1, 300), (1, 4096)], 64, 32, 8, 128, 1, "joint"),
    ([(1, 40000)], 128, 16, 2, 128, 1, "plain"),
    ([(37, 37), (300, 1211), (1, 5), (0, 90), (129, 130), (64, 4000)], 48, 14, 2, 80, 1, "plain"),
    ([(128, 128), (256, 256), (257, 600)], 32, 4, 4, 128, 1, "heads"),
    ([(700, 2000)], 256, 3, 3, 48, 100, "wide"),
    ([(500, 1000), (333, 333)], 80, 6, 2, 112, 0, "joint"),
    ([(10, 3), (5, 0), (4, 700)], 16, 2, 1, 32, 0, "plain"),  # fewer tokens than new rows, and none
    ([(9, 800)], 16, 128, 1, 64, 1, "plain"),                 # a full tile of heads to a token
    ([(50, 900)], 16, 65, 1, 96, 3, "plain"),                 # a token to a tile, with rows left over
    ([(1, 100 + 37 * b) for b in range(90)], 16, 4, 4, 64, 1, "joint"),
    ([(1 + b % 5, 2 + 11 * (b % 70)) for b in range(400)], 32, 5, 1, 32, 1, "plain"),
    ([(1500, 3100)], 16, 16, 16, 128, 500, "plain"),
    ([(2100, 2100), (1, 17000)], 112, 7, 7, 64, 1, "plain"),
]


@pytest.mark.parametrize("lens,page,heads,kv_heads,d,block,layout", PAGED)
def test_paged_attention_matches_64_bits(lens, page, heads, kv_heads, d, block, layout):
    c = Cache(lens, page, kv_heads, d, layout, seed=20, lead=1, tail=2)
    q = rnd((c.rows, heads, d), 21, 2.0)
    o = paged(c, q, None, block)
    check_paged(c, q, o, None, block, "paged")
    for _ in range(2):  # the same every time
        assert same_bits(paged(c, q, None, block), o)


@pytest.mark.parametrize("scale,size", [(1.0, 1.0), (0.5, 6.0), (3.0, 3.0), (1e-4, 1.0)])
def test_paged_attention_with_sharp_and_flat_weights(scale, size):
    c = Cache([(70, 700), (1, 1500)], 16, 4, 64, seed=22)
    q = rnd((c.rows, 8, 64), 23, size)
    check_paged(c, q, paged(c, q, scale, 1), scale, 1, "scaled")


@pytest.mark.parametrize("rising", [True, False])
def test_running_maximum_that_moves(rising):
    # scores that climb (or fall) by thousands over the cache: every tile moves the running maximum
    c = Cache([(60, 1500), (1, 1300)], 32, 2, 64, seed=24)
    for b, (_, kv) in enumerate(c.lens):
        at = torch.arange(kv, device=DEV) if rising else torch.arange(kv - 1, -1, -1, device=DEV)
        c.k[c.slots(b, 0, kv)] = ((at[:, None, None] * 0.05).to(BF16) * torch.ones((1, 2, 64), device=DEV)).to(BF16)
    q = (torch.ones((c.rows, 4, 64), device=DEV) + rnd((c.rows, 4, 64), 25, 0.1)).to(BF16)
    check_paged(c, q, paged(c, q, 1.0, 1), 1.0, 1, "moving")


def test_what_lies_behind_a_sequence_does_not_matter():
    lens = [(40, 333), (1, 65), (1, 1), (150, 150)]
    c = Cache(lens, 48, 2, 80, seed=26)
    q = rnd((c.rows, 6, 80), 27, 2.0)
    clean = paged(c, q, None, 1)
    keep = torch.zeros(c.k.shape[:2], dtype=torch.bool, device=DEV)
    for b, (_, kv) in enumerate(lens):
        keep[c.slots(b, 0, kv)] = True
    for fill in (float("nan"), float("inf"), -float("inf"), 3e38):
        c.k[~keep], c.v[~keep] = fill, fill
        assert same_bits(paged(c, q, None, 1), clean)


def test_nan_and_infinity_within_a_sequence_stay_in_it():
    c = Cache([(3, 300), (3, 300), (3, 300)], 16, 2, 64, seed=28)
    q = rnd((c.rows, 2, 64), 29)
    clean = paged(c, q, None, 0)
    page, slot = c.slots(1, 250, 251)
    c.v[page, slot, 0, 3] = float("nan")
    c.k[page, slot, 1, 3] = float("nan")
    o = paged(c, q, None, 0)
    assert same_bits(o[:3], clean[:3]) and same_bits(o[6:], clean[6:])
    assert bool(o[3:6, 0, 3].isnan().all()) and bool(o[3:6, 1].isnan().all())
    assert not bool(o[3:6, 0, :3].isnan().any())


def test_paged_attention_reports_bad_plans():
    cases = {
        "page": lambda c: c.table[1].fill_(c.k.shape[0]), "negative page": lambda c: c.table[1].fill_(-1),
        "one page": lambda c: c.table[1, 1:2].fill_(2147483647),
        "too long": lambda c: c.kv_lens[1:2].fill_(2147483647), "too short": lambda c: c.kv_lens[1:2].fill_(3),
        "negative": lambda c: c.kv_lens[1:2].fill_(-5),
        "falling": lambda c: c.offsets[2:3].fill_(c.offsets_host[1] - 1),
        "rows": lambda c: c.offsets[3:].fill_(1000000),
    }
    for what, spoil in cases.items():
        c = Cache([(4, 20), (5, 30), (3, 200)], 16, 1, 32, seed=30)
        q = rnd((c.rows, 2, 32), 31)
        spoil(c)
        o, ws = Guarded(tuple(q.shape)), workspace(api.cc_attn_paged_workspace_bytes(c.rows, 3, 2, 1, 32))
        api.cc_attn_paged(q, c.k, c.v, o.t, *c.plan, ws.t)
        with pytest.raises(api.CCError) as e:
            api.cc_check_device()
        assert e.value.status == 5, what
        api.cc_check_device()
        assert o.bands_intact() and ws.bands_intact(), what
        k, v = c.seq(0)  # a good sequence (but for its last row, which a falling offset gives to another one too)
        want, bound = ref.attend(q[:4], k, v, ref.limits(4, 20, 1, DEV), 32 ** -0.5)
        ref.assert_close(o.t[:3], want[:3], bound[:3], what)


def test_offsets_that_pass_32_bits():
    # a cache of more than 2^32 elements, of which the last pages are used
    pages, page, kv_heads, d = 262144 + 64, 16, 8, 128
    k = torch.zeros((pages, page, kv_heads, d), dtype=BF16, device=DEV)
    v = torch.zeros((pages, page, kv_heads, d), dtype=BF16, device=DEV)
    assert k.numel() > 2 ** 32
    lens = [(1, 500), (30, 300)]
    c = Cache(lens, page, kv_heads, d, seed=32, spare=0)
    small_k, small_v, shift = c.k, c.v, pages - c.k.shape[0]
    k[shift:], v[shift:] = small_k, small_v
    q = rnd((c.rows, 8, d), 33, 2.0)
    want = paged(c, q, None, 1)
    c.k, c.v, c.table = k, v, torch.where(c.table >= 0, c.table + shift, c.table)
    assert same_bits(paged(c, q, None, 1), want)
    packed = rnd((c.rows, 24, d), 34)
    api.cc_qk_norm_rope_append(packed[:, :8], packed[:, 8:16], packed[:, 16:], None, None, None, None,
                               torch.empty_like(q), k, v, *c.plan)
    api.cc_check_device()
    at = c.slots(1, 270, 300)
    assert same_bits(v[at[0] + shift, at[1]], packed[1:, 16:]) and not bool(k[:shift].any())


CROSS = [  # n, lq, lk, heads, kv_heads, d, lens
    (1, 1, 1, 1, 1, 16, None), (2, 5, 77, 10, 10, 64, None), (5, 111, 77, 10, 10, 64, [77, 0, 1, 50, 76]),
    (32, 1, 512, 32, 8, 128, None), (3, 300, 513, 12, 4, 96, [513, 128, 129]), (1, 3432, 512, 16, 16, 128, None),
    (4, 257, 1000, 7, 1, 128, [1000, 3, 999, 256]), (2, 50, 0, 2, 2, 32, None), (2, 130, 30, 5, 5, 112, [0, 0]),
    (70, 3, 20, 8, 8, 48, None), (1, 2, 9000, 4, 2, 80, [8999]), (6, 600, 600, 3, 3, 64, [600, 1, 300, 128, 599, 0]),
]


@pytest.mark.parametrize("n,lq,lk,heads,kv_heads,d,lens", CROSS)
def test_cross_attention_matches_64_bits(n, lq, lk, heads, kv_heads, d, lens):
    packed = rnd((n, lk, 2 * kv_heads, d), 40)
    k, v = packed[:, :, :kv_heads], packed[:, :, kv_heads:]
    q = rnd((n, lq, heads + 1, d), 41, 2.0)[:, :, :heads]  # rows at a stride
    for b, length in enumerate(lens or []):
        packed[b, length:] = float("nan")  # padding may hold anything
    o, ws = Guarded((n, lq, heads, d)), workspace(api.cc_attn_cross_workspace_bytes(n, lq, lk, heads, kv_heads, d))
    api.cc_attn_cross(q, k, v, o.t, ints(lens) if lens else None, ws.t)
    api.cc_check_device()
    assert o.bands_intact() and ws.bands_intact()
    first = o.t.clone()
    for b in range(n):
        length = lens[b] if lens else lk
        limit = torch.full((lq,), length, device=DEV)
        ref.assert_close(first[b], *ref.attend(q[b], k[b, :length], v[b, :length], limit, d ** -0.5), f"instance {b}")
    api.cc_attn_cross(q, k, v, o.t, ints(lens) if lens else None, ws.t)
    assert same_bits(o.t, first)


def test_cross_attention_takes_bad_lengths_as_the_nearest():
    q, k, v = rnd((3, 4, 2, 32), 42), rnd((3, 40, 2, 32), 43), rnd((3, 40, 2, 32), 44)
    o, ws = Guarded((3, 4, 2, 32)), workspace(api.cc_attn_cross_workspace_bytes(3, 4, 40, 2, 2, 32))
    api.cc_attn_cross(q, k, v, o.t, ints([41, -1, 2147483647]), ws.t)
    with pytest.raises(api.CCError) as e:
        api.cc_check_device()
    assert e.value.status == 5 and o.bands_intact() and ws.bands_intact()
    want = torch.empty_like(q)
    api.cc_attn_cross(q, k, v, want, ints([40, 0, 40]), ws.t)
    api.cc_check_device()
    assert same_bits(o.t, want) and not bool(want[1].any())


# -------------------------------------------------------------------------------------------------------- together --

class Block:
    """A decoder block's attention half, chunk after chunk: q, k, v projected in 8 bits, normed, rotated and
    appended; attention over the cache; projection with the residual; attention to a text; the same again."""

    def __init__(self, seed=60, seqs=2, chunk=96, chunks=3, c=256, heads=4, page=32, text=50):
        self.c, self.heads, self.d, self.chunk, self.seqs = c, heads, c // heads, chunk, seqs
        self.page, self.per = page, -(-chunk * chunks // page)
        pages = seqs * self.per
        self.k, self.v = (torch.zeros((pages, page, heads, self.d), dtype=BF16, device=DEV) for _ in range(2))
        self.table = torch.randperm(pages, generator=gen(seed), device=DEV).to(I32).view(seqs, self.per)
        self.offsets, self.lens = ints([chunk * b for b in range(seqs + 1)]), ints([0] * seqs)
        self.rot = rot_table(chunk * chunks, self.d)
        self.w = [rnd((c, c), seed + 1 + i, c ** -0.5) for i in range(7)]  # q k v o, q2 o2 and the text's
        self.text = rnd((seqs, text, c), seed + 20)
        self.text_lens = ints([text, text // 2])
        self.gq, self.gk = rnd((self.d,), seed + 21, 0.2, 1.0), rnd((self.d,), seed + 22, 0.2, 1.0)
        nb = -(-c // 128)
        self.wq = [torch.empty((c, c), dtype=torch.float8_e4m3fn, device=DEV) for _ in self.w]
        self.sw = [torch.empty((nb, nb), device=DEV) for _ in self.w]
        for w, q, s in zip(self.w, self.wq, self.sw):
            api.cc_gemm_fp8_prepare(w, q, s)
        rows = seqs * chunk
        self.x, self.y = (torch.zeros((rows, c), dtype=BF16, device=DEV) for _ in range(2))
        self.h8, self.s8 = torch.empty((rows, c), dtype=torch.float8_e4m3fn, device=DEV), torch.empty((rows, nb), device=DEV)
        self.qkv = torch.empty((rows, 3, heads, self.d), dtype=BF16, device=DEV)
        self.q, self.o = (torch.empty((rows, heads, self.d), dtype=BF16, device=DEV) for _ in range(2))
        self.mid = torch.empty((rows, c), dtype=BF16, device=DEV)
        self.tk, self.tv = (torch.empty((seqs, text, heads, self.d), dtype=BF16, device=DEV) for _ in range(2))
        t8, ts = torch.empty((seqs, text, c), dtype=torch.float8_e4m3fn, device=DEV), torch.empty((seqs, text, nb), device=DEV)
        api.cc_fp8_quantize(self.text, t8, ts)
        for i, out in ((4, self.tk), (5, self.tv)):
            api.cc_gemm_fp8(t8, ts, self.wq[i], self.sw[i], None, None, out.view(seqs, text, c))
        need = max(api.cc_attn_paged_workspace_bytes(rows, seqs, heads, heads, self.d),
                   api.cc_attn_cross_workspace_bytes(seqs, chunk, text, heads, heads, self.d))
        self.ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def step(self, stream=None):
        rows, c, flat = self.x.shape[0], self.c, lambda t: t.view(-1, self.c)
        api.cc_rms_norm_act_fp8(self.x, None, self.h8, self.s8, act="none", stream=stream)
        for i in range(3):
            api.cc_gemm_fp8(self.h8, self.s8, self.wq[i], self.sw[i], None, None,
                            self.qkv.view(rows, 3 * c)[:, i * c:(i + 1) * c], stream=stream)
        api.cc_qk_norm_rope_append(self.qkv[:, 0], self.qkv[:, 1], self.qkv[:, 2], self.gq, self.gk, self.rot, None,
                                   self.q, self.k, self.v, self.offsets, self.lens, self.table, stream=stream)
        api.cc_attn_paged(self.q, self.k, self.v, self.o, self.offsets, self.lens, self.table, self.ws,
                          causal_block=self.chunk // 2, stream=stream)
        api.cc_fp8_quantize(flat(self.o), self.h8, self.s8, stream=stream)
        api.cc_gemm_fp8(self.h8, self.s8, self.wq[3], self.sw[3], None, self.x, self.mid, stream=stream)
        # the text's half
        api.cc_rms_norm_act_fp8(self.mid, None, self.h8, self.s8, act="none", stream=stream)
        api.cc_gemm_fp8(self.h8, self.s8, self.wq[6], self.sw[6], None, None, flat(self.q), stream=stream)
        api.cc_qk_norm_rope(self.q, None, self.gq, None, None, None, self.q, None, stream=stream)
        shape = (self.seqs, self.chunk, self.heads, self.d)
        api.cc_attn_cross(self.q.view(shape), self.tk, self.tv, self.o.view(shape), self.text_lens, self.ws,
                          stream=stream)
        api.cc_fp8_quantize(flat(self.o), self.h8, self.s8, stream=stream)
        api.cc_gemm_fp8(self.h8, self.s8, self.wq[3], self.sw[3], None, self.mid, self.y, stream=stream)

    def run(self, i, seed=80, stream=None, step=None):
        self.x.copy_(rnd(tuple(self.x.shape), seed + i))
        self.lens.fill_(self.chunk * (i + 1))
        (step or self.step)(**({} if step else {"stream": stream}))


def test_chunks_of_a_block_run_together():
    blk, d = Block(), 64
    rows = blk.x.shape[0]
    keys = [[] for _ in range(blk.seqs)]
    values = [[] for _ in range(blk.seqs)]
    for i in range(3):
        blk.run(i)
        api.cc_check_device()
        # each operator on what the ones in front of it left: the cache holds every chunk so far ...
        pos = (torch.arange(blk.chunk) + i * blk.chunk).repeat(blk.seqs)
        want_k = ref.rotated(blk.qkv[:, 1], blk.gk, blk.rot, pos, 1e-6, "pairs")
        for b in range(blk.seqs):
            r = slice(b * blk.chunk, (b + 1) * blk.chunk)
            at = torch.arange(i * blk.chunk, (i + 1) * blk.chunk, device=DEV)
            page, slot = blk.table[b].long()[at // blk.page], at % blk.page
            ref.assert_close(blk.k[page, slot], want_k[0][r], want_k[1][r], f"chunk {i}")
            assert same_bits(blk.v[page, slot], blk.qkv[r, 2])
            keys[b].append(blk.k[page, slot].clone())
            values[b].append(blk.v[page, slot].clone())
        # ... the text's attention follows from its queries, and the block's output from it
        q = blk.q.view(blk.seqs, blk.chunk, blk.heads, d)
        for b, length in enumerate(blk.text_lens.tolist()):
            limit = torch.full((blk.chunk,), length, device=DEV)
            ref.assert_close(blk.o.view(q.shape)[b], *ref.attend(q[b], blk.tk[b, :length], blk.tv[b, :length], limit,
                                                                d ** -0.5), f"text {i}")
    # the attention over all three chunks, from the cache as it was filled
    o = torch.empty_like(blk.o)
    q = ref.rotated(blk.qkv[:, 0], blk.gq, blk.rot, pos, 1e-6, "pairs")[0].to(BF16)
    api.cc_attn_paged(q, blk.k, blk.v, o, blk.offsets, blk.lens, blk.table, blk.ws, causal_block=blk.chunk // 2)
    for b in range(blk.seqs):
        r = slice(b * blk.chunk, (b + 1) * blk.chunk)
        limit = ref.limits(blk.chunk, 3 * blk.chunk, blk.chunk // 2, DEV)
        ref.assert_close(o[r], *ref.attend(q[r], torch.cat(keys[b]), torch.cat(values[b]), limit, d ** -0.5), f"all {b}")
    assert rows == blk.y.shape[0] and bool(blk.y.isfinite().all())


def test_a_block_replays_from_a_graph_while_the_plan_grows():
    eager, blk = Block(), Block()
    want = []
    for i in range(3):
        eager.run(i)
        want.append(eager.y.clone())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        blk.run(0)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk.step()
    for i in range(3):  # one graph for all lengths: they are read on the device
        blk.y.zero_()
        blk.run(i, step=graph.replay)
        torch.cuda.synchronize()
        assert same_bits(blk.y, want[i]), f"chunk {i}"
    api.cc_check_device()


def test_blocks_on_two_streams_and_from_two_graphs():
    blocks = [Block(seed=60 + 100 * i) for i in range(4)]
    want = []
    for i in range(2):
        ref_block = Block(seed=60 + 100 * i)
        for j in range(3):
            ref_block.run(j, seed=80 + i)
        want.append(ref_block.y.clone())
    for i in range(2):
        blocks[2 + i] = Block(seed=60 + 100 * i)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            blocks[2 + i].step()
        graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for j in range(3):
        for i in range(4):
            with torch.cuda.stream(streams[i]):
                if i < 2:
                    blocks[i].run(j, seed=80 + i, stream=streams[i])
                else:
                    blocks[i].run(j, seed=80 + i - 2, step=graphs[i - 2].replay)
    torch.cuda.synchronize()
    api.cc_check_device()
    for i in range(4):
        assert same_bits(blocks[i].y, want[i % 2]), i


def test_two_graphs_with_one_workspace_one_after_the_other():
    cases = [Cache([(1, 30000)], 16, 2, 128, seed=90), Cache([(300, 1200), (1, 9000)], 32, 2, 128, seed=92)]
    q = [rnd((c.rows, 8, 128), 94 + i, 2.0) for i, c in enumerate(cases)]
    o = [torch.empty_like(t) for t in q]
    need = max(api.cc_attn_paged_workspace_bytes(c.rows, len(c.lens), 8, 2, 128) for c in cases)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    want, graphs = [], []
    for c, qi, oi in zip(cases, q, o):
        api.cc_attn_paged(qi, c.k, c.v, oi, *c.plan, ws)
        torch.cuda.synchronize()
        want.append(oi.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.cc_attn_paged(qi, c.k, c.v, oi, *c.plan, ws)
        graphs.append(g)
    for _ in range(3):
        ws.fill_(0xFF)
        for oi in o:
            oi.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(o, want))
    api.cc_check_device()
