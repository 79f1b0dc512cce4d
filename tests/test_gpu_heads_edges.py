"""The attentions with heads at the borders of their variants: both sides of the rule for few rows, outputs whose rows
start anywhere, many sequences of several items, items cut into many pieces, blocks of any size, pages and lengths that
sequences share, single tokens step by step and from graphs, calls side by side on streams."""

import pytest
import torch

import heads_ref as ref
from causal_convolution_gb300 import api
from gpu_util import ensure_built
from test_gpu_guard_bands import Guarded
from test_gpu_heads import BF16, DEV, Cache, check_paged, ints, paged, rnd, rot_table, same_bits, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    return ensure_built()


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("group,lens", [
    (1, [(8, 8), (8, 200), (8, 65), (8, 1000)]),      # eight rows to a sequence: the most of the variant for few
    (1, [(9, 9), (8, 200), (8, 65), (8, 1000)]),      # one more
    (1, [(20, 700), (0, 3), (2, 64), (5, 6), (1, 1)]),  # few on average only: several items to a sequence
    (3, [(2, 300), (3, 3), (1, 640), (4, 129)]),      # tokens of three heads: two of them to an item, and two rows idle
    (5, [(1, 385), (2, 2), (1, 63)]), (7, [(1, 257), (1, 1), (1, 64)]), (8, [(1, 2000), (1, 33)]),
    (8, [(2, 2000), (1, 33)]), (9, [(1, 500), (1, 1)]),
])
def test_both_sides_of_the_rule_for_few_rows(group, lens, d):
    c = Cache(lens, 16, 2, d, "joint" if d % 32 else "heads", seed=100, lead=3, tail=1)
    q = rnd((c.rows, 2 * group, d), 101, 2.0)
    for block in (1, 0, 3):
        o = paged(c, q, None, block)
        check_paged(c, q, o, None, block, f"block {block}")


@pytest.mark.parametrize("lens", [[(1, 900), (1, 50)], [(150, 900), (3, 50)], [(40, 7000)]])
@pytest.mark.parametrize("shift,extra", [(8, 0), (0, 8), (8, 8)])
def test_outputs_whose_rows_start_on_any_16_bytes(lens, shift, extra):
    c = Cache(lens, 48, 3, 80, seed=102)
    q = rnd((c.rows, 6, 80), 103, 2.0)
    want = paged(c, q, None, 1)
    wide = Guarded((c.rows, 480 + extra + shift))
    wide.t.fill_(7.0)
    o = wide.t[:, shift:shift + 480].unflatten(1, (6, 80))
    api.cc_attn_paged(q, c.k, c.v, o, *c.plan, workspace(api.cc_attn_paged_workspace_bytes(c.rows, len(lens), 6, 3, 80)).t)
    api.cc_check_device()
    assert same_bits(o, want) and wide.bands_intact()
    assert bool((wide.t[:, :shift] == 7.0).all()) and bool((wide.t[:, shift + 480:] == 7.0).all())


def test_many_sequences_of_several_items():
    lens = [(1 + 71 * b % 400, 400 + 13 * b) for b in range(75)]
    c = Cache(lens, 32, 1, 64, seed=104, lead=1, tail=5)
    q = rnd((c.rows, 3, 64), 105, 2.0)
    for block in (1, 90):
        check_paged(c, q, paged(c, q, None, block), None, block, f"block {block}")


@pytest.mark.parametrize("new,heads,kv_heads,d", [(1, 1, 1, 128), (1, 8, 1, 64), (8, 1, 1, 96), (1, 16, 1, 128),
                                                  (16, 16, 1, 128), (130, 2, 1, 64), (3, 7, 1, 16)])
def test_one_sequence_cut_over_all_of_the_grid(new, heads, kv_heads, d):
    c = Cache([(new, 61001)], 16, kv_heads, d, seed=106)
    q = rnd((new, heads, d), 107, 3.0)
    o = paged(c, q, None, 1)
    check_paged(c, q, o, None, 1, "cut")
    assert same_bits(paged(c, q, None, 1), o)


@pytest.mark.parametrize("block", [1 << 30, 2 ** 31 - 1, 333])
def test_blocks_larger_than_the_chunk(block):
    c = Cache([(333, 500), (1, 70), (20, 20)], 16, 2, 32, seed=108)
    q = rnd((c.rows, 4, 32), 109, 2.0)
    assert same_bits(paged(c, q, None, block), paged(c, q, None, 0))


def test_sequences_share_pages_and_a_table_names_one_twice():
    c = Cache([(2, 200), (70, 200), (1, 200)], 16, 2, 64, seed=110)
    c.table_host[1][:10] = c.table_host[0][:10]  # a shared prefix
    c.table_host[2][:12] = c.table_host[2][:1] * 12
    c.table = ints(c.table_host)
    q = rnd((c.rows, 4, 64), 111, 2.0)
    check_paged(c, q, paged(c, q, None, 1), None, 1, "shared")


def test_plans_without_work():
    # no sequence has new tokens, none has any keys, and no rows at all: nothing is written but zeros where rows see none
    c = Cache([(0, 100), (0, 0)], 16, 2, 64, seed=112, lead=2, tail=2)
    q = rnd((c.rows, 4, 64), 113)
    assert bool((paged(c, q, None, 1) == 7.0).all())
    c = Cache([(3, 0), (200, 0)], 16, 2, 64, seed=114)
    o = paged(c, rnd((c.rows, 4, 64), 115), None, 0)
    assert not bool(o.any())
    empty = torch.empty((0, 4, 64), dtype=BF16, device=DEV)
    api.cc_attn_paged(empty, c.k, c.v, empty, *c.plan, None)
    api.cc_attn_cross(empty[None], rnd((1, 5, 2, 64), 116), rnd((1, 5, 2, 64), 117), empty[None], None, None)
    api.cc_check_device()


@pytest.mark.parametrize("new", [130, 3])
def test_infinite_scores(new):
    # a key whose scores are +inf gives NaN, one of -inf weighs nothing, a row of nothing but -inf is NaN: as the formula
    c = Cache([(1, 150), (1, 150), (1, 150), (new, 150), (1, 150)], 16, 1, 16, seed=118)
    q = rnd((c.rows, 1, 16), 119).abs() + 0.5
    inf = float("inf")
    c.k[(*c.slots(0, 70, 71), 0, 3)] = inf
    c.k[(*c.slots(1, 70, 71), 0, 3)] = -inf
    c.k[(*c.slots(2, 0, 150), 0, 3)] = -inf
    c.k[(*c.slots(3, 0, 100), 0, 3)] = -inf
    o = paged(c, q, None, 1)
    assert bool(o[0].isnan().all()) and bool(o[2].isnan().all())
    keep = torch.arange(150, device=DEV) != 70
    k, v = c.seq(1)
    limit = torch.full((1,), 149, device=DEV)
    ref.assert_close(o[1:2], *ref.attend(q[1:2], k[keep], v[keep], limit, 0.25), "-inf")
    k, v = c.seq(3)
    rows, sees = o[3:3 + new], torch.arange(151 - new, 151, device=DEV)
    assert bool(rows[sees <= 100].isnan().all())
    ref.assert_close(rows[sees > 100], *ref.attend(q[3:3 + new][sees > 100], k[100:], v[100:], sees[sees > 100] - 100, 0.25),
                     "late")
    ref.assert_close(o[3 + new:], *ref.attend(q[3 + new:], *c.seq(4), limit + 1, 0.25), "finite")


class Decoder:
    """Single tokens, step by step: norm, rotation and append, then attention over the cache."""

    def __init__(self, seed, seqs=5, heads=8, kv_heads=2, d=64, page=16, most=300):
        self.seqs, self.heads, self.kv_heads, self.d, self.page = seqs, heads, kv_heads, d, page
        per = -(-most // page)
        self.k, self.v = (torch.full((seqs * per, page, kv_heads, d), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
        self.table = torch.randperm(seqs * per, generator=torch.Generator().manual_seed(seed)).view(seqs, per)
        self.rot, self.gamma = rot_table(most, d), rnd((d,), seed, 0.2, 1.0)
        self.plan = ints(list(range(seqs + 1))), ints([0] * seqs), self.table.to(torch.int32).to(DEV)
        self.x = torch.empty((seqs, heads + 2 * kv_heads, d), dtype=BF16, device=DEV)
        self.q, self.o = (torch.empty((seqs, heads, d), dtype=BF16, device=DEV) for _ in range(2))
        self.ws = torch.empty(api.cc_attn_paged_workspace_bytes(seqs, seqs, heads, kv_heads, d), dtype=torch.uint8, device=DEV)

    def step(self, stream=None):
        h, kv = self.heads, self.kv_heads
        api.cc_qk_norm_rope_append(self.x[:, :h], self.x[:, h:h + kv], self.x[:, h + kv:], self.gamma, self.gamma, self.rot,
                                   None, self.q, self.k, self.v, *self.plan, style="halves", stream=stream)
        api.cc_attn_paged(self.q, self.k, self.v, self.o, *self.plan, self.ws, stream=stream)

    def inputs(self, step, seed):
        self.x.copy_(rnd(tuple(self.x.shape), 1000 * seed + step))
        self.plan[1].copy_(ints([step + 1 + 50 * (b > 0) * (step > 3) for b in range(self.seqs)]))


def test_single_tokens_step_by_step():
    dec, past = Decoder(120, seqs=1), []
    for step in range(200):
        dec.inputs(step, 1)
        dec.step()
        past.append(dec.x.clone())
        if step in (0, 1, 15, 16, 63, 64, 150, 199):
            api.cc_check_device()
            x, pos = torch.cat(past), torch.arange(step + 1)
            k, bound = ref.rotated(x[:, 8:10], dec.gamma, dec.rot, pos, 1e-6, "halves")
            at = dec.table[0][pos // dec.page].to(DEV), (pos % dec.page).to(DEV)
            ref.assert_close(dec.k[at], k, bound, f"keys at {step}")
            limit = torch.full((1,), step + 1, device=DEV)
            ref.assert_close(dec.o, *ref.attend(dec.q, dec.k[at], x[:, 10:], limit, dec.d ** -0.5), f"step {step}")


def test_single_tokens_from_graphs_beside_chunks_on_other_streams():
    chunk = Cache([(300, 900), (64, 3000)], 32, 2, 128, seed=121)
    cq = rnd((chunk.rows, 8, 128), 122, 2.0)
    want_chunk = paged(chunk, cq, None, 1)
    plain, want = Decoder(123), []
    plain.k.zero_(), plain.v.zero_()
    for step in range(8):
        plain.inputs(step, 2)
        plain.step()
        want.append(plain.o.clone())
    decs, graphs = [Decoder(123) for _ in range(2)], []
    for dec in decs:
        dec.k.zero_(), dec.v.zero_()
        graph = torch.cuda.CUDAGraph()
        dec.inputs(0, 2)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            dec.step()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    co = torch.empty_like(cq)
    cws = torch.empty(api.cc_attn_paged_workspace_bytes(chunk.rows, 2, 8, 2, 128), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for step in range(8):
        for dec, graph, stream in zip(decs, graphs, streams):
            with torch.cuda.stream(stream):
                dec.inputs(step, 2)
                graph.replay()
        api.cc_attn_paged(cq, chunk.k, chunk.v, co, *chunk.plan, cws, stream=streams[2])
        torch.cuda.synchronize()
        assert same_bits(co, want_chunk) and all(same_bits(dec.o, want[step]) for dec in decs), step
    api.cc_check_device()


@pytest.mark.parametrize("n,lq,lk,heads,kv_heads,d,lens", [
    (3, 8, 700, 4, 4, 64, [700, 0, 333]), (3, 9, 700, 4, 4, 64, [700, 0, 333]),  # both sides of the rule for few rows
    (2, 4, 1300, 6, 3, 112, None), (40, 1, 513, 8, 1, 16, None), (1, 1, 100000, 1, 1, 128, [99999]),
    (1, 500, 20000, 1, 1, 96, [19999]), (35, 300, 130, 2, 2, 32, [(7 * b) % 131 for b in range(35)]),
])
def test_cross_attention_at_the_borders(n, lq, lk, heads, kv_heads, d, lens):
    q, k, v = rnd((n, lq, heads, d), 130, 2.0), rnd((n, lk, kv_heads, d), 131), rnd((n, lk, kv_heads, d), 132)
    for b, length in enumerate(lens or []):
        k[b, length:], v[b, length:] = float("nan"), float("inf")
    o = Guarded((n, lq, heads, d))
    ws = workspace(api.cc_attn_cross_workspace_bytes(n, lq, lk, heads, kv_heads, d))
    api.cc_attn_cross(q, k, v, o.t, ints(lens) if lens else None, ws.t, scale=0.2)
    api.cc_check_device()
    assert o.bands_intact() and ws.bands_intact()
    for b in range(n):
        length = lens[b] if lens else lk
        limit = torch.full((lq,), length, device=DEV)
        ref.assert_close(o.t[b], *ref.attend(q[b], k[b, :length], v[b, :length], limit, 0.2), f"instance {b}")


def test_the_largest_heads_and_groups():
    # 128 query heads to a key head, 16 key heads: an item is two tokens
    c = Cache([(5, 1000), (2, 31)], 16, 16, 128, seed=133)
    q = rnd((c.rows, 2048, 128), 134, 2.0)
    check_paged(c, q, paged(c, q, None, 1), None, 1, "wide")
    x = rnd((3, 2048 + 16, 256), 135)
    qo, ko = Guarded((3, 2048, 256)), Guarded((3, 16, 256))
    rot = rot_table(3, 256)
    api.cc_qk_norm_rope(x[:, :2048], x[:, 2048:], None, None, rot, None, qo.t, ko.t)
    api.cc_check_device()
    assert qo.bands_intact() and ko.bands_intact()
    ref.assert_close(qo.t, *ref.rotated(x[:, :2048], None, rot, [0, 1, 2], 1e-6, "pairs"), "q")
    ref.assert_close(ko.t, *ref.rotated(x[:, 2048:], None, rot, [0, 1, 2], 1e-6, "pairs"), "k")


@pytest.mark.parametrize("lens", [[(1, 700), (1, 33)], [(200, 700), (9, 33)]])
def test_keys_and_values_of_different_layouts(lens):
    c = Cache(lens, 48, 2, 96, "plain", seed=140)
    q = rnd((c.rows, 4, 96), 141, 2.0)
    want = paged(c, q, None, 1)
    c.v = c.v.transpose(1, 2).contiguous().transpose(1, 2)     # a head's tokens side by side
    wide = rnd((*c.k.shape[:3], 200), 142)
    wide[..., 16:112] = c.k
    c.k = wide[..., 16:112]                                    # channels of wider rows
    assert same_bits(paged(c, q, None, 1), want)


@pytest.mark.parametrize("page", [16 * 37, 4096])
def test_large_pages(page):
    for lens in ([(1, 5000), (1, 4096), (1, 1)], [(300, 5000), (130, 4097)]):
        c = Cache(lens, page, 1, 48, "heads", seed=143)
        q = rnd((c.rows, 3, 48), 144, 2.0)
        check_paged(c, q, paged(c, q, None, 1), None, 1, "large pages")


@pytest.mark.parametrize("new", [2, 150])
def test_queries_that_are_not_numbers_stay_alone(new):
    c = Cache([(new, 600), (1, 600)], 16, 2, 64, seed=145)
    q = rnd((c.rows, 4, 64), 146, 2.0)
    q[0, 1, 7], q[1, 2, 3] = float("nan"), float("inf")
    o = paged(c, q, None, 1)
    assert bool(o[0, 1].isnan().all()) and bool(o[1, 2].isnan().all())
    k, v = c.seq(0)
    want, bound = ref.attend(q[:new].nan_to_num(0, 0, 0), k, v, ref.limits(new, 600, 1, DEV), 0.125)
    keep = torch.ones((new, 4), dtype=torch.bool, device=DEV)
    keep[0, 1] = keep[1, 2] = False
    ref.assert_close(o[:new][keep], want[keep], bound[keep], "the others")
    ref.assert_close(o[new:], *ref.attend(q[new:], *c.seq(1), ref.limits(1, 600, 1, DEV), 0.125), "another sequence")
