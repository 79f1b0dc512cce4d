"""What the operators with heads refuse, on the host: by the C entry points' argument checks and by the binding's checks
of shapes. Nothing here reaches a device."""

import ctypes
import os

import pytest
import torch

from causal_convolution_gb300 import _lib, api
from test_norm_fp8_shapes_host import BF16, F32, Calls, t

F = ctypes.c_float
I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from causal_convolution_gb300 import build
        build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(1 << 12)
    p.keep = buf
    return (ctypes.addressof(buf) + 15) // 16 * 16


@pytest.fixture
def calls(monkeypatch):
    calls = Calls()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(api, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(_lib, "load", lambda: calls)
    return calls


ROPE = ["q", "k", "gamma_q", "gamma_k", "rot", "pos", "q_out", "k_out", "rows", "heads", "kv_heads", "d", "rd",
        "positions", "ld_q", "ld_k", "ld_qo", "ld_ko", "eps", "style", "stream"]
APPEND = ["q", "k", "v", "gamma_q", "gamma_k", "rot", "pos", "q_out", "k_cache", "v_cache", "q_offsets", "kv_lens",
          "page_table", "rows", "seqs", "max_pages", "pages", "page_size", "heads", "kv_heads", "d", "rd", "positions",
          "ld_q", "ld_k", "ld_v", "ld_qo", "k_page", "k_token", "k_head", "v_page", "v_token", "v_head", "eps", "style",
          "stream"]
PAGED = ["q", "k_cache", "v_cache", "o", "q_offsets", "kv_lens", "page_table", "rows", "seqs", "max_pages", "pages",
         "page_size", "heads", "kv_heads", "d", "ld_q", "ld_o", "k_page", "k_token", "k_head", "v_page", "v_token",
         "v_head", "scale", "causal_block", "ws", "ws_bytes", "stream"]
CROSS = ["q", "k", "v", "o", "kv_lens", "n", "lq", "lk", "heads", "kv_heads", "d", "ld_q", "ld_k", "ld_v", "ld_o",
         "scale", "ws", "ws_bytes", "stream"]
SIZES = dict(rows=4, seqs=2, max_pages=3, pages=7, page_size=16, heads=4, kv_heads=2, d=64, rd=64, positions=9,
             ld_q=256, ld_k=128, ld_v=128, ld_qo=256, ld_ko=128, ld_o=256, k_page=2048, k_token=128, k_head=64,
             v_page=2048, v_token=128, v_head=64, eps=1e-6, style=0, scale=0.125, causal_block=1, ws_bytes=1 << 40,
             stream=None, n=2, lq=2, lk=5)


def call(lib, name, names, p, **changes):
    values = [changes.get(n, SIZES.get(n, p)) for n in names]
    return getattr(lib, name)(*values), lib.cc_last_error().decode()


def refusals(lib, p, name, names, cases):
    for changes, status, text in cases:
        st, msg = call(lib, name, names, p, **changes)
        assert st == status and text in msg, (name, changes, st, msg)


NULLS = "null"


def test_norm_and_rotation_refusals(lib, p):
    shared = [({n: None}, 1, NULLS) for n in ("q", "k", "q_out")] + [
        (dict(gamma_q=p + 2), 1, "aligned"), (dict(rot=p + 8), 1, "aligned"), (dict(q=p + 4), 1, "aligned"),
        (dict(heads=-1), 1, "negative"), (dict(d=0), 1, "positive"), (dict(d=72, rd=64), 2, "multiple of 16"),
        (dict(d=272, ld_q=2000), 2, "256"), (dict(rd=-16), 1, "rotated"), (dict(rd=8), 1, "rotated"),
        (dict(rd=80), 1, "rotated"), (dict(rot=None), 1, "table"), (dict(positions=0), 1, "table"),
        (dict(ld_q=248), 1, "strides"), (dict(ld_q=260), 1, "strides"), (dict(ld_k=120), 1, "strides"),
        (dict(ld_qo=248), 1, "strides"), (dict(eps=0.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
        (dict(style=2), 1, "style"), (dict(rows=-1), 1, "negative"),
        (dict(heads=65537, ld_q=1 << 23, ld_qo=1 << 23), 2, "65536")]
    refusals(lib, p, "cc_qk_norm_rope", ROPE, shared + [
        (dict(k_out=None), 1, NULLS), (dict(ld_ko=120), 1, "strides"), (dict(ld_ko=132), 1, "strides"),
        (dict(pos=None, rows=10), 1, "positions"), (dict(heads=0, kv_heads=0), 1, "positive")])
    refusals(lib, p, "cc_qk_norm_rope_append", APPEND, shared + PLAN + [
        (dict(v=None), 1, NULLS), (dict(v_cache=None), 1, NULLS), (dict(v=p + 8), 1, "aligned"),
        (dict(ld_v=120), 1, "strides"), (dict(kv_heads=0), 1, "at least one head")])
    assert call(lib, "cc_qk_norm_rope", ROPE, None, rows=0)[0] == 0
    assert call(lib, "cc_qk_norm_rope_append", APPEND, None, rows=0)[0] == 0
    assert call(lib, "cc_qk_norm_rope_append", APPEND, None, seqs=0)[0] == 0


PLAN = [({n: None}, 1, NULLS) for n in ("q_offsets", "kv_lens", "page_table", "k_cache")] + [
    (dict(kv_lens=4), 1, "aligned"), (dict(max_pages=0), 1, "positive"), (dict(pages=0), 1, "positive"),
    (dict(page_size=0), 1, "positive"), (dict(page_size=24), 2, "multiple of 16"),
    (dict(pages=1 << 28), 2, "2^31"), (dict(k_page=56), 1, "strides"), (dict(k_token=68), 1, "strides"),
    (dict(v_head=56), 1, "strides"), (dict(v_page=1 << 38), 2, "2^38"), (dict(seqs=-1), 1, "negative")]
ATTN = [({n: None}, 1, NULLS) for n in ("q", "o")] + [
    (dict(q=8), 1, "aligned"), (dict(heads=3), 1, "multiple"), (dict(heads=0), 1, "multiple"),
    (dict(kv_heads=-2), 1, "multiple"), (dict(d=0), 1, "multiple"), (dict(d=72, ld_q=288, ld_o=288), 2, "multiple of 16"),
    (dict(d=144, ld_q=576, ld_o=576), 2, "128"), (dict(ld_q=248), 1, "strides"), (dict(ld_o=260), 1, "strides"),
    (dict(heads=258, ld_q=1 << 15, ld_o=1 << 15), 2, "128 to a key head"), (dict(scale=0.0), 1, "scale"),
    (dict(scale=-1.0), 1, "scale"), (dict(scale=float("inf")), 1, "scale"), (dict(scale=float("nan")), 1, "scale")]


def test_attention_refusals(lib, p):
    refusals(lib, p, "cc_attn_paged", PAGED, ATTN + PLAN + [
        (dict(rows=-1), 1, "negative"), (dict(rows=(1 << 30) + 1), 2, "2^30"), (dict(causal_block=-1), 1, "causal block"), (dict(v_cache=None), 1, NULLS)])
    refusals(lib, p, "cc_attn_cross", CROSS, ATTN + [
        (dict(k=None), 1, NULLS), (dict(v=None), 1, NULLS), (dict(n=-1), 1, "negative"), (dict(lq=-1), 1, "negative"),
        (dict(lk=-1), 1, "negative"), (dict(kv_lens=8), 1, "aligned"), (dict(ld_k=120), 1, "strides"),
        (dict(ld_v=132), 1, "strides"), (dict(n=1 << 16, lq=1 << 16), 2, "2^30")])
    assert call(lib, "cc_attn_paged", PAGED, None, rows=0)[0] == 0
    assert call(lib, "cc_attn_paged", PAGED, None, seqs=0)[0] == 0
    assert call(lib, "cc_attn_cross", CROSS, None, n=0)[0] == 0
    assert call(lib, "cc_attn_cross", CROSS, None, lq=0)[0] == 0


def test_attention_workspaces(lib, p):
    paged, cross = lib.cc_attn_paged_workspace_bytes, lib.cc_attn_cross_workspace_bytes
    part = lambda slots, rows, d: slots * (rows * (4 * d + 8) + 16)  # sums, (c, l) and a directory entry to a slot
    assert paged(1, 1, 8, 1, 128) == part(608, 8, 128)          # few rows: eight to a slot, two CTAs to an SM
    assert paged(2, 1, 8, 1, 128) == part(304, 16, 128)
    assert paged(1, 1, 9, 1, 64) == part(304, 9, 64)
    assert paged(1000, 2, 9, 1, 64) == part(304, 256, 64)
    assert cross(2, 9, 1537, 4, 4, 48) == part(304, 9, 48)
    assert cross(2, 9, 1536, 4, 4, 48) == 0                     # nothing is cut
    assert cross(2, 8, 769, 4, 4, 48) == part(608, 8, 48) and cross(2, 8, 768, 4, 4, 48) == 0
    assert cross(2, 8, 385, 4, 4, 80) == part(608, 8, 80) and cross(2, 8, 384, 4, 4, 80) == 0
    for sizes in ((0, 1, 8, 1, 64), (1, 0, 8, 1, 64), (-1, 1, 8, 1, 64), (1, 1, 3, 2, 64), (1, 1, 8, 0, 64),
                  (1, 1, 129, 1, 64), (1, 1, 8, 1, 72), (1, 1, 8, 1, 144), (1, 1, 8, 1, 0)):
        assert paged(*sizes) == 0
    assert cross(0, 1, 999, 1, 1, 64) == 0 and cross(1, -1, 999, 1, 1, 64) == 0
    need = paged(4, 2, 4, 2, 64)
    many = dict(max_pages=97)  # 1552 keys: tiles enough to cut
    refusals(lib, p, "cc_attn_paged", PAGED, [
        (dict(ws=None, **many), 1, "null workspace"), (dict(ws=p + 8, **many), 1, "aligned"),
        (dict(ws_bytes=need - 1, **many), 1, "workspace of"), (dict(ws_bytes=0, **many), 1, "workspace of"),
        (dict(rows=1 << 30, max_pages=1 << 20), 2, "2^31 tiles")])
    refusals(lib, p, "cc_attn_cross", CROSS, [
        (dict(ws=None, lk=769), 1, "null workspace"), (dict(ws_bytes=8, lk=769), 1, "workspace of"),
        (dict(n=1 << 15, lq=1 << 15, lk=1 << 20), 2, "2^31 tiles"), (dict(ld_k=1 << 30, lk=1 << 10), 2, "2^38")])


# ------------------------------------------------------------------------------------------------------- binding --

def i32(*shape):
    return t(*shape, dtype=I32)


def cache(pages=7, page=16, heads=2, d=64):
    return t(pages, page, heads, d)


def test_binding_passes_shapes_and_strides(calls):
    packed = t(6, 8, 64)
    api.cc_qk_norm_rope(packed[:, :4], packed[:, 4:6], None, t(64), t(9, 16, 2, dtype=F32), i32(6), t(6, 4, 64), t(6, 2, 64))
    name, args = calls.seen[-1]
    assert name == "cc_qk_norm_rope" and args[8:18] == (6, 4, 2, 64, 32, 9, 512, 512, 256, 128)
    both = t(7, 2, 16, 2, 64)
    plan = (i32(4), i32(3), i32(3, 5))
    api.cc_qk_norm_rope_append(packed[:, :4], packed[:, 4:6], packed[:, 6:], None, None, None, None, t(6, 4, 64),
                               both[:, 0], both[:, 1], *plan)
    assert calls.seen[-1][1][13:33] == (6, 3, 5, 7, 16, 4, 2, 64, 0, 0, 512, 512, 512, 256, 4096, 128, 64, 4096, 128, 64)
    q = t(6, 4, 64)
    swapped = t(7, 2, 16, 64).transpose(1, 2)
    api.cc_attn_paged(q, swapped, swapped, t(6, 4, 64), *plan, None, causal_block=3)
    assert calls.seen[-1][1][7:25] == (6, 3, 5, 7, 16, 4, 2, 64, 256, 256, 2048, 64, 1024, 2048, 64, 1024, 0.125, 3)
    kv = t(3, 5, 4, 64)
    api.cc_attn_cross(t(3, 2, 4, 64), kv[:, :, :2], kv[:, :, 2:], t(3, 2, 4, 64), i32(3), None, scale=0.5)
    assert calls.seen[-1][1][5:16] == (3, 2, 5, 4, 2, 64, 256, 256, 256, 256, 0.5)
    api.cc_attn_cross(t(1, 2, 4, 64), t(1, 0, 2, 64), t(1, 0, 2, 64), t(1, 2, 4, 64), None, None)
    assert calls.seen[-1][1][5:11] == (1, 2, 0, 4, 2, 64)


def test_binding_refuses_shapes(calls):
    q, k, rot = t(6, 4, 64), t(6, 2, 64), t(9, 32, 2, dtype=F32)
    plan = (i32(4), i32(3), i32(3, 5))

    def rope(q=q, k=k, gq=None, gk=None, rot=rot, pos=None, qo=q, ko=k, **kw):
        api.cc_qk_norm_rope(q, k, gq, gk, rot, pos, qo, ko, **kw)

    def append(q=q, k=k, v=k, rot=rot, pos=None, qo=q, kc=cache(), vc=cache(), plan=plan):
        api.cc_qk_norm_rope_append(q, k, v, None, None, rot, pos, qo, kc, vc, *plan)

    def paged(q=q, kc=cache(), vc=cache(), o=q, plan=plan, **kw):
        api.cc_attn_paged(q, kc, vc, o, *plan, None, **kw)

    def cross(q=t(3, 2, 4, 64), k=t(3, 5, 2, 64), v=t(3, 5, 2, 64), o=t(3, 2, 4, 64), lens=None):
        api.cc_attn_cross(q, k, v, o, lens, None)

    rope(), append(), paged(), cross()
    before = len(calls.seen)
    bad = [
        lambda: rope(q=None), lambda: rope(ko=None), lambda: rope(q=None, k=None, qo=None, ko=None),
        lambda: rope(q=t(5, 4, 64), qo=t(5, 4, 64)), lambda: rope(k=t(6, 2, 32), ko=t(6, 2, 32)),
        lambda: rope(qo=t(6, 4, 32)), lambda: rope(ko=t(6, 3, 64)), lambda: rope(gq=t(32)), lambda: rope(gk=t(65)),
        lambda: rope(rot=t(9, 64, dtype=F32)), lambda: rope(rot=t(9, 32, 3, dtype=F32)), lambda: rope(pos=i32(5)),
        lambda: rope(style="quarters"), lambda: rope(q=t(6, 64), qo=t(6, 64)),
        lambda: rope(q=t(6, 64, 4).transpose(1, 2)), lambda: rope(q=t(6, 4, 128)[..., :64]),
        lambda: rope(pos=t(6, dtype=torch.int64)), lambda: rope(q=t(6, 4, 64, dtype=F32)),
        lambda: rope(q=t(3, 3, 4, 64)[:, :2], k=None, ko=None, qo=t(3, 2, 4, 64)),
        lambda: append(v=t(6, 3, 64)), lambda: append(k=t(5, 2, 64)), lambda: append(kc=cache(heads=3)),
        lambda: append(kc=cache(heads=3), vc=cache(heads=3)), lambda: append(kc=cache(d=32), vc=cache(d=32)),
        lambda: append(qo=t(6, 5, 64)), lambda: append(pos=i32(7)),
        lambda: append(plan=(i32(3), i32(3), i32(3, 5))), lambda: append(plan=(i32(4), i32(2), i32(3, 5))),
        lambda: append(plan=(i32(4), i32(3), i32(15))), lambda: append(plan=(i32(4), i32(3), t(3, 5, dtype=torch.int64))),
        lambda: append(plan=(i32(4), i32(3), i32(3, 6)[:, :5])),
        lambda: paged(o=t(6, 4, 32)), lambda: paged(vc=cache(pages=8)), lambda: paged(kc=cache(d=32), vc=cache(d=32)),
        lambda: paged(kc=t(7, 16, 128), vc=t(7, 16, 128)), lambda: paged(causal_block=1 << 32),
        lambda: paged(kc=t(7, 16, 64, 2).transpose(2, 3)), lambda: paged(plan=(i32(5), i32(3), i32(3, 5))),
        lambda: cross(q=t(6, 4, 64), o=t(6, 4, 64)), lambda: cross(k=t(2, 5, 2, 64), v=t(2, 5, 2, 64)),
        lambda: cross(v=t(3, 4, 2, 64)), lambda: cross(o=t(3, 2, 4, 32)), lambda: cross(lens=i32(2)),
        lambda: cross(k=t(3, 5, 2, 32), v=t(3, 5, 2, 32)), lambda: cross(lens=t(3, dtype=torch.int64)),
        lambda: cross(k=t(3, 9, 2, 64)[:, :5]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            print("not refused:", i)
    assert len(calls.seen) == before
    with pytest.raises(TypeError):
        rope(q=[1, 2])
    with pytest.raises(ValueError):
        rope(q=torch.zeros(6, 4, 64, dtype=BF16))  # not on the GPU
