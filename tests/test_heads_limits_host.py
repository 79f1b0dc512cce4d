"""Argument checks of the operators with heads at the largest sizes and the loosest strides, on the host."""

import pytest

from test_heads_host import APPEND, CROSS, PAGED, call, lib, p  # noqa: F401 (fixtures)


def test_workspaces_of_refused_sizes_are_none(lib, p):
    """0 bytes for every size that the call refuses, and for the largest that it takes a workspace."""
    paged, cross = lib.cc_attn_paged_workspace_bytes, lib.cc_attn_cross_workspace_bytes
    heads = dict(heads=131072, kv_heads=1024, d=16, ld_q=1 << 21, ld_o=1 << 21, ld_k=1 << 14, ld_v=1 << 14)
    assert call(lib, "cc_attn_paged", PAGED, p, **heads)[0] == 2 and paged(4, 2, 131072, 1024, 16) == 0
    assert call(lib, "cc_attn_cross", CROSS, p, **heads)[0] == 2 and cross(2, 2, 5000, 131072, 1024, 16) == 0
    assert paged(4, 2, 65536, 512, 16) > 0 and cross(2, 2, 5000, 65536, 512, 16) > 0
    rows = (1 << 30) + 1
    assert call(lib, "cc_attn_paged", PAGED, p, rows=rows)[0] == 2 and paged(rows, 2, 4, 2, 64) == 0
    assert paged(1 << 30, 2, 4, 2, 64) > 0
    assert call(lib, "cc_attn_cross", CROSS, p, n=3, lq=1 << 29)[0] == 2 and cross(3, 1 << 29, 5000, 4, 2, 64) == 0
    assert cross(2, 1 << 29, 5000, 4, 2, 64) > 0
    assert call(lib, "cc_attn_cross", CROSS, p, n=1 << 15, lq=1 << 15, lk=1 << 20)[0] == 2
    assert cross(1 << 15, 1 << 15, 1 << 20, 4, 2, 64) == 0 and cross(1 << 15, 1 << 9, 1 << 12, 4, 2, 64) > 0
    span = dict(n=1, lq=1, lk=1 << 30, heads=2, kv_heads=2, d=128)
    assert call(lib, "cc_attn_cross", CROSS, p, ld_k=256, ld_v=256, **span)[0] == 2
    assert cross(1, 1, 1 << 30, 2, 2, 128) == 0 and cross(1, 1, (1 << 30) - 1, 2, 2, 128) > 0


def test_sequences_beyond_what_a_cta_can_count_in_time_are_refused(lib, p):
    paged, cross = lib.cc_attn_paged_workspace_bytes, lib.cc_attn_cross_workspace_bytes
    most = 1 << 20
    for name, names, key in (("cc_attn_paged", PAGED, "seqs"), ("cc_attn_cross", CROSS, "n")):
        st, msg = call(lib, name, names, p, lq=1, **{key: most + 1})
        assert st == 2 and "2^20" in msg, (name, st, msg)
    assert paged(4, most, 4, 2, 64) > 0 and paged(4, most + 1, 4, 2, 64) == 0
    assert cross(most, 1, 5000, 4, 2, 64) > 0 and cross(most + 1, 1, 5000, 4, 2, 64) == 0


@pytest.mark.parametrize("side", ["k", "v"])
def test_strides_of_sizes_of_one_are_not_looked_at(lib, p, side):
    """A page or a head that is the only one has no neighbour, so its stride may be anything (0 in an expanded tensor).
    The refusal behind that of strides, of the rows, tells that they were accepted."""
    one_head = dict(heads=4, kv_heads=1, k_token=64, v_token=64)
    for stride in (0, 1, 8, -64, 1 << 50):
        for sizes in ({**one_head, side + "_head": stride}, {"pages": 1, side + "_page": stride}):
            st, msg = call(lib, "cc_attn_paged", PAGED, p, rows=(1 << 30) + 1, **sizes)
            assert st == 2 and "2^30 rows" in msg, (sizes, st, msg)
        for sizes in ({side + "_head": stride}, {side + "_page": stride}, {"pages": 1, side + "_head": stride},
                      {**one_head, side + "_page": stride}, {**one_head, "pages": 1, side + "_token": stride}):
            st, msg = call(lib, "cc_attn_paged", PAGED, p, rows=(1 << 30) + 1, **sizes)
            assert st in (1, 2) and "strides" in msg, (sizes, st, msg)
            st, msg = call(lib, "cc_qk_norm_rope_append", APPEND, p, **sizes)
            assert st in (1, 2) and "strides" in msg, (sizes, st, msg)


def test_scales_that_pass_fp32_as_powers_of_two_are_refused(lib, p):
    """Scores are taken times scale * log2(e) in fp32: as infinity it would turn a score of 0 into NaN."""
    for name, names, key in (("cc_attn_paged", PAGED, "seqs"), ("cc_attn_cross", CROSS, "n")):
        for scale, text in ((2.4e38, "scale"), (3.4e38, "scale"), (2.3e38, "2^20"), (1e-45, "2^20")):
            st, msg = call(lib, name, names, p, scale=scale, lq=1, **{key: (1 << 20) + 1})
            assert st == (1 if text == "scale" else 2) and text in msg, (name, scale, st, msg)
