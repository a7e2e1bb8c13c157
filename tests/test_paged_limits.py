"""Sizes of the paged-cache calls at the edge of 32-bit counts: what passes it is
refused on the host (every case fails before a launch)."""
import pytest

import context_exact_attention_ring_b200 as ra
from tests.test_paged_refusals import (APPEND, BOUNDS, DECODE, EXTEND, SCORES, SELECT, TRIM, E, built,  # noqa: F401
                                        call)    # built: fixture

BIG = dict(N=1 << 20, sp=1 << 16)


@pytest.mark.parametrize("kw", [
    # a segment is a kv head's group of 8 query heads (float32) or 16 (bf16), and counts its tiles of 128 keys and its
    # fixed cost: 2 (float32, bf16 above 8 heads) or 1; 2^31 of them are one too many
    dict(dtype=1, out_dtype=1, B=1 << 20, Hq=1, Hkv=1, ps=128, W=2046, ts=2046),
    dict(dtype=1, out_dtype=1, B=1 << 14, Hq=64 * 16, Hkv=64, ps=128, W=1022, ts=1022, qb=1 << 16),
    dict(dtype=1, out_dtype=1, B=33554431, Hq=1, Hkv=1, ps=128, W=63, ts=63),
    dict(dtype=1, out_dtype=1, B=1 << 20, Hq=1, Hkv=1, ps=128, W=8, ts=8, sel=1 << 16, n_sel=1 << 16, K=2046),
    dict(B=1 << 20, Hq=1, Hkv=1, ps=128, W=2047, ts=2047),
    dict(B=1 << 16, Hq=16 * 16, Hkv=16, ps=128, W=2046, ts=2046, qb=1 << 16),
    # products of sizes that pass 64 bits
    dict(B=1 << 30, Hq=1 << 30, Hkv=1, W=1, ts=1, qb=1 << 35), dict(B=1 << 30, Hq=1 << 30, Hkv=1 << 30, W=1, ts=1, qb=1 << 35),
    dict(B=(1 << 31) - 1, Hq=(1 << 31) - 1, Hkv=(1 << 31) - 1, ps=128, W=1 << 20, ts=1 << 20, qb=1 << 35),
])
def test_decode_units_are_counted_with_their_kernels_cost(kw):
    assert call("ring_attn_decode_paged", {**DECODE, **BIG}, **kw) == E


TOP = (1 << 31) - 1


@pytest.mark.parametrize("B", [TOP, TOP - 1022])
def test_sequence_counts_that_the_scan_would_step_past(B):
    # the block that scans takes 1024 sequences at a time, the last step's end included
    assert call("ring_attn_page_extend", EXTEND, B=B) == E
    assert call("ring_attn_page_trim", TRIM, B=B) == E


@pytest.mark.parametrize("kw", [dict(K=TOP), dict(K=TOP - 1000, ps=8), dict(K=1 << 28, ps=8), dict(K=1 << 27, ps=16)])
def test_select_lists_longer_than_any_sequence(kw):
    # as for the decode that reads them: K pages hold fewer than 2^31 tokens
    assert call("ring_attn_page_select", SELECT, **kw) == E


@pytest.mark.parametrize("kw", [dict(Hkv=1 << 26, D=128), dict(Hkv=1 << 25, D=64), dict(Hkv=1 << 25, D=128, dtype=1),
                                dict(Hkv=TOP, D=64, dtype=1)])
def test_bounds_of_rows_beyond_32_bits(kw):
    assert call("ring_attn_page_bounds", BOUNDS, B=1, **kw) == E


PACKED_INTS = {
    "ring_attn_page_extend": (EXTEND, "B W ps max_free max_tokens"),
    "ring_attn_page_trim": (TRIM, "B W ps max_free"),
    "ring_attn_paged_append": (APPEND, "T Hkv D N ps dtype"),
    "ring_attn_decode_paged": (DECODE, "B Hq Hkv D N ps W K dtype out_dtype"),
    "ring_attn_page_bounds": (BOUNDS, "B Hkv D N ps W dtype"),
    "ring_attn_page_scores": (SCORES, "B Hq Hkv D N ps W dtype"),
    "ring_attn_page_select": (SELECT, "B Hkv W ps K first last"),
}


@pytest.mark.parametrize("name", sorted(PACKED_INTS))
def test_packed_integers_are_not_cut_to_32_bits(name):
    base, ints = PACKED_INTS[name]
    no, words, n = ra._PACKED[name]
    fn = ra.lib().ring_attn_paged_packed
    for arg in ints.split():
        for off in (1 << 32, -1 << 32, 1 << 62, 1 << 31):
            args = {**base, arg: (base[arg] or 0) + off}
            assert fn(no, words.pack(*[0 if v is None else v for v in args.values()]), n, None) == E, (arg, off)


def test_binding_refuses_what_is_no_64_bit_integer():
    with pytest.raises(ValueError, match="64-bit"):
        ra._launch("ring_attn_page_trim", 0, *[1 << 64] * 10)
