"""Tensor memory is allocated by a wait without limit, and CTAs of any launches may share an
SM: no mix of the feed-forward kernels' CTAs whose shared memory fits an SM may want more than
its 512 columns (host arithmetic; no GPU)."""

import random

import pytest

import implicit_gemm_conv_tcgen05_gb300 as igc

SMEM = 228 * 1024      # of an SM, of which every CTA takes 1 KB besides its own
COLUMNS = 512
OPS = [(igc.PLAN_FFN_LINEAR, 1), (igc.PLAN_FFN_GATED, 1), (igc.PLAN_FFN_GRAD_X, 1),
       (igc.PLAN_FFN_GRAD_X, 2), (igc.PLAN_FFN_GRAD_W, 1), (igc.PLAN_FFN_GRAD_W, 2)]


def most_columns(kinds):
    """The most columns that CTAs of the kinds (columns, dynamic bytes) can want together on
    one SM: an unbounded knapsack over pieces of 128 bytes."""
    best = [0] * (SMEM // 128 + 1)
    items = {(c, (s + 1024) // 128) for c, s in kinds}
    for room in range(len(best)):
        for c, s in items:
            if s <= room:
                best[room] = max(best[room], best[room - s] + c)
    return best[-1]


def sizes(seed, n):
    rng = random.Random(seed)
    for _ in range(n):
        yield tuple(int(2 ** rng.uniform(0, hi)) for hi in (13, 14, 14))


def test_two_launches_that_could_meet():
    """A gated product of 144-row blocks (256 columns) beside one token's (32 columns)."""
    kinds = [igc._ffn_cta_resources(igc.PLAN_FFN_GATED, 139, 1690, 637),
             igc._ffn_cta_resources(igc.PLAN_FFN_LINEAR, 1, 1000, 777)]
    assert [c for c, _ in kinds] == [256, 32]
    assert most_columns(kinds) <= COLUMNS


def test_no_mix_of_launches_exceeds_the_columns():
    kinds = {igc._ffn_cta_resources(op, *mnk, count)
             for op, count in OPS for mnk in sizes(op * 2 + count, 1500)}
    assert {c for c, _ in kinds} == {32, 64, 128, 256, 512}
    assert all(c % 32 == 0 and 0 < s <= 227 * 1024 for c, s in kinds)
    assert most_columns(kinds) <= COLUMNS


@pytest.mark.parametrize("width", [128, 256])
def test_forced_tiles(width):
    igc.igc_set_tile_width(width)
    try:
        forced = [igc._ffn_cta_resources(op, 64, 300, 200, count) for op, count in OPS]
    finally:
        igc.igc_set_tile_width(0)
    small = [igc._ffn_cta_resources(igc.PLAN_FFN_LINEAR, 1, 64, 64)]
    assert all(c == 2 * width for c, _ in forced)
    assert most_columns(forced + small) <= COLUMNS


def test_192_wide_tiles():
    wide = igc._ffn_cta_resources(igc.PLAN_FFN_LINEAR, 3630, 702, 2944)
    small = igc._ffn_cta_resources(igc.PLAN_FFN_LINEAR, 1, 64, 64)
    assert wide[0] == 512 and most_columns([wide, small]) <= COLUMNS
