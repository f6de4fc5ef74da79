"""Attention over the 8-bit cache where the sizes of its pages, of its scores and
of its queries lie far apart: the definition's result is an ordinary number, and
no factor on the way to it may leave float32's range.

Keys differ in their first value alone, which sets their score; what the scores
of a page are, log2 of a probability against the largest, is part of the case.
Tolerances are those of test_cache8, but relative ones where an output is small:
its absolute term (1e-30) would hide it.
"""
import math

import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk
from test_cache8 import BF16, DEV, Ref, tables

pytestmark = pytest.mark.gpu
T = 16
# heads of a key head, new tokens: one 8-row tile, one of 16 rows, teams of them
ROWS = [(1, 1), (4, 2), (5, 2), (5, 7), (8, 16)]
# pages of a sequence: in a chunk with the first, in the first chunk of another warp, in the same warp's second chunk
PLACES = [(0, 1), (1, 0), (0, 16), (16, 0), (0, 3), (31, 2)]


def filled(pages_of, M, Hk, d, group, Nq, step=1.0):
    """(cache, table, lengths, Q, scale) of one sequence of M pages, written by append.  pages_of[m] = (score, size): the
    log2 score of the page's keys (as e4m3 rounds it), in units of `step`, and the size of its values; others: (0, 0)."""
    table, pages = tables(1, M, seed=M)
    cache = sk.Cache8.empty(pages, Hk, T, d, DEV)
    g = torch.Generator(device=DEV).manual_seed(M)
    k = torch.zeros(1, Hk, M * T, d, device=DEV)
    v = (torch.rand(1, Hk, M * T, d, generator=g, device=DEV) + 1) / 2
    for m in range(M):
        score, size = pages_of.get(m, (0.0, 0.0))
        k[:, :, m * T:(m + 1) * T, 0] = score / step
        v[:, :, m * T:(m + 1) * T] *= size
    Q = torch.zeros(1, Hk * group, Nq, d, dtype=BF16, device=DEV)
    Q[..., 0] = 1
    sk.cache8_append(cache, table, torch.zeros(1, dtype=torch.int32, device=DEV), k.to(BF16), v.to(BF16))
    return cache, table, torch.tensor([M * T], dtype=torch.int32, device=DEV), Q, step * math.log(2.0)


def relative(O, want, bound):
    err = ((O.double() - want) / want).abs()
    assert bool((err <= bound).all()), float(err.max())


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("places", PLACES, ids=str)
@pytest.mark.parametrize("group,Nq", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_a_page_of_zeros_has_the_largest_score(d, group, Nq, places, splits):
    """Its values' scale is 2^-100.  Others lie 118 and 130 (log2) behind it and are of sizes that make them the output."""
    for a, b in (((-118.0, 448 * 2.0 ** 22), (-130.0, 448 * 2.0 ** 60)), ((-118.0, 448 * 2.0 ** 22), (-118.0, 448 * 2.0 ** 21)),
                 ((-130.0, 448 * 2.0 ** 60), (-20.0, 2.0 ** -90)), ((-200.0, 448 * 2.0 ** 110), (-100.0, 448.0))):
        cache, table, n, Q, scale = filled({places[0]: a, places[1]: b}, 34, 2, d, group, Nq)
        assert float(cache.v_scale.min()) == 2.0 ** -100
        O, LSE = sk.attn_cache8(Q, cache, table, n, scale=scale, num_splits=splits)
        ref = Ref(Q, cache, table, n, scale)
        assert bool(ref.O.abs().max() < 1e38) and bool(ref.O.abs().min() > 1e-38)
        ref.check(O, LSE)
        relative(O, ref.O, 2.0 ** -11 + 2.0 ** -8 + 4 * ref.delta + ref.acc)


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("places", PLACES, ids=str)
@pytest.mark.parametrize("group,Nq", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_at_both_ends_of_the_range(d, group, Nq, places, splits):
    """Values up to 2^127 with a score up to 8 behind which the reference of the probabilities may stay; values whose output
    is about 2^-118 beside zeros with larger scores."""
    for pages_of in ({places[0]: (0.0, 448 * 2.0 ** 100), places[1]: (7.5, 2.0 ** 127)},
                     {places[0]: (-128.0, 448 * 2.0 ** 6), places[1]: (-144.0, 448 * 2.0 ** 20)}):
        cache, table, n, Q, scale = filled(pages_of, 34, 1, d, group, Nq, step=0.5)
        if pages_of[places[1]][0] > 0:  # a scale that the page had before it held smaller values
            page = int(table[0, places[1]])
            small = cache.v.view(torch.uint8)[page].view(torch.float8_e4m3fn).float() * (cache.v_scale[page] / 2.0 ** 127)[:, None, None]
            cache.v.view(torch.uint8)[page] = small.to(torch.float8_e4m3fn).view(torch.uint8)
            cache.v_scale[page] = 2.0 ** 127
        O, LSE = sk.attn_cache8(Q, cache, table, n, scale=scale, num_splits=splits)
        ref = Ref(Q, cache, table, n, scale)
        assert bool((ref.O.abs() < 3e38).all()) and bool((ref.O.abs() > 2.0 ** -125).all())
        ref.check(O, LSE)
        relative(O, ref.O, 2.0 ** -11 + 2.0 ** -8 + 4 * ref.delta + ref.acc)


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("group,Nq", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_large_queries_over_keys_of_zeros_with_a_large_scale(d, group, Nq, splits):
    """A page that held large keys and holds zeros now: its scores are 0, whatever 2^70 (the queries) times 2^80 (the scale)
    is.  The other pages' keys are small ones."""
    cache, table, n, Q, scale = filled({3: (2.0, 1.0), 16: (-3.0, 5.0)}, 34, 2, d, group, Nq)
    cache.k_scale *= 2.0 ** -70
    Q *= 2.0 ** 70
    for m in (0, 5, 19):
        page = int(table[0, m])
        assert not bool(cache.k.view(torch.uint8)[page].any())
        cache.k_scale[page] = 2.0 ** 80
    O, LSE = sk.attn_cache8(Q, cache, table, n, scale=scale, num_splits=splits)
    Ref(Q, cache, table, n, scale).check(O, LSE)


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("places", PLACES, ids=str)
@pytest.mark.parametrize("group,Nq", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [2.0 ** 17, 2.0 ** 20, 2.0 ** 23, 2.0 ** 60])
def test_scores_so_large_that_one_is_below_their_last_bit(step, d, group, Nq, places, splits):
    """Scores of up to 64 steps are whole multiples of one number, exactly: two pages tie, the rest have no weight.  LSE is
    off by the roundings of the scale in both bases."""
    pages_of = {places[0]: (64 * step, 448 * 2.0 ** 3), places[1]: (64 * step, 448 * 2.0 ** -20), 5: (60 * step, 448 * 2.0 ** 40)}
    cache, table, n, Q, scale = filled(pages_of, 34, 2, d, group, Nq, step=step)
    O, LSE = sk.attn_cache8(Q, cache, table, n, scale=scale, num_splits=splits)
    at = table[0, list(places)].long()
    v = (cache.v.double() * cache.v_scale.double()[..., None, None])[at].mean((0, 2)).repeat_interleave(group, 0)
    relative(O, v[None, :, None].expand_as(O), 2.0 ** -11 + 2.0 ** -8 + 2.0 ** -16)
    want = 64 * step * math.log(2.0) + math.log(32)
    assert bool(((LSE.double() - want).abs() <= 2.0 ** -21 * want).all())


@pytest.mark.parametrize("splits", [0, 2, 3, 40])
@pytest.mark.parametrize("group,Nq", [(1, 8), (4, 2), (1, 13), (5, 7), (8, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing_of_a_share(d, group, Nq, splits):
    """CTAs take whole steps of 256 keys: behind a multiple of them stand keys that the first rows do not see."""
    for behind in sorted({1, 2, Nq - 1}):
        M = 49
        cache, table, n, _, _ = filled({m: (float(m % 5), 1.0 + m) for m in range(M)}, M, 2, d, group, Nq)
        Q = torch.randn(1, 2 * group, Nq, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)).to(BF16)
        for steps in (0, 1, 2, 3):
            n.fill_(256 * steps + behind)
            O, LSE = sk.attn_cache8(Q, cache, table, n, num_splits=splits)
            Ref(Q, cache, table, n).check(O, LSE)


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("places", PLACES, ids=str)
@pytest.mark.parametrize("group,Nq", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [2.0 ** 60, 2.0 ** 95, 2.0 ** 119])
def test_scores_far_below_0_and_on_both_sides_of_it(step, d, group, Nq, places, splits):
    """The largest are 32 steps below 0, or above it with all others as far below it; two pages have it."""
    for top, rest in ((-32.0, -64.0), (64.0, -64.0)):
        pages_of = {m: (rest * step, 448.0 * 2.0 ** (m % 7)) for m in range(34)}
        pages_of[places[0]], pages_of[places[1]] = (top * step, 448 * 2.0 ** 3), (top * step, 448 * 2.0 ** -20)
        cache, table, n, Q, scale = filled(pages_of, 34, 2, d, group, Nq, step=step)
        O, LSE = sk.attn_cache8(Q, cache, table, n, scale=scale, num_splits=splits)
        at = table[0, list(places)].long()
        v = (cache.v.double() * cache.v_scale.double()[..., None, None])[at].mean((0, 2)).repeat_interleave(group, 0)
        relative(O, v[None, :, None].expand_as(O), 2.0 ** -11 + 2.0 ** -8 + 2.0 ** -16)
        want = top * step * math.log(2.0)
        assert bool(((LSE.double() - want).abs() <= 2.0 ** -21 * abs(want)).all())
