"""Keys, values and output gradients with a NaN or an infinity that rows do see: what the
formulas give there, wherever the token stands in its tile.

A key that scores -inf has a probability of 0: LSE, O, dK and dV are those of the other
keys, its own dK and dV are 0, and dQ is 0 * (-inf) = NaN in the feature that is infinite,
in the rows that see the key.  dV has no values in it, so that a broken value reaches O, dQ
and dK alone.  Tolerances as in test_attn, of the same tensors without the broken token.
"""
import math

import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk
from test_attn import BF16, DEV, Ref, inputs, masks
from test_attn_calls import spread
from test_attn_broken_value import AT, F, SHAPES, plain_ranges

pytestmark = pytest.mark.gpu


def without(t, at):
    return torch.cat((t[:, :, :at], t[:, :, at + 1:]), 2).contiguous()


def ranges_without(ranges, Nk, at):
    begin, end, offset = ranges
    assert offset is None
    return begin - (begin > at).int(), end - (end > at).int(), None


def grad_like(Q):
    return torch.randn(Q.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(BF16)


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("kind", ["full", "causal", "window", "two ends"])
@pytest.mark.parametrize("value", [-math.inf, math.inf])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_key_that_scores_minus_infinity(shape, value, kind, splits):
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape)
    Q[..., F] = Q[..., F].abs() + 0.25
    if value > 0:
        Q[..., F] = -Q[..., F]
    dO = grad_like(Q)
    K[:, :, AT, F] = value
    ranges = plain_ranges(kind, B, Nq, Nk)
    ref = Ref(Q, without(K, AT), without(V, AT), ranges_without(ranges, Nk, AT))
    O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    ref.check(O, LSE)
    ref.check(*sk.attn_fwd(Q, K, V, ranges=ranges))
    dQ, dK, dV = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges, num_splits=splits)
    sees = ((ranges[0] <= AT) & (ranges[1] > AT))[:, None].expand(B, H, Nq)
    nan = torch.zeros_like(dQ, dtype=torch.bool)
    nan[..., F] = sees
    assert torch.equal(dQ.isnan(), nan)
    assert bool((dK[:, :, AT] == 0).all()) and bool((dV[:, :, AT] == 0).all())
    want = ref.grads(dO)[0][0]
    ref.check_grads(dO, torch.where(nan, want.to(BF16), dQ), without(dK, AT), without(dV, AT))
    again = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges, num_splits=splits)
    assert torch.equal(again[1], dK) and torch.equal(again[2], dV) and torch.equal(again[0].isnan(), nan)


@pytest.mark.parametrize("how", ["rows by token", "padded rows", "heads first", "every second token"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_such_a_key_in_another_layout(shape, how):
    Q, K, V = inputs(*shape)
    Q[..., F] = Q[..., F].abs() + 0.25
    dO = grad_like(Q)
    K[:, -1, AT, F], K[0, 0, 17, 2 * F] = -math.inf, math.nan
    want = sk.attn_fwd(Q, K, V, causal=True, rest=True)
    grads = sk.attn_bwd(dO, Q, K, V, *want[:2], rest=want[2], causal=True)
    views = [spread(t, how) for t in (Q, K, V)]
    got = sk.attn_fwd(*views, causal=True, rest=True)
    again = sk.attn_bwd(spread(dO, how), *views, *got[:2], rest=got[2], causal=True)
    for a, b in zip((*got, *again), (*want, *grads)):
        assert torch.equal(a.isnan(), b.isnan())
    same = [torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) for a, b in zip((*got, *again[1:]), (*want, *grads[1:]))]
    assert all(same) and bool(grads[0].isnan().any()) and not bool(grads[0].isnan().all())


@pytest.mark.parametrize("kind", ["full", "causal", "two ends"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_score_below_the_range_of_float32(shape, kind):
    """Finite tokens whose product is not: the score is -inf in float32 and the probability 0; no gradient is NaN."""
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape)
    Q[..., F], K[..., F] = 1e25, 0
    K[:, :, AT, F] = -1e25
    dO = grad_like(Q)
    ranges = plain_ranges(kind, B, Nq, Nk)
    ref = Ref(Q, without(K, AT), without(V, AT), ranges_without(ranges, Nk, AT))
    O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    ref.check(O, LSE)
    dQ, dK, dV = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges)
    assert bool((dK[:, :, AT] == 0).all()) and bool((dV[:, :, AT] == 0).all())
    ref.check_grads(dO, dQ, without(dK, AT), without(dV, AT))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kind", ["full", "causal", "window", "two ends"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_broken_value_does_not_reach_dv(shape, kind, value):
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape)
    dO = grad_like(Q)
    ranges = plain_ranges(kind, B, Nq, Nk)
    ref = Ref(Q, K, V, ranges)
    V[:, :, AT, F] = value
    sees = ((ranges[0] <= AT) & (ranges[1] > AT))[:, None].expand(B, H, Nq)
    O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    dQ, dK, dV = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges)
    assert torch.equal(dQ.isnan().any(-1), sees)
    want, tol = ref.grads(dO)
    assert bool(((dV.double() - want[2]).abs() <= tol[2] * 1.01 + 2.0 ** -8 * want[2].abs() + 1e-30).all())
    err = (dQ.double() - want[0]).abs() - (tol[0] * 1.01 + 2.0 ** -8 * want[0].abs() + 1e-30)
    assert bool((err[~sees] <= 0).all())


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("kind", ["full", "causal", "two ends"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_broken_output_gradient(shape, kind, value):
    """It reaches its own row of dQ, and dK and dV of the keys that this row sees."""
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape)
    dO = grad_like(Q)
    ranges = plain_ranges(kind, B, Nq, Nk)
    O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    clean = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges)
    row = 417
    dO[:, :, row, F] = value
    dQ, dK, dV = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges)
    assert bool((~dQ[:, :, row].isfinite()).any(-1).all()) and int((~dQ.isfinite()).any(-1).sum()) == B * H
    keys = torch.arange(Nk, device=DEV)
    seen = (keys >= ranges[0][0, row]) & (keys < ranges[1][0, row])
    assert bool((~dV[:, :, seen, F].isfinite()).all()) and bool((~dK[:, :, seen].isfinite()).any(-1).all())
    assert torch.equal(dK[:, :, ~seen], clean[1][:, :, ~seen]) and torch.equal(dV[:, :, ~seen], clean[2][:, :, ~seen])


@pytest.mark.parametrize("d", [64, 128])
def test_a_broken_key_and_a_broken_output_gradient_meet(d):
    """A probability of 0 times an infinite dO is NaN in dV of the key, as in dV of the row's other keys."""
    Q, K, V = inputs(1, 2, 1, 500, 500, d)
    Q[..., F] = Q[..., F].abs() + 0.25
    K[:, :, AT, F] = -math.inf
    dO = grad_like(Q)
    O, LSE, rest = sk.attn_fwd(Q, K, V, causal=True, rest=True)
    for row in (AT, AT + 3, 490):  # in a tile that some rows do not see all of, and behind it
        g = dO.clone()
        g[:, :, row, 9] = math.inf
        dQ, dK, dV = sk.attn_bwd(g, Q, K, V, O, LSE, rest=rest, causal=True)
        assert bool((~dV[:, :, :row + 1, 9].isfinite()).all()) and bool(dV[:, :, row + 1:].isfinite().all())
        assert bool((~dK[:, :, :row + 1].isfinite()).any(-1).all()) and bool(dK[:, :, row + 1:].isfinite().all())


@pytest.mark.parametrize("masked", ["docs", "padded"])
def test_packed_and_padded_batches_with_broken_tokens(masked):
    """A document's or a padded sequence's NaN key, value or query stays within it."""
    B, H, Hk, Nq, Nk, d = 2, 4, 2, 700, 700, 64
    Q, K, V = inputs(B, H, Hk, Nq, Nk, d)
    dO = grad_like(Q)
    ranges = masks(masked, B, Nq, Nk)
    want = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    clean = sk.attn_bwd(dO, Q, K, V, *want[:2], rest=want[2], ranges=ranges)
    lo, hi = (350, 623) if masked == "docs" else (0, 700)  # the token's document; sequence 0
    for which in range(3):
        t = [Q.clone(), K.clone(), V.clone()]
        t[which][0, :, 400, F] = math.nan
        got = sk.attn_fwd(*t, ranges=ranges, rest=True)
        grads = sk.attn_bwd(dO, *t, *got[:2], rest=got[2], ranges=ranges)
        inside = torch.zeros(B, Nq, dtype=torch.bool, device=DEV)
        inside[0, lo:hi] = True
        out = ~inside[:, None].expand(B, H, Nq)
        assert torch.equal(got[0][out], want[0][out]) and torch.equal(got[1][out], want[1][out])
        out = ~inside[:, None].expand(B, Hk, Nk)
        assert torch.equal(grads[1][out], clean[1][out]) and torch.equal(grads[2][out], clean[2][out])
        assert bool(grads[0][~inside[:, None].expand(B, H, Nq)].isfinite().all())
