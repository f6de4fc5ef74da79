"""Scores whose largest keep rising, or rise late: every form of the forward brings its sums to the new maximum.

One feature of the keys climbs along them, by more than the 8 (log2) that a maximum may
stay behind, from one key tile of 128 to the next; bounds as in test_attn.
"""
import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk
from test_attn import BF16, DEV, Ref, inputs

pytestmark = pytest.mark.gpu
# pairs of heads and of query tiles, one tile, few rows with every second key tile each, parts of rows
SHAPES = [(1, 4, 2, 300, 900, 128), (1, 2, 2, 520, 520, 64), (1, 1, 1, 100, 700, 64), (2, 8, 2, 1, 5000, 128), (1, 3, 1, 40, 1500, 64),
          (1, 5, 1, 7, 2049, 128)]


def climbing(shape, how):
    Q, K, V = inputs(*shape, peak=0.3)
    Nk, d = shape[4:]
    Q[..., 0] = 2.0
    tile = torch.arange(Nk, device=DEV) // 128
    if how == "up":
        level = 10.0 * tile
    elif how == "every second tile up":
        level = 10.0 * tile * (tile % 2)
    elif how == "at the last key":
        level = torch.where(torch.arange(Nk, device=DEV) == Nk - 1, 40.0, 0.0)
    else:
        assert how == "just within the slack, then up"
        level = torch.where(tile % 3 == 2, 7.9, 0.0) + 20.0 * (tile // 3)
    K[..., 0] = (level * 0.6931 / (2.0 * d ** -0.5)).to(BF16)
    return Q, K, V


@pytest.mark.parametrize("splits", [0, 1, 2, 5])
@pytest.mark.parametrize("how", ["up", "every second tile up", "at the last key", "just within the slack, then up"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, how, splits):
    t = climbing(shape, how)
    ref = Ref(*t, causal=True)
    ref.check(*sk.attn_fwd(*t, causal=True, num_splits=splits))
    O, LSE, rest = sk.attn_fwd(*t, causal=True, num_splits=splits, rest=True)
    ref.check(O, LSE)
    assert bool(((O.double() + rest.double() - ref.O).abs() <= ref.two_terms).all())
    if splits < 2:
        dO = torch.randn(t[0].shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(BF16)
        ref.check_grads(dO, *sk.attn_bwd(dO, *t, O, LSE, rest=rest, causal=True))


@pytest.mark.parametrize("peak", [0.3, 2.0])
@pytest.mark.parametrize("d", [64, 128])
def test_gradients_of_values_with_a_common_offset(d, peak):
    """dV has one rounding of each probability and one of its own, 2^-8 / sqrt 3 of the norm each at most (a rounding is off by
    half a step, evenly spread, and probabilities' roundings add up in no common direction), a third of both for the rest."""
    Q, K, V = inputs(1, 4, 2, 500, 500, d, peak=peak)
    K[..., : d // 8] += 16.0
    V += 4.0
    dO = torch.randn((1, 4, 500, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(BF16)
    O, LSE, rest = sk.attn_fwd(Q, K, V, causal=True, rest=True)
    dV = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, causal=True)[2]
    want = Ref(Q, K, V, causal=True).grads(dO)[0][2]
    err = float((dV.double() - want).norm() / want.norm())
    assert err <= 2.0 ** -8 * (2 / 3) ** 0.5 * 4 / 3, err
