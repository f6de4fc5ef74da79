"""A value with a NaN or an infinity that rows do see: it reaches their outputs, wherever
the token stands in its tile, and not their LSE, which has no values in it.
"""
import math

import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk
from test_attn import DEV, inputs

pytestmark = pytest.mark.gpu
SHAPES = [(1, 4, 2, 600, 600, 128), (2, 3, 1, 900, 900, 64)]
AT, F = 333, 5  # the token, and its feature that is broken


def plain_ranges(kind, B, Nq, Nk):
    """begin and end per row, the mask's offset worked into them."""
    if kind == "full":
        return torch.zeros(B, Nq, dtype=torch.int32, device=DEV), torch.full((B, Nq), Nk, dtype=torch.int32, device=DEV), None
    if kind == "causal":
        end = torch.arange(1, Nq + 1, dtype=torch.int32, device=DEV) + (Nk - Nq)
        return torch.zeros(B, Nq, dtype=torch.int32, device=DEV), end.repeat(B, 1), None
    if kind == "window":
        end = torch.arange(1, Nq + 1, dtype=torch.int32, device=DEV)
        return (end - 100).clamp(min=0).repeat(B, 1), end.repeat(B, 1), None
    assert kind == "two ends"  # rows in turn see keys up to the token and from it on
    row = torch.arange(Nq, device=DEV)
    begin = torch.where(row % 2 == 0, 300, AT).int().repeat(B, 1)
    end = torch.where(row % 2 == 0, AT, Nk).int().repeat(B, 1)
    return begin, end, None


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kind", ["full", "causal", "window", "two ends"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_broken_value_leaves_lse_alone(shape, kind, value):
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape)
    ranges = plain_ranges(kind, B, Nq, Nk)
    clean = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    once = sk.attn_fwd(Q, K, V, ranges=ranges)
    V2 = V.clone()
    V2[:, :, AT, F] = value
    sees = ((ranges[0] <= AT) & (ranges[1] > AT))[:, None].expand(B, H, Nq)
    O, LSE, rest = sk.attn_fwd(Q, K, V2, ranges=ranges, rest=True)
    O1, LSE1 = sk.attn_fwd(Q, K, V2, ranges=ranges)
    for o, lse, want in ((O, LSE, clean), (O1, LSE1, once)):
        assert torch.equal(lse, want[1])
        assert torch.equal(~o.isfinite().all(-1), sees) and torch.equal(o[~sees], want[0][~sees])


@pytest.mark.parametrize("splits", [0, 1, 3, 7])
@pytest.mark.parametrize("shape", [(2, 8, 2, 1, 5000, 128), (1, 3, 1, 40, 1500, 64), (1, 6, 2, 7, 1025, 64), (1, 2, 2, 130, 1100, 128)], ids=str)
def test_a_broken_value_with_split_keys(shape, splits):
    """Few rows over long keys, every second key tile each, and parts of rows: LSE is that of the scores."""
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape)
    for at in (Nk - 1, Nk - Nq, 700):
        V2 = V.clone()
        V2[:, :, at, F] = math.nan
        for rest in (False, True):
            want = sk.attn_fwd(Q, K, V, causal=True, num_splits=splits, rest=rest)
            got = sk.attn_fwd(Q, K, V2, causal=True, num_splits=splits, rest=rest)
            sees = (torch.arange(Nq, device=DEV) + Nk - Nq >= at).expand(B, H, Nq)
            assert torch.equal(got[1], want[1])
            assert torch.equal(got[0].isnan().any(-1), sees) and torch.equal(got[0][~sees], want[0][~sees])
