"""bf16 gradients of the score-modified divergence are its float32 gradients,
rounded once.

In dQ = dS K whatever all keys have in common cancels (a row of dS sums to zero
where no cap bends the scores), its rounding errors do not: dS has to enter the
products with the same bits for either type of the outputs.  dK is a sum in a
fixed order, so its bf16 form is the rounded float32 form bit for bit.  dQ is
added up over the T key tiles in float32 in no fixed order: two runs differ by
at most 2 T 2^-24 of the sum of magnitudes |dS| |K|, and the bf16 form by half
a step (2^-8 of the value) more.
"""
import pytest
import torch

from attention_kl_divergence_gb300 import make_qk, streamkl as sk
from test_score import BF16, DEV, Ref, ranges

pytestmark = pytest.mark.gpu


def offset_keys(B, H, Hk, N, d, offset, seed):
    """Keys with `offset` in each of the last 16 channels, where the queries are zero: the scores do not change, dQ's
    sums of these channels cancel."""
    qk = [t.clone() for t in make_qk(B, H, N, N, d, 0.3, seed=seed, device=DEV, H_kv=Hk)]
    for q in (qk[0], qk[2]):
        q[..., -16:] = 0
    for k in (qk[1], qk[3]):
        k[..., -16:] += offset
    return qk


@pytest.mark.parametrize("offset", [0.0, 16.0])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("kind", ["plain", "capped", "wide", "bias"])
@pytest.mark.parametrize("d", [64, 128])
def test_bf16_gradients_are_the_rounded_float32_ones(d, kind, splits, offset):
    B, H, Hk, N = 1, 4, 2, 700
    qk = offset_keys(B, H, Hk, N, d, offset, seed=d)
    caps = {"plain": (0.0, 0.0), "capped": (50.0, 30.0), "wide": (50.0, 0.0), "bias": (0.0, 20.0)}[kind]
    slopes = torch.tensor([0.5, 0.1, 0.02, 0.004], device=DEV) if kind == "bias" else None
    begin, end, pos0 = ranges(docs=[0, 450, 700])(B, N, N)
    sc = sk.Scores(*caps, slopes, slopes, begin, end, pos0)
    rows = sk.kl_score_fwd(sc, *qk)
    g = torch.rand(B, H, N, device=DEV)
    ref = Ref(*qk, begin, end, torch.arange(N, device=DEV)[None], None, *caps, slopes, slopes)
    for setting in (1, 2):
        a = sk.kl_score_bwd(setting, sc, g, *qk, *rows, num_splits=splits)
        b = sk.kl_score_bwd(setting, sc, g, *qk, *rows, num_splits=splits, grad_dtype=BF16)
        ref.check_grads(setting, g, *a)
        assert torch.equal(b[1], a[1].to(BF16))
        f, p, K = (ref.f2, ref.p2 - ref.p1, qk[3]) if setting == 1 else (ref.f1, ref.p1 * (ref.ratio - ref.KL[..., None]), qk[1])
        size = (g.double()[..., None] * p * f * ref.scale).abs() @ K.double().abs().repeat_interleave(H // Hk, 1)
        tiles = (N + 127) // 128
        # `size` is the definition's: the recomputed dS are within 5 percent of it in the sum
        tol = 2.0 ** -8 * a[0].double().abs() + 2 * tiles * 2.0 ** -24 * 1.05 * size
        err = (b[0].double() - a[0].double()).abs()
        assert bool((err <= tol).all()), float((err / tol.clamp_min(1e-30)).max())


@pytest.mark.parametrize("setting", [1, 2])
def test_common_offset_of_the_keys_costs_the_autograd_function_no_accuracy(setting):
    """Against float64 in the norm.  Half a step of every value is at most 2^-8 of the norm; the float32 gradients'
    own distance from the definition is measured and allowed on top."""
    qk = offset_keys(1, 4, 2, 700, 128, 16.0, seed=3)
    begin, end, pos0 = ranges()(1, 700, 700)
    sc = sk.Scores(begin=begin, end=end, offset=pos0)
    ref = Ref(*qk, begin, end, torch.arange(700, device=DEV)[None])
    g = torch.rand(1, 4, 700, device=DEV)
    want = ref.grads(setting, g)[0]
    f32 = sk.kl_score_bwd(setting, sc, g, *qk, *sk.kl_score_fwd(sc, *qk))
    side = 2 if setting == 1 else 0
    leaves = [t.clone().requires_grad_() if side <= k < side + 2 else t for k, t in enumerate(qk)]
    grads = torch.autograd.grad(sk.ScoredAttentionKL.apply(*leaves, sc), leaves[side:side + 2], g)
    for got, wide, exact in zip(grads, f32, want):
        off = float((got.double() - exact).norm() / exact.norm())
        assert off <= 2.0 ** -8 + float((wide.double() - exact).norm() / exact.norm()), off
