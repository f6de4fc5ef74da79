"""Hidden NaN, infinities and huge values have no effect on bf16 gradients either,
nor on those of the autograd function."""
import pytest
import torch

from attention_kl_divergence_gb300 import make_qk, streamkl as sk
from test_score import BAD, BF16, DEV, SCORES, Ref, ranges

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("value", BAD)
@pytest.mark.parametrize("kind", ["plain", "capped", "one_side", "all"])
@pytest.mark.parametrize("d", [64, 128])
def test_padding(d, kind, value, splits):
    kw = dict(SCORES[kind])
    bias, peak = kw.pop("bias", False), kw.pop("peak", 1.0)
    B, H, Hk, N, n = 2, 2, 1, 200, [90, 161]
    qk = make_qk(B, H, N, N, d, 0.3, teacher_scale=peak, seed=d, device=DEV, H_kv=Hk)
    begin, end, offset = ranges(q_lengths=n, k_lengths=n)(B, N, N)
    sl = torch.tensor([0.5, 0.1], device=DEV) if bias else None
    sc = sk.Scores(begin=begin, end=end, offset=offset, slopes1=sl, slopes2=sl, **kw)
    ref = Ref(*qk, begin, end, torch.arange(N, device=DEV).expand(B, N), None, slopes1=sl, slopes2=sl, **kw)
    dirty = [t.clone() for t in qk]
    for t in dirty:
        for b in range(B):
            t[b, :, n[b]:] = value
    g = torch.randn(B, H, N, device=DEV)
    rows = sk.kl_score_fwd(sc, *dirty)
    for setting in (1, 2):
        clean = sk.kl_score_bwd(setting, sc, g, *qk, *sk.kl_score_fwd(sc, *qk), grad_dtype=BF16, num_splits=splits)
        dQ, dK = sk.kl_score_bwd(setting, sc, g, *dirty, *rows, grad_dtype=BF16, num_splits=splits)
        ref.check_grads(setting, g, dQ, dK)
        assert torch.equal(dK, clean[1])
        for b in range(B):
            assert bool((dQ[b, :, n[b]:] == 0).all()) and bool((dK[b, :, n[b]:] == 0).all())
    leaves = [t.requires_grad_() for t in dirty]
    KL = sk.ScoredAttentionKL.apply(*leaves, sc)
    grads = torch.autograd.grad(KL, leaves, g)
    assert torch.equal(KL, rows[0])
    ref.check_grads(2, g, *grads[:2])
    ref.check_grads(1, g, *grads[2:])


@pytest.mark.parametrize("value", BAD[:3])
@pytest.mark.parametrize("where", [0, 1, 2, 3])
def test_a_bad_token_stays_in_its_document(where, value):
    B, H, N, d = 1, 2, 300, 128
    qk = list(make_qk(B, H, N, N, d, 0.3, seed=4, device=DEV))
    begin, end, offset = ranges(docs=[0, 130, 170, 300])(B, N, N)
    sc = sk.Scores(50.0, 50.0, begin=begin, end=end, offset=offset)
    ref = Ref(*qk, begin, end, torch.arange(N, device=DEV)[None], None, 50.0, 50.0)
    qk[where] = qk[where].clone()
    qk[where][0, 1, 150, 7] = value
    leaves = [t.clone().requires_grad_() for t in qk]
    g = torch.rand(B, H, N, device=DEV)
    grads = torch.autograd.grad(sk.ScoredAttentionKL.apply(*leaves, sc), leaves, g)
    other = torch.ones(B, H, N, dtype=torch.bool, device=DEV)
    other[0, 1, 130:170] = False
    for setting, got2 in ((2, grads[:2]), (1, grads[2:])):
        for got, want, tol in zip(got2, *ref.grads(setting, g, BF16)):
            assert bool(((got.double() - want).abs() <= tol + 2.0 ** -8 * want.abs())[other].all())
            assert not bool(torch.isfinite(got[0, 1, 150]).all())
