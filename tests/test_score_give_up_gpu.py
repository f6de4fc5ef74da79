"""After a bounded wait has given up, every output holds its value or NaN, never
what was in memory before: the caller may have dropped the workspace with the
status word.

The test aid makes the first CTA wait on a barrier that nothing arrives on, for
20 ms.  Outputs and workspace hold finite values beforehand.
"""
import pytest
import torch

from attention_kl_divergence_gb300 import make_qk, streamkl as sk
from test_score import BF16, DEV, ranges

pytestmark = pytest.mark.gpu
STALL = dict(wait_limit_ns=20_000_000, debug_flags=sk.DEBUG_INJECT_STALL)
STALE = 7.0


def stale_workspace(nbytes):
    ws = torch.full(((nbytes + 255) // 256 * 64,), STALE, dtype=torch.float32, device=DEV).view(torch.uint8)
    ws[:256] = 0
    return ws


def right_or_nan(got, want):
    """The rows of `got` that are marked; the others are `want` bit for bit."""
    lost = torch.isnan(got)
    assert bool((lost | (got == want)).all())
    return lost


# H, Nq, splits: decode; fewer work items than SMs; more, so that the stalled CTA has claimed another one; with parts of rows
CASES = [(2, 8, 0), (2, 8, 3), (2, 300, 1), (2, 300, 2), (128, 300, 1), (128, 300, 2), (40, 2000, 1)]


@pytest.mark.parametrize("kind", ["plain", "capped"])
@pytest.mark.parametrize("H,Nq,splits", CASES)
def test_forward_rows_are_right_or_marked(H, Nq, splits, kind):
    qk = make_qk(1, H, Nq, 600, 64, 0.3, seed=5, device=DEV, H_kv=2)
    begin, end, offset = ranges(docs=[0, 250, 600])(1, Nq, 600) if Nq < 600 else (None, None, None)
    sc = sk.Scores(*((50.0, 50.0) if kind == "capped" else (0.0, 0.0)), begin=begin, end=end, offset=offset)
    want = sk.kl_score_fwd(sc, *qk, num_splits=splits)
    ws = stale_workspace(sk.score_fwd_plan(*qk[:2], num_splits=splits).workspace_bytes)
    out = tuple(torch.full_like(t, STALE) for t in want)
    sk.kl_score_fwd(sc, *qk, num_splits=splits, workspace=ws, out=out, **STALL)
    assert sk.workspace_status(ws) != 0
    lost = [right_or_nan(a, b) for a, b in zip(out, want)]
    assert bool(lost[0].any()) and all(torch.equal(lost[0], t) for t in lost)
    # an autograd user has the outputs alone
    assert bool(torch.isnan(sk.kl_score_fwd(sc, *qk, num_splits=splits, **STALL)[0]).any())
    got = sk.kl_score_fwd(sc, *qk, num_splits=splits, workspace=ws, out=out)
    assert sk.workspace_status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


# H, Nq, splits, type: one part of dK, several; bf16 goes through float32 sums of dQ
@pytest.mark.parametrize("setting", [1, 2])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("d,Nq,splits", [(64, 8, 1), (64, 300, 1), (128, 300, 3), (128, 600, 2)])
def test_gradients_are_right_or_marked(d, Nq, splits, dtype, setting):
    qk = make_qk(1, 4, Nq, 600, d, 0.3, seed=5, device=DEV, H_kv=2)
    sc = sk.Scores(50.0, 50.0)
    rows = sk.kl_score_fwd(sc, *qk)
    g = torch.rand(1, 4, Nq, device=DEV)
    want = sk.kl_score_bwd(setting, sc, g, *qk, *rows, num_splits=splits, grad_dtype=dtype)
    ws = stale_workspace(sk.score_bwd_plan(*qk[:2], setting, grad_dtype=dtype, num_splits=splits).workspace_bytes)
    out = tuple(torch.full_like(t, STALE) for t in want)
    sk.kl_score_bwd(setting, sc, g, *qk, *rows, num_splits=splits, grad_dtype=dtype, workspace=ws, out=out, **STALL)
    assert sk.workspace_status(ws) != 0
    # the first CTA: the first key tile of the first key head, and rows of its two query heads
    lost = right_or_nan(out[1], want[1])
    assert bool(lost[0, 0, :128].all()) and not bool(lost[0, 0, 128:].any()) and not bool(lost[0, 1].any())
    lost = torch.isnan(out[0])
    assert bool(lost.any()) and not bool(lost[0, 2:].any()) and bool(lost.eq(lost[..., :1]).all())
    # sums of up to 5 key tiles in another order: 2 * 5 * 2^-24 of the magnitudes, taken as the largest value; one step of bf16
    near = (out[0].double() - want[0].double()).abs() <= 1e-5 * want[0].double().abs().max() + \
        (2.0 ** -7 * want[0].double().abs() if dtype == BF16 else 0)
    assert bool((lost | near).all())
    got = sk.kl_score_bwd(setting, sc, g, *qk, *rows, num_splits=splits, grad_dtype=dtype, workspace=ws, out=out)
    assert sk.workspace_status(ws) == 0 and torch.equal(got[1], want[1]) and bool(torch.isfinite(got[0].float()).all())
