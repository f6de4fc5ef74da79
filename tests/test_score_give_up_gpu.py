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
