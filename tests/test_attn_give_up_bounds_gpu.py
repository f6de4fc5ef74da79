"""A wait that gives up costs the rows of its own CTA, and no others: outputs and LSE elsewhere are the usual bits."""
import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk
from test_attn import inputs
from test_attn_calls import STALL, STALE
from test_cache8 import BF16, DEV, pool, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("shape", [(1, 1, 1, 9, 100, 64), (1, 4, 2, 300, 600, 128), (2, 8, 2, 1, 3000, 128), (1, 2, 2, 700, 1500, 64),
                                   (4, 64, 8, 300, 300, 64), (3, 32, 8, 1000, 1000, 128)], ids=str)
def test_forward(shape, splits, rest):
    """The first CTA has two tiles of up to 128 rows of the first key head."""
    t = inputs(*shape)
    want = sk.attn_fwd(*t, causal=True, num_splits=splits, rest=rest)
    out = torch.full_like(t[0], STALE)
    got = sk.attn_fwd(*t, causal=True, num_splits=splits, rest=rest, out=out, **STALL)
    lost = got[1].isnan()
    assert 1 <= int(lost.sum()) <= 256
    assert not bool(lost[1:].any()) and not bool(lost[:, shape[1] // shape[2]:].any())
    for a, b in zip(got, want):
        assert torch.equal(a[~lost], b[~lost]) and bool(a[lost].isnan().all())


@pytest.mark.parametrize("splits", [0, 1, 3, 20])
@pytest.mark.parametrize("group,Nq", [(1, 1), (4, 2), (4, 9), (8, 16)])
@pytest.mark.parametrize("lengths", [(1000, 300, 1024), (0, 700, 20), (16, 1, 1024)], ids=str)
def test_cache(lengths, group, Nq, splits):
    """The first CTA has a share of the first segment (sequence and key head), or the first share of all segments' keys."""
    B, Hk, T, d, M = 3, 2, 16, 128, 64
    table, pages = tables(B, M)
    cache = pool(pages, Hk, T, d)
    Q = torch.randn(B, group * Hk, Nq, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF16)
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    plan = sk.attn_cache8_plan(Q, cache, table, n, num_splits=splits)
    want = sk.attn_cache8(Q, cache, table, n, num_splits=splits)
    work = sk.new_workspace(plan.workspace_bytes, DEV)
    got = sk.attn_cache8(Q, cache, table, n, num_splits=splits, workspace=work, wait_limit_ns=10 ** 7, debug_flags=sk.DEBUG_INJECT_STALL)
    # chunks of 16 keys for 8-row tiles, of 32 for others, 256 keys in a step; equal shares in whole steps
    keys = 16 if group * Nq <= 8 else 32
    chunks = [-(-length // keys) for length in lengths]
    if plan.launches == 1:
        touched = 1
    else:
        step = 256 // keys
        share = max(-(-(-(-sum(chunks) * Hk // plan.num_ctas)) // step) * step, step)
        ends = torch.tensor([c for c in chunks for _ in range(Hk)]).cumsum(0)
        touched = int((ends < share).sum()) + 1
    segment = torch.arange(B * Hk, device=DEV).view(B, Hk, 1, 1).expand(B, Hk, group, Nq).reshape(B, Hk * group, Nq)
    out = segment >= touched
    assert bool(out.any()) or splits == 1  # one CTA takes all segments
    for a, b in zip(got, want):
        assert torch.equal(a[out], b[out])
    lost = got[1].isnan()
    live = want[1] > float("-inf")
    if plan.launches > 1 or lengths[0] > 0:
        assert sk.workspace_status(work) != 0 and bool(lost.any())
    assert torch.equal(lost, live & ~out) and torch.equal(got[0].isnan().all(-1), lost) and torch.equal(got[0].isnan().any(-1), lost)
