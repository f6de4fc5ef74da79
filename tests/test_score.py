"""Divergence of attentions with capped or biased scores and a key range per
row, and its gradients, against the definition in float64.

Tolerances, from the arithmetic.  A product z is a float32 sum of d exact
products, in any order off by at most d 2^-24 of the sum of their magnitudes; a
score adds a polynomial's 2^-23 and a few roundings of |S|.  With
A = max scale |q|.|k| and M = max |S| that is  del = (d + 32) 2^-24 A + 2^-20 M.
A key's error counts by its probability: for the rows' outputs M is the largest
sum over a row of P |S| (a bias makes far scores large and their P nothing).
LSE is off by at most del + a rounding; KL = E[S1 - S2] + LSE2 - LSE1 by
del (4 + 4 max |S1 - S2|) (each P is off by a factor 1 +- 2 del).  dS is off by
g (P1 + P2) 4 del (setting 1) or g P1 6 del (1 + |ratio - KL|) (setting 2) and
enters the gradient products as two bf16 terms (2^-16 of it) for float32
gradients and as one (rounded: 2^-8 of it) for bf16 gradients; the products
accumulate in float32 ((N + 128) 2^-24 of the sum of magnitudes).  bf16 outputs
add 2^-8 of the value.
"""
import ctypes
import math
import threading

import pytest
import torch

from attention_kl_divergence_gb300 import make_qk, streamkl as sk

gpu = pytest.mark.gpu
F64, BF16 = torch.float64, torch.bfloat16
DEV = "cuda"


# ---------------------------------------------------------------------------
# the definition in float64
# ---------------------------------------------------------------------------
def visible(begin, end, Nk):
    j = torch.arange(Nk, device=begin.device)
    return (j >= begin[..., None]) & (j < end[..., None])  # [B, Nq, Nk]


def scores64(Q, K, scale, cap, slopes, pos):
    """S [B, H, Nq, Nk] and the slope of the cap."""
    H, Hk, Nk = Q.shape[1], K.shape[1], K.shape[2]
    s = Q @ K.repeat_interleave(H // Hk, 1).transpose(2, 3) * scale
    slope = torch.ones_like(s)
    if cap > 0:
        t = torch.tanh(s / cap)
        s, slope = cap * t, 1 - t * t
    if slopes is not None:
        j = torch.arange(Nk, device=Q.device)
        s = s - slopes.double()[None, :, None, None] * (pos[:, None, :, None] - j).abs().double()
    return s, slope


def softmax64(s, vis):
    z = s.masked_fill(~vis, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None]).masked_fill(~vis, 0.0)
    return lse, p


class Ref:
    def __init__(self, Q1, K1, Q2, K2, begin, end, pos, scale=None, cap1=0.0, cap2=0.0, slopes1=None, slopes2=None):
        self.qk = [t.double() for t in (Q1, K1, Q2, K2)]
        Q1, K1, Q2, K2 = self.qk
        self.scale = Q1.shape[3] ** -0.5 if scale is None else scale
        self.vis = visible(begin, end, K1.shape[2])[:, None]
        s1, self.f1 = scores64(Q1, K1, self.scale, cap1, slopes1, pos)
        s2, self.f2 = scores64(Q2, K2, self.scale, cap2, slopes2, pos)
        self.L1, self.p1 = softmax64(s1, self.vis)
        self.L2, self.p2 = softmax64(s2, self.vis)
        self.live = self.vis.any(-1).expand_as(self.L1)
        z = torch.zeros_like(self.L1)
        ratio = (s1 - torch.where(self.live, self.L1, z)[..., None]) - (s2 - torch.where(self.live, self.L2, z)[..., None])
        self.ratio = ratio.masked_fill(~self.vis, 0.0)
        self.KL = (self.p1 * self.ratio).sum(-1)
        m = lambda t: float(t.masked_fill(~self.vis, 0.0).abs().max())  # noqa: E731
        G = Q1.shape[1] // K1.shape[1]
        A = max(m(q.abs() @ k.abs().repeat_interleave(G, 1).transpose(2, 3)) for q, k in ((Q1, K1), (Q2, K2))) * self.scale
        self.delta = (Q1.shape[3] + 32) * 2.0 ** -24 * A + 2.0 ** -20 * max(m(s1), m(s2))
        self.spread = m(s1 - s2)
        near = max(float((p * s.abs()).masked_fill(~self.vis, 0.0).sum(-1).max()) for p, s in ((self.p1, s1), (self.p2, s2)))
        weighted = float((self.p1 * (s1 - s2).abs()).masked_fill(~self.vis, 0.0).sum(-1).max())
        self.delta_row = (Q1.shape[3] + 32) * 2.0 ** -24 * A + 2.0 ** -20 * near
        self.spread_row = weighted

    def grads(self, setting, g, dtype=torch.float32):
        """(dQ, dK) and the bounds of their errors before the output's rounding."""
        Q1, K1, Q2, K2 = self.qk
        B, H, Nq, d = Q1.shape
        Hk, Nk = K1.shape[1], K1.shape[2]
        g = g.double()[..., None]
        dev = (self.ratio - self.KL[..., None]).masked_fill(~self.vis, 0.0)
        if setting == 1:
            dz, err, f, Q, K = g * (self.p2 - self.p1), g.abs() * (self.p1 + self.p2) * 4 * self.delta, self.f2, Q2, K2
        else:
            dz, err, f, Q, K = g * self.p1 * dev, g.abs() * self.p1 * (1 + dev.abs()) * 6 * self.delta, self.f1, Q1, K1
        dz = dz * f * self.scale
        err = err * self.scale + dz.abs() * (2.0 ** -16 + 2.0 ** -18 if dtype == torch.float32 else 2.0 ** -8)
        kx = K.repeat_interleave(H // Hk, 1)
        back = lambda t, q: (t.transpose(2, 3) @ q).reshape(B, Hk, H // Hk, Nk, d).sum(2)  # noqa: E731
        acc = 2.0 ** -24 * (max(Nk, Nq * (H // Hk)) + 128)
        dQ, dK = dz @ kx, back(dz, Q)
        return (dQ, dK), ((err + acc * dz.abs()) @ kx.abs() + 1e-30, back(err + acc * dz.abs(), Q.abs()) + 1e-30)

    def check_rows(self, KL, L1, L2):
        for got, want in ((L1, self.L1), (L2, self.L2)):
            got = got.double()
            assert torch.equal(got == -math.inf, ~self.live)
            err = (got - want)[self.live].abs()
            assert bool((err <= self.delta_row + 2.0 ** -23 * want[self.live].abs()).all()), float(err.max())
        err = (KL.double() - self.KL).abs()
        assert bool((KL[~self.live] == 0).all())
        # dKL = sum P1 (dS1 (ratio - KL) + dS1 - dS2) + dLSE: the spread counts by P1 too
        bound = self.delta_row * (4 + 4 * self.spread_row)
        assert bool((err <= bound).all()), (float(err.max()), bound)

    def check_grads(self, setting, g, dQ, dK):
        for name, got, want, tol in zip(("dQ", "dK"), (dQ, dK), *self.grads(setting, g, dQ.dtype)):
            if got.dtype == BF16:
                tol = tol + 2.0 ** -8 * want.abs()
            err = (got.double() - want).abs()
            assert bool((err <= tol).all()), (name, float((err / tol).max()))


def run_case(B, H, Hk, Nq, Nk, d, mask, cap1=0.0, cap2=0.0, bias=False, settings=(1, 2), peak=1.0, seed=0, scale=None,
             grad_dtype=torch.float32, num_splits=0, bwd_splits=0):
    Q1, K1, Q2, K2 = make_qk(B, H, Nq, Nk, d, 0.3, teacher_scale=peak, seed=seed, device=DEV, H_kv=Hk)
    begin, end, offset = mask(B, Nq, Nk)
    pos = torch.arange(Nq, device=DEV) + offset[:, None].long()
    s1 = torch.tensor([2.0 ** (-8 * (h + 1) / H) for h in range(H)], device=DEV) if bias else None
    s2 = s1 * 0.7 if bias else None
    sc = sk.Scores(cap1, cap2, s1, s2, begin, end, offset)
    ref = Ref(Q1, K1, Q2, K2, begin, end, pos, scale, cap1, cap2, s1, s2)
    rows = sk.kl_score_fwd(sc, Q1, K1, Q2, K2, scale=scale, num_splits=num_splits)
    ref.check_rows(*rows)
    g = torch.randn((B, H, Nq), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))
    for setting in settings:
        dQ, dK = sk.kl_score_bwd(setting, sc, g, Q1, K1, Q2, K2, *rows, scale=scale, grad_dtype=grad_dtype, num_splits=bwd_splits)
        assert dQ.dtype == dK.dtype == grad_dtype
        ref.check_grads(setting, g, dQ, dK)
    return ref


def ranges(**kw):
    def make(B, Nq, Nk):
        own = {k: (torch.tensor(v, dtype=torch.int32, device=DEV) if isinstance(v, list) else v) for k, v in kw.items()}
        return sk.key_ranges(B, Nq, Nk, DEV, **own)
    return make


def random_ranges(B, Nq, Nk):
    """Ranges of any kind: outside the keys, backwards, empty, one key wide."""
    g = torch.Generator().manual_seed(Nq + Nk)
    begin = torch.randint(-20, Nk + 20, (B, Nq), generator=g, dtype=torch.int32)
    end = begin + torch.randint(-10, Nk // 2 + 2, (B, Nq), generator=g, dtype=torch.int32)
    begin[:, ::7] = -2 ** 31
    end[:, ::11] = 2 ** 31 - 1
    offset = torch.randint(-5, 6, (B,), generator=g, dtype=torch.int32)
    return begin.to(DEV), end.to(DEV), offset.to(DEV)


CAUSAL, FULL = ranges(causal=True), ranges(causal=False)

# B, H, Hk, Nq, Nk, d, mask
PROBLEMS = {
    "one": (1, 1, 1, 1, 1, 64, CAUSAL),
    "one_row": (1, 2, 1, 1, 300, 128, CAUSAL),
    "seventeen": (1, 2, 2, 17, 17, 64, CAUSAL),
    "odd": (2, 4, 2, 130, 257, 128, CAUSAL),
    "docs": (2, 2, 1, 333, 333, 64, ranges(docs=[[0, 1, 100, 128, 129, 300], [0, 0, 64, 333, 333, 333]])),
    "window": (1, 2, 2, 300, 300, 128, ranges(window=37)),
    "window_both": (1, 2, 1, 200, 200, 64, ranges(causal=False, window=5)),
    "prefix": (2, 4, 4, 260, 260, 128, ranges(prefix=[150, 0])),
    "padded": (3, 2, 2, 200, 200, 128, ranges(q_lengths=[200, 1, 70], k_lengths=[200, 1, 70])),
    "empty_item": (2, 2, 1, 150, 150, 64, ranges(q_lengths=[0, 150], k_lengths=[0, 150])),
    "more_rows": (1, 2, 2, 300, 140, 64, CAUSAL),
    "decode": (3, 8, 2, 1, 1000, 128, ranges(k_lengths=[1000, 1, 513])),
    "decode_rows": (2, 4, 2, 5, 700, 64, ranges(k_lengths=[700, 3])),
    "decode_docs": (1, 4, 1, 4, 500, 128, ranges(docs=[0, 100, 498, 500])),
    "random": (2, 2, 1, 190, 310, 128, random_ranges),
    "random_decode": (2, 6, 2, 3, 400, 64, random_ranges),
    "full": (1, 3, 3, 64, 128, 128, FULL),
}
SCORES = {
    "plain": dict(),
    "capped": dict(cap1=50.0, cap2=50.0, peak=1.6),
    "low_cap": dict(cap1=2.0, cap2=5.0, peak=2.0),       # |scale z| up to many times the cap
    "huge_cap": dict(cap1=1000.0, cap2=60.0),            # no fixed reference for 2^1000
    "one_side": dict(cap2=20.0, peak=1.6),
    "bias": dict(bias=True),
    "all": dict(cap1=30.0, cap2=15.0, bias=True, peak=1.6),
}


@gpu
@pytest.mark.parametrize("kind", SCORES)
@pytest.mark.parametrize("problem", PROBLEMS)
def test_forward_and_gradients(problem, kind):
    B, H, Hk, Nq, Nk, d, mask = PROBLEMS[problem]
    run_case(B, H, Hk, Nq, Nk, d, mask, seed=Nq + Nk, **SCORES[kind])


@gpu
@pytest.mark.parametrize("mask", ["causal", "full", "prefix"])
@pytest.mark.parametrize("d", [64, 128])
def test_far_keys_cost_a_biased_row_no_precision(d, mask):
    """Steep and shallow slopes over a long row: scores of far keys reach -3000."""
    make = {"causal": CAUSAL, "full": FULL, "prefix": ranges(prefix=[1300])}[mask]
    run_case(1, 4, 2, 2100, 2100, d, make, bias=True, seed=5, settings=(1,), peak=1.6)
    run_case(1, 4, 2, 3, 2500, d, FULL if mask == "full" else CAUSAL, bias=True, seed=6, settings=(2,), cap1=30.0)


@gpu
@pytest.mark.parametrize("kind", ["plain", "capped", "all"])
def test_bf16_gradients_and_other_scale(kind):
    run_case(2, 4, 2, 150, 150, 128, ranges(docs=[0, 60, 150]), seed=3, grad_dtype=BF16, scale=0.2, **SCORES[kind])


@gpu
@pytest.mark.parametrize("splits", [1, 2, 5, 64])
@pytest.mark.parametrize("Nq", [2, 40])
def test_split_counts(Nq, splits):
    run_case(1, 4, 2, Nq, 900, 64, ranges(k_lengths=[770]), settings=(), num_splits=splits, cap1=30.0, cap2=30.0)
    run_case(1, 4, 2, Nq, 900, 64, random_ranges, settings=(), num_splits=splits, bias=True)


@gpu
@pytest.mark.parametrize("splits", [0, 5])
@pytest.mark.parametrize("kind", ["plain", "capped", "bias"])
def test_more_work_items_than_ctas_that_fit(kind, splits):
    """CTAs that take over the items of CTAs not started, most of them empty or short."""
    run_case(2, 32, 8, 300, 400, 64, random_ranges, seed=splits, num_splits=splits, settings=(1,), **SCORES[kind])
    lengths = [(37 * b) % 131 for b in range(24)]
    run_case(24, 16, 4, 130, 130, 64, ranges(q_lengths=lengths, k_lengths=lengths), num_splits=splits, settings=(2,), **SCORES[kind])


@gpu
def test_many_items_replay_from_a_graph_and_run_beside_another_stream():
    qk = make_qk(4, 32, 256, 256, 64, 0.3, seed=9, device=DEV, H_kv=8)
    begin, end, _ = ranges(docs=[0, 100, 256])(4, 256, 256)
    sc = sk.Scores(50.0, 50.0, begin=begin, end=end)
    want = sk.kl_score_fwd(sc, *qk)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = sk.kl_score_fwd(sc, *qk)
    for _ in range(3):
        graph.replay()
        with torch.cuda.stream(side):
            other = sk.kl_score_fwd(sc, *qk)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, other))


@gpu
@pytest.mark.parametrize("grad_dtype", [torch.float32, BF16])
@pytest.mark.parametrize("splits", [1, 3, 16, 64])
def test_backward_split_counts(splits, grad_dtype):
    """More splits than a key tile has iterations, too: some do nothing."""
    run_case(2, 4, 1, 200, 300, 128, ranges(docs=[0, 190, 300]), cap1=30.0, cap2=30.0, bwd_splits=splits, grad_dtype=grad_dtype)
    run_case(1, 2, 2, 130, 130, 64, random_ranges, bias=True, bwd_splits=splits, grad_dtype=grad_dtype)


@gpu
def test_long_decode_and_long_rows():
    run_case(2, 8, 2, 1, 50001, 128, ranges(k_lengths=[50001, 33333]), settings=(), cap1=50.0, cap2=50.0)
    run_case(1, 2, 1, 1500, 1500, 128, ranges(docs=[0, 700, 701, 1500]), cap1=50.0, cap2=30.0, peak=1.6)


@gpu
def test_agrees_with_the_unmodified_divergence():
    """Plain scores and a causal mask are what kl_fwd and kl_bwd compute."""
    Q1, K1, Q2, K2 = make_qk(1, 4, 300, 400, 128, 0.3, seed=1, device=DEV)
    a, b = sk.kl_fwd(Q1, K1, Q2, K2, causal=True), sk.kl_score_fwd(sk.Scores(), Q1, K1, Q2, K2, causal=True)
    for x, y in zip(a, b):
        assert float((x - y).abs().max()) <= 1e-4
    g = torch.rand(1, 4, 300, device=DEV)
    for setting in (1, 2):
        for x, y in zip(sk.kl_bwd(setting, g, Q1, K1, Q2, K2, *a, causal=True),
                        sk.kl_score_bwd(setting, sk.Scores(), g, Q1, K1, Q2, K2, *b, causal=True)):
            assert float((x - y).abs().max()) <= 1e-3 * float(x.abs().max())


@gpu
def test_agrees_with_the_unmodified_divergence_over_a_long_sequence():
    """20000 keys, shared by two query heads: windows of the whole length are the causal mask."""
    N = 20000
    qk = make_qk(1, 4, N, N, 128, 0.3, seed=12, device=DEV, H_kv=2)
    begin, end, _ = sk.key_ranges(1, N, N, DEV, window=N)
    a, b = sk.kl_fwd(*qk, causal=True), sk.kl_score_fwd(sk.Scores(begin=begin, end=end), *qk)
    for x, y in zip(a, b):
        assert float((x - y).abs().max()) <= 1e-4
    g = torch.rand(1, 4, N, device=DEV) / N
    for x, y in zip(sk.kl_bwd(1, g, *qk, *a, causal=True), sk.kl_score_bwd(1, sk.Scores(begin=begin, end=end), g, *qk, *b)):
        assert float((x - y).norm()) <= 1e-4 * float(x.norm())


@gpu
@pytest.mark.parametrize("kind", ["plain", "capped", "all"])
def test_difference_quotient(kind):
    """The gradients against differences of the forward's KL along random directions.  The inputs are bf16, so the
    forward's definition in float64 is differenced (which the other tests tie the forward to)."""
    kw = dict(SCORES[kind])
    bias, peak = kw.pop("bias", False), kw.pop("peak", 1.0)
    B, H, N, d = 1, 2, 40, 64
    Q1, K1, Q2, K2 = make_qk(B, H, N, N, d, 0.3, teacher_scale=peak, seed=8, device=DEV)
    begin, end, offset = sk.key_ranges(B, N, N, DEV, docs=torch.tensor([0, 13, 40], dtype=torch.int32, device=DEV))
    sl = torch.tensor([0.5, 0.1], device=DEV) if bias else None
    sc = sk.Scores(begin=begin, end=end, offset=offset, slopes1=sl, slopes2=sl, **kw)
    pos = torch.arange(N, device=DEV)[None]
    rows = sk.kl_score_fwd(sc, Q1, K1, Q2, K2)
    g = torch.rand(B, H, N, device=DEV)
    for setting, side in ((1, 2), (2, 0)):
        grads = sk.kl_score_bwd(setting, sc, g, Q1, K1, Q2, K2, *rows)
        for k in range(2):
            x = [t.double() for t in (Q1, K1, Q2, K2)]
            v = torch.randn(x[side + k].shape, device=DEV, dtype=F64, generator=torch.Generator(device=DEV).manual_seed(k))

            def f(h):
                y = list(x)
                y[side + k] = x[side + k] + h * v
                return float((Ref(*y, begin, end, pos, None, slopes1=sl, slopes2=sl, **kw).KL * g.double()).sum())

            want = (f(1e-5) - f(-1e-5)) / 2e-5
            got = float((grads[k].double() * v).sum())
            assert abs(got - want) <= 1e-3 * float(grads[k].double().norm() * 1.0) + 1e-6, (setting, k, got, want)


BAD = [float("nan"), float("inf"), -float("inf"), 3.0e38]


@gpu
@pytest.mark.parametrize("value", BAD)
@pytest.mark.parametrize("kind", ["plain", "capped", "all"])
@pytest.mark.parametrize("d", [64, 128])
def test_hidden_values_have_no_effect(d, kind, value):
    """Rows behind each sequence of a padded batch hold NaN, infinities or huge values, in every input."""
    kw = dict(SCORES[kind])
    bias, peak = kw.pop("bias", False), kw.pop("peak", 1.0)
    B, H, Hk, N = 2, 2, 1, 200
    n = [90, 161]
    qk = make_qk(B, H, N, N, d, 0.3, teacher_scale=peak, seed=d, device=DEV, H_kv=Hk)
    L = torch.tensor(n, dtype=torch.int32, device=DEV)
    begin, end, offset = sk.key_ranges(B, N, N, DEV, q_lengths=L, k_lengths=L)
    sl = torch.tensor([0.5, 0.1], device=DEV) if bias else None
    sc = sk.Scores(begin=begin, end=end, offset=offset, slopes1=sl, slopes2=sl, **kw)
    pos = torch.arange(N, device=DEV).expand(B, N)
    ref = Ref(*qk, begin, end, pos, None, slopes1=sl, slopes2=sl, **kw)
    clean = sk.kl_score_fwd(sc, *qk)
    dirty = [t.clone() for t in qk]
    for t in dirty:
        for b in range(B):
            t[b, :, n[b]:] = value
    rows = sk.kl_score_fwd(sc, *dirty)
    assert all(torch.equal(a, b) for a, b in zip(rows, clean))
    g = torch.randn(B, H, N, device=DEV)
    rows = [t.clone() for t in rows]
    for setting in (1, 2):
        dQ, dK = sk.kl_score_bwd(setting, sc, g, *dirty, *rows)
        ref.check_grads(setting, g, dQ, dK)
        for b in range(B):
            assert bool((dQ[b, :, n[b]:] == 0).all()) and bool((dK[b, :, n[b]:] == 0).all())


@gpu
@pytest.mark.parametrize("value", BAD[:3])
@pytest.mark.parametrize("where", [0, 1, 2, 3])
def test_a_bad_token_stays_in_its_document(where, value):
    B, H, N, d = 1, 2, 300, 128
    qk = list(make_qk(B, H, N, N, d, 0.3, seed=4, device=DEV))
    begin, end, offset = sk.key_ranges(B, N, N, DEV, docs=torch.tensor([0, 130, 170, 300], dtype=torch.int32, device=DEV))
    sc = sk.Scores(50.0, 50.0, begin=begin, end=end, offset=offset)
    pos = torch.arange(N, device=DEV)[None]
    ref = Ref(*qk, begin, end, pos, None, 50.0, 50.0)
    qk[where] = qk[where].clone()
    qk[where][0, 1, 150, 7] = value
    rows = sk.kl_score_fwd(sc, *qk)
    other = torch.ones(B, H, N, dtype=torch.bool, device=DEV)
    other[0, 1, 130:170] = False
    for got, want in zip(rows, (ref.KL, ref.L1, ref.L2)):
        assert bool(((got.double() - want).abs() <= ref.delta * (4 + 4 * ref.spread))[other].all())
    assert bool(torch.isfinite(rows[0][0, 1, 130:150]).all()) and not bool(torch.isfinite(rows[0][0, 1, 150]))
    g = torch.rand(B, H, N, device=DEV)
    for setting in (1, 2):
        grads = sk.kl_score_bwd(setting, sc, g, *qk, *rows)
        for got, want, tol in zip(grads, *ref.grads(setting, g)):
            assert bool(((got.double() - want).abs() <= tol)[other].all())
            assert not bool(torch.isfinite(got[0, 1, 150]).all())


@gpu
def test_strided_views_and_large_strides():
    B, H, Hk, N, d = 2, 4, 2, 140, 128
    g = torch.Generator().manual_seed(11)
    t = lambda h: (torch.randn((B, N, h, d), generator=g) * 0.5).to(BF16).to(DEV).transpose(1, 2)  # noqa: E731
    qk = [t(H), t(Hk), t(H), t(Hk)]
    begin, end, offset = CAUSAL(B, N, N)
    ref = Ref(*qk, begin, end, torch.arange(N, device=DEV).expand(B, N), None, 20.0, 20.0)
    sc = sk.Scores(20.0, 20.0, begin=begin, end=end)
    rows = sk.kl_score_fwd(sc, *qk)
    ref.check_rows(*rows)
    up = torch.rand(B, H, N, device=DEV)
    ref.check_grads(2, up, *sk.kl_score_bwd(2, sc, up, *qk, *rows))
    # key caches whose second item lies past 2^31 elements
    step = 2 ** 31 + 64
    caches = []
    for k in (qk[1], qk[3]):
        c = torch.empty(step + Hk * N * d, dtype=BF16, device=DEV).as_strided((B, Hk, N, d), (step, N * d, d, 1))
        c.copy_(k)
        caches.append(c)
    for rows_of in (slice(None), slice(N - 1, N)):
        q1, q2 = qk[0][:, :, rows_of].contiguous(), qk[2][:, :, rows_of].contiguous()
        b, e = begin[:, rows_of].contiguous(), end[:, rows_of].contiguous()
        want = sk.kl_score_fwd(sk.Scores(20.0, 20.0, begin=b, end=e), q1, qk[1].contiguous(), q2, qk[3].contiguous())
        got = sk.kl_score_fwd(sk.Scores(20.0, 20.0, begin=b, end=e), q1, caches[0], q2, caches[1])
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@gpu
def test_autograd_function_settings():
    qk = make_qk(1, 4, 90, 90, 64, 0.3, seed=2, device=DEV, H_kv=2)
    begin, end, offset = ranges(docs=[0, 40, 90])(1, 90, 90)
    sc = sk.Scores(50.0, 30.0, begin=begin, end=end, offset=offset)
    g = torch.rand(1, 4, 90, device=DEV)
    leaves = [t.clone().requires_grad_() for t in qk]
    KL = sk.ScoredAttentionKL.apply(*leaves, sc)
    grads = torch.autograd.grad(KL, leaves, g)
    ref = Ref(*qk, begin, end, torch.arange(90, device=DEV)[None], None, 50.0, 30.0)
    ref.check_grads(2, g, *grads[:2])
    ref.check_grads(1, g, *grads[2:])
    student = [qk[0], qk[1], leaves[2], qk[3]]
    (dQ,) = torch.autograd.grad(sk.ScoredAttentionKL.apply(*student, sc).sum(), leaves[2])  # a broadcast upstream gradient
    (want, _), (tol, _) = ref.grads(1, torch.ones_like(g), BF16)
    assert bool(((dQ.double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all())
    with pytest.raises(ValueError):
        sk.ScoredAttentionKL.apply(*leaves, sk.Scores(slopes1=torch.ones(4, device=DEV, requires_grad=True)))


@gpu
def test_wait_limit_is_shorter_than_a_work_item():
    """The limit holds for a step of the pipeline, not for a row's whole length: 320 work items of 8192 key tiles
    take several milliseconds each, with a limit of 2."""
    B, H, N, M, d = 1, 320, 17, 1 << 20, 64
    x = [0.3 * torch.randn(B, h, n, d, device=DEV).to(BF16) for h, n in ((H, N), (1, M), (H, N), (1, M))]
    for sc in (sk.Scores(), sk.Scores(50.0, 50.0)):
        plan = sk.score_fwd_plan(x[0], x[1], num_splits=1)
        assert plan.num_ctas > torch.cuda.get_device_properties(0).multi_processor_count
        ws = sk.new_workspace(plan.workspace_bytes, DEV)
        got = sk.kl_score_fwd(sc, *x, num_splits=1, workspace=ws, wait_limit_ns=2_000_000)
        assert sk.workspace_status(ws) == 0
        want = sk.kl_score_fwd(sc, *x, num_splits=1)
        for a, b in zip(got, want):
            assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


@gpu
def test_first_call_of_a_host_thread():
    """A thread that has made no CUDA call yet, with every buffer at hand: nothing before the library's own calls
    binds the device's context to it."""
    qk = make_qk(1, 2, 64, 64, 64, 0.3, seed=2, device=DEV)
    g = torch.ones(1, 2, 64, device=DEV)
    ws = sk.new_workspace(1 << 20, DEV)
    rows = [torch.empty(1, 2, 64, device=DEV) for _ in range(3)]
    grads = [torch.empty(1, 2, 64, 64, device=DEV) for _ in range(2)]
    calls = [lambda: sk.kl_score_fwd(sk.Scores(), *qk, workspace=ws, out=rows),
             lambda: sk.kl_score_bwd(1, sk.Scores(), g, *qk, *rows, workspace=ws, out=grads),
             lambda: sk.kl_fwd(*qk, workspace=ws, out=rows)]
    for call in calls:
        call()
        torch.cuda.synchronize()
        failed = []

        def work():
            try:
                call()
            except Exception as e:
                failed.append(e)

        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not failed, failed


@gpu
def test_replays_from_a_graph_on_another_stream():
    qk = make_qk(2, 4, 200, 200, 128, 0.3, seed=7, device=DEV)
    L = torch.tensor([200, 120], dtype=torch.int32, device=DEV)
    g = torch.rand(2, 4, 200, device=DEV)

    def step():
        begin, end, offset = sk.key_ranges(2, 200, 200, DEV, q_lengths=L, k_lengths=L)
        sc = sk.Scores(50.0, 50.0, begin=begin, end=end, offset=offset)
        rows = sk.kl_score_fwd(sc, *qk)
        return rows + sk.kl_score_bwd(1, sc, g, *qk, *rows, grad_dtype=BF16)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for lengths in ([200, 120], [3, 199]):
        L.copy_(torch.tensor(lengths, dtype=torch.int32))
        want = step()
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
        assert torch.equal(got[4], want[4])  # dK: each CTA's own sum
        assert float((got[3].float() - want[3].float()).abs().max()) <= 2.0 ** -7 * float(want[3].float().abs().max())


@gpu
@pytest.mark.parametrize("H,Nq", [(2, 8), (2, 300), (128, 300)])
def test_bounded_waits_give_up_and_are_reported(H, Nq):
    """Test aid: the first CTA waits on a barrier that nothing arrives on, for 20 ms.  128 heads: more work items than
    fit at a time, which the other CTAs take over."""
    qk = make_qk(1, H, Nq, 300, 128, 0.3, seed=5, device=DEV)
    sc = sk.Scores(50.0, 50.0)
    ws = sk.new_workspace(max(sk.score_fwd_plan(qk[0], qk[1]).workspace_bytes,
                              sk.score_bwd_plan(qk[0], qk[1], 1).workspace_bytes), DEV)
    rows = sk.kl_score_fwd(sc, *qk, workspace=ws, wait_limit_ns=20_000_000, debug_flags=sk.DEBUG_INJECT_STALL)
    assert sk.workspace_status(ws) != 0 and bool(torch.isnan(rows[0]).any())
    rows = sk.kl_score_fwd(sc, *qk, workspace=ws)
    assert sk.workspace_status(ws) == 0 and bool(torch.isfinite(rows[0]).all())
    g = torch.rand(1, H, Nq, device=DEV)
    sk.kl_score_bwd(1, sc, g, *qk, *rows, workspace=ws, wait_limit_ns=20_000_000, debug_flags=sk.DEBUG_INJECT_STALL)
    assert sk.workspace_status(ws) != 0
    want = sk.kl_score_bwd(1, sc, g, *qk, *rows)
    got = sk.kl_score_bwd(1, sc, g, *qk, *rows, workspace=ws)
    assert sk.workspace_status(ws) == 0 and torch.equal(got[1], want[1])


# ---------------------------------------------------------------------------
# key ranges
# ---------------------------------------------------------------------------
def ranges_plain(B, Nq, Nk, causal, window, prefix, docs, ql, kl):
    """Row by row, from the set of visible keys."""
    begin, end = [[0] * Nq for _ in range(B)], [[0] * Nq for _ in range(B)]
    off = []
    for b in range(B):
        q, k = (Nq if ql is None else ql[b]), (Nk if kl is None else kl[b])
        off.append(k - q)
        bounds = None if docs is None else (docs[b] if isinstance(docs[0], list) else docs)
        for i in range(q):
            p = i + k - q
            keys = [j for j in range(k) if (not causal or j <= p or (prefix is not None and j < prefix[b]))
                    and (not window or p - window < j < p + window)
                    and (bounds is None or any(lo <= p < hi and lo <= j < hi for lo, hi in zip(bounds, bounds[1:])))]
            if keys:
                assert keys == list(range(keys[0], keys[-1] + 1))
                begin[b][i], end[b][i] = keys[0], keys[-1] + 1
    return begin, end, off


@gpu
@pytest.mark.parametrize("B,Nq,Nk,kw", [
    (1, 1, 1, {}),
    (2, 30, 30, dict(q_lengths=[30, 0], k_lengths=[30, 0])),
    (2, 5, 40, dict(k_lengths=[40, 3])),
    (2, 33, 20, {}),
    (1, 40, 40, dict(window=1)),
    (1, 40, 50, dict(window=7, causal=False)),
    (2, 300, 300, dict(docs=[0, 5, 5, 20, 290])),
    (2, 25, 25, dict(docs=[[0, 10, 25], [3, 20, 20]], causal=False)),
    (1, 25, 30, dict(docs=[0, 10, 28, 30], window=4)),
    (2, 20, 20, dict(prefix=[12, 0], q_lengths=[20, 7], k_lengths=[20, 7])),
    (2, 20, 20, dict(prefix=[99, 5], k_lengths=[18, 20])),
])
def test_key_ranges(B, Nq, Nk, kw):
    got = sk.key_ranges(B, Nq, Nk, DEV, **{k: torch.tensor(v, dtype=torch.int32, device=DEV) if isinstance(v, list) else v
                                           for k, v in kw.items()})
    want = ranges_plain(B, Nq, Nk, kw.get("causal", True), kw.get("window", 0), kw.get("prefix"), kw.get("docs"),
                        kw.get("q_lengths"), kw.get("k_lengths"))
    assert [t.tolist() for t in got] == list(want)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
@gpu
def test_refusals():
    qk = make_qk(2, 4, 40, 40, 64, 0.3, device=DEV, H_kv=2)
    begin, end, offset = CAUSAL(2, 40, 40)
    i32 = dict(dtype=torch.int32, device=DEV)

    def bad(scores, q=qk, **kw):
        with pytest.raises((ValueError, sk.StreamKLError)):
            sk.kl_score_fwd(scores, *q, **kw)

    bad(None)
    bad(sk.Scores(begin=begin[:1]))
    bad(sk.Scores(begin=begin.long()))
    bad(sk.Scores(end=end.cpu()))
    bad(sk.Scores(end=end.t().contiguous().t()))
    bad(sk.Scores(offset=offset[:1]))
    bad(sk.Scores(slopes1=torch.ones(2, device=DEV)))
    bad(sk.Scores(slopes2=torch.ones(4, dtype=F64, device=DEV)))
    bad(sk.Scores(cap1=-1.0))
    bad(sk.Scores(cap2=float("nan")))
    bad(sk.Scores(cap2=float("inf")))
    bad(sk.Scores(cap1=1e9))    # scale / cap below what the polynomials carry
    bad(sk.Scores(cap1=1e-8))
    bad(sk.Scores(), q=[t.float() for t in qk])
    bad(sk.Scores(), q=[t.cpu() for t in qk])
    bad(sk.Scores(), q=[t[:, :, :0] for t in qk])
    bad(sk.Scores(), workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    bad(sk.Scores(), num_splits=-1)
    rows = sk.kl_score_fwd(sk.Scores(), *qk)
    g = torch.ones(2, 4, 40, device=DEV)
    for args in ((3, sk.Scores(), g, *qk, *rows), (1, sk.Scores(), g[:1], *qk, *rows), (1, sk.Scores(), g.double(), *qk, *rows),
                 (1, sk.Scores(cap1=-2.0), g, *qk, *rows)):
        with pytest.raises((ValueError, sk.StreamKLError)):
            sk.kl_score_bwd(*args)
    with pytest.raises(ValueError):
        sk.kl_score_bwd(1, sk.Scores(), g, *qk, *rows, grad_dtype=torch.float16)
    for kw in (dict(window=-1), dict(prefix=torch.ones(2, **i32), window=3), dict(docs=torch.zeros(1, **i32)),
               dict(docs=torch.zeros(3, 4, **i32)), dict(prefix=torch.ones(3, **i32)), dict(q_lengths=[1, 2])):
        with pytest.raises((ValueError, sk.StreamKLError)):
            sk.key_ranges(2, 40, 40, DEV, **kw)
    with pytest.raises(ValueError):
        sk.key_ranges(2, 40, 40, "cpu")


def _shape(**kw):
    s = dict(B=1, H=2, Nq=256, Nk=256, d=64, H_kv=0)
    s.update(kw)
    d, Nq, Nk, H = s["d"], s["Nq"], s["Nk"], s["H"]
    return sk.Shape(s["B"], H, Nq, Nk, d, H * Nq * d, Nq * d, d, H * Nk * d, Nk * d, d, s["H_kv"])


def test_abi_rejects_bad_arguments_without_a_device():
    lib, P = sk.load(), ctypes.c_void_p

    def fwd(shape, score=None, ptrs=(256,) * 7, ws=256):
        return lib.streamkl_score_fwd(ctypes.byref(shape) if shape else None, ctypes.byref(score) if score else None,
                                      *[P(p) for p in ptrs[:4]], ctypes.c_float(0.0), 1, *[P(p) for p in ptrs[4:]], P(ws),
                                      4096, None, P(0))

    def bwd(shape, score=None, ptrs=(256,) * 10, ws=256, setting=1):
        return lib.streamkl_score_bwd(ctypes.byref(shape) if shape else None, ctypes.byref(score) if score else None, setting,
                                      *[P(p) for p in ptrs[:8]], ctypes.c_float(0.0), 1, *[P(p) for p in ptrs[8:]], P(ws),
                                      4096, None, P(0))

    for call, n in ((fwd, 7), (bwd, 10)):
        assert call(None) == sk.ERR_INVALID_ARG
        assert call(_shape(B=0)) == sk.ERR_INVALID_ARG
        assert call(_shape(Nq=0)) == sk.ERR_INVALID_ARG
        assert call(_shape(Nk=0)) == sk.ERR_INVALID_ARG
        assert call(_shape(d=96)) == sk.ERR_UNSUPPORTED
        assert call(_shape(H=6, H_kv=4)) == sk.ERR_INVALID_ARG
        for i in range(n):
            assert call(_shape(), ptrs=tuple(0 if j == i else 256 for j in range(n))) == sk.ERR_INVALID_ARG
        for cap in (-1.0, float("nan"), float("inf")):
            assert call(_shape(), sk.Score(cap, 0.0)) == sk.ERR_INVALID_ARG
            assert call(_shape(), sk.Score(0.0, cap)) == sk.ERR_INVALID_ARG
        assert call(_shape(), sk.Score(1e9, 0.0)) == sk.ERR_UNSUPPORTED
        for k in range(5):
            assert call(_shape(), sk.Score(0.0, 0.0, *(258 if j == k else 256 for j in range(5)))) == sk.ERR_INVALID_ARG
        assert call(_shape(), ws=0) == sk.ERR_WORKSPACE
        assert call(_shape(), ws=8) == sk.ERR_WORKSPACE
    assert bwd(_shape(), setting=3) == sk.ERR_INVALID_ARG

    def rng(B=1, Nq=4, Nk=4, window=0, prefix=0, docs=0, n=0, out=(256, 256, 256)):
        return lib.streamkl_key_ranges(B, Nq, Nk, 1, window, P(0), P(0), P(prefix), P(docs), n, 0, *[P(o) for o in out], P(0))

    assert rng(B=0) == rng(Nq=0) == rng(Nk=0) == rng(window=-1) == rng(docs=256, n=1) == rng(n=3) == sk.ERR_INVALID_ARG
    assert rng(out=(0, 256, 256)) == rng(out=(256, 258, 256)) == sk.ERR_INVALID_ARG
    assert rng(prefix=256, window=2) == rng(prefix=256, docs=256, n=2) == sk.ERR_UNSUPPORTED
