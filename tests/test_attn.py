"""Attention over whole prompts and its gradients against the definition in float64.

Tolerances, from the arithmetic.  A product z is a float32 sum of d exact
products, off by at most d 2^-24 of the sum of their magnitudes; the exponent
adds a few roundings of |S|.  With A = max scale |q|.|k| and M = max |S| over
the visible pairs a score is off by  del = (d + 32) 2^-24 A + 2^-20 (M + 1).
LSE is off by at most del + N 2^-24 (the sum of up to N terms) + its rounding.
A probability enters the product with V rounded to bf16 (2^-8 of it) from a
value off by a factor 1 +- 2 del, the product accumulates in float32, and O is
rounded once:  (2^-8 + 4 del + (N + 128) 2^-24) sum P |V| + 2^-8 |O|.  With `rest`
they are two bf16 terms, off by 2^-16, and O + rest is off by
(2^-16 + 4 del + (N + 128) 2^-24) sum P |V| + 2^-16 |O|.

Gradients.  P is off by a factor 1 +- 2 del and enters dV rounded (2^-8 of it).
dP is a float32 sum, off by (d + 32) 2^-24 of |dO| |V|^T; D is a float32 sum of
products with O + rest.  dS = P (dP - D) takes its share of all of these; it
enters dQ and dK as two terms (2^-16), sums are float32 ((N + 128) 2^-24 of the
magnitudes), outputs are rounded once (2^-8).
"""
import math

import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk

gpu = pytest.mark.gpu
F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
DEV = "cuda"


def inputs(B, H, Hk, Nq, Nk, d, seed=0, peak=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    new = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    return (new(B, H, Nq, d) * peak).to(BF16), (new(B, Hk, Nk, d) * peak).to(BF16), new(B, Hk, Nk, d).to(BF16)


class Ref:
    """The definition in 64 bits, and the bounds of the errors."""

    def __init__(self, Q, K, V, ranges=None, causal=False, scale=None):
        B, H, Nq, d = Q.shape
        Hk, Nk = K.shape[1], K.shape[2]
        self.G, self.Hk = H // Hk, Hk
        self.scale = d ** -0.5 if scale is None else scale
        j = torch.arange(Nk, device=DEV)
        begin, end, offset = ranges if ranges is not None else (None, None, None)
        lo = torch.zeros((B, Nq), dtype=torch.int64, device=DEV) if begin is None else begin.long()
        hi = torch.full((B, Nq), Nk, dtype=torch.int64, device=DEV) if end is None else end.long()
        if causal:
            off = torch.full((B,), Nk - Nq, device=DEV) if offset is None else offset.long()
            hi = torch.minimum(hi, torch.arange(Nq, device=DEV) + off[:, None] + 1)
        self.vis = ((j >= lo[..., None]) & (j < hi[..., None]))[:, None]
        rep = lambda t: t.double().repeat_interleave(self.G, 1)  # noqa: E731
        self.q, self.k, self.v = Q.double(), rep(K), rep(V)
        s = (self.q @ self.k.transpose(2, 3) * self.scale).masked_fill(~self.vis, -math.inf)
        self.LSE = torch.logsumexp(s, -1)
        self.live = self.vis.any(-1).expand_as(self.LSE)
        self.p = torch.exp(s - torch.where(self.live, self.LSE, 0.0)[..., None]).masked_fill(~self.vis, 0.0)
        v = self.v if bool(torch.isfinite(self.v).all()) else torch.nan_to_num(self.v, 0.0, 0.0, 0.0)
        self.O = self.p @ v
        big = lambda t: float(torch.nan_to_num(t).masked_fill(~self.vis, 0.0).abs().max())  # noqa: E731
        A = big(self.q.abs() @ self.k.abs().transpose(2, 3)) * self.scale
        self.delta = (d + 32) * 2.0 ** -24 * A + 2.0 ** -20 * (big(s) + 1)
        self.acc = (Nk + 128) * 2.0 ** -24
        mag = self.p @ v.abs()
        self.o_tol = (2.0 ** -8 + 4 * self.delta + self.acc) * mag + 2.0 ** -8 * self.O.abs() + 1e-30
        self.two_terms = (2.0 ** -16 + 4 * self.delta + self.acc) * mag + 2.0 ** -16 * self.O.abs() + 1e-30

    def grads(self, dO):
        """(dQ, dK, dV) and the bounds of their errors but for the outputs' rounding."""
        B, H, Nq, d = self.q.shape
        Nk = self.k.shape[2]
        g = dO.double().masked_fill(~self.live[..., None], 0.0)
        back = lambda t: t.reshape(B, self.Hk, self.G, Nk, d).sum(2)  # noqa: E731
        mag = g.abs() @ self.v.abs().transpose(2, 3)
        dP = g @ self.v.transpose(2, 3)
        D = (g * self.O).sum(-1, keepdim=True)
        d_err = ((self.two_terms + (d + 32) * 2.0 ** -24 * self.O.abs()) * g.abs()).sum(-1, keepdim=True)
        dS = self.p * (dP - D) * self.scale
        err = self.p * self.scale * (2 * self.delta * (dP - D).abs() + (d + 32) * 2.0 ** -24 * mag + d_err)
        acc = 2.0 ** -24 * (max(Nk, Nq * self.G) + 128)
        want = dS @ self.k, back(dS.transpose(2, 3) @ self.q), back(self.p.transpose(2, 3) @ g)
        tol = ((err + (2.0 ** -16 + acc) * dS.abs()) @ self.k.abs(),
               back((err + (2.0 ** -16 + acc) * dS.abs()).transpose(2, 3) @ self.q.abs()),
               back((self.p * (2.0 ** -8 + 2 * self.delta + acc)).transpose(2, 3) @ g.abs()))
        return want, tol

    def check_grads(self, dO, dQ, dK, dV):
        for name, got, w, t in zip(("dQ", "dK", "dV"), (dQ, dK, dV), *self.grads(dO)):
            bound = t * 1.01 + 2.0 ** -8 * w.abs() + 1e-30  # 1.01: products of the terms above
            e = (got.double() - w).abs()
            assert bool((e <= bound).all()), (name, float((e / bound).max()))

    def check(self, O, LSE):
        assert torch.equal(LSE == -math.inf, ~self.live)
        err = (LSE.double() - self.LSE)[self.live].abs()
        tol = self.delta + self.acc + 2.0 ** -23 * self.LSE[self.live].abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        assert bool((O[~self.live] == 0).all())
        err = (O.double() - self.O).abs()
        assert bool((err <= self.o_tol).all()), float((err / self.o_tol).max())


def masks(kind, B, Nq, Nk):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if kind == "full":
        return sk.key_ranges(B, Nq, Nk, DEV, causal=False)
    if kind == "causal":
        return sk.key_ranges(B, Nq, Nk, DEV)
    if kind == "window":
        return sk.key_ranges(B, Nq, Nk, DEV, window=max(1, Nk // 5))
    if kind == "docs":
        bounds = sorted({0, Nk // 7, Nk // 7 + 1, Nk // 2, Nk - Nk // 9, Nk})
        return sk.key_ranges(B, Nq, Nk, DEV, docs=i32(*bounds))
    if kind == "padded":
        n = [max(1, Nk - b * (Nk // 3) - (b > 0)) for b in range(B)]
        return sk.key_ranges(B, Nq, Nk, DEV, q_lengths=i32(*[min(Nq, x) for x in n]), k_lengths=i32(*n))
    assert kind == "two ends"  # rows in turn see keys at the start and at the end; every fifth row nothing
    row = torch.arange(Nq, device=DEV)
    begin = torch.where(row % 2 == 0, 0, max(0, Nk - 3)).int().repeat(B, 1)
    end = torch.where(row % 2 == 0, min(2, Nk), Nk).int().repeat(B, 1)
    end[:, ::5] = 0
    return begin, end, None


SHAPES = [
    # B, H, Hk, Nq, Nk, d
    (1, 1, 1, 1, 1, 64), (1, 4, 2, 1, 300, 128), (2, 8, 2, 5, 777, 64), (1, 6, 2, 33, 129, 128), (2, 3, 1, 128, 128, 64),
    (1, 4, 4, 129, 129, 128), (1, 2, 1, 257, 1000, 128), (2, 6, 2, 300, 300, 64), (1, 16, 2, 16, 4097, 128),
    (1, 5, 1, 200, 513, 64), (1, 2, 2, 1024, 1024, 128), (3, 3, 3, 64, 640, 64),
    (3, 3, 1, 1001, 1001, 64), (1, 4, 1, 1500, 1500, 128), (1, 1, 1, 700, 2600, 64),
]


@gpu
@pytest.mark.parametrize("kind", ["full", "causal", "window", "docs", "padded", "two ends"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, kind):
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape, seed=Nk)
    ranges = masks(kind, B, Nq, Nk)
    O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    ref = Ref(Q, K, V, ranges)
    ref.check(O, LSE)
    err = (O.double() + rest.double() - ref.O).abs()
    assert bool((err <= ref.two_terms).all()), float((err / ref.two_terms).max())
    plain = sk.attn_fwd(Q, K, V, ranges=ranges)
    ref.check(*plain)
    for got in (sk.attn_fwd(Q, K, V, ranges=ranges, rest=True), sk.attn_fwd(Q, K, V, ranges=ranges) + (None,)):
        want = (O, LSE, rest) if got[2] is not None else plain
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a row with one key alone has its value, bit for bit
    one = (ref.vis.sum(-1) == 1).expand_as(LSE)
    rows = torch.where(one[..., None], ref.O, 0.0)
    assert torch.equal(torch.where(one[..., None], plain[0].double(), 0.0), rows)


@gpu
@pytest.mark.parametrize("kind", ["full", "causal", "window", "docs", "padded", "two ends"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, kind):
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape, seed=Nk + 1)
    dO = torch.randn((B, H, Nq, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(BF16)
    ranges = masks(kind, B, Nq, Nk)
    O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    grads = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges)
    Ref(Q, K, V, ranges).check_grads(dO, *grads)
    again = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges)
    assert torch.equal(again[1], grads[1]) and torch.equal(again[2], grads[2])


@gpu
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64])
@pytest.mark.parametrize("shape", [(2, 8, 2, 1, 5000, 128), (1, 3, 3, 40, 1500, 64), (2, 4, 2, 130, 1100, 128), (1, 6, 2, 7, 1025, 64)], ids=str)
def test_forward_with_split_keys(shape, splits):
    Q, K, V = inputs(*shape)
    for kind in ("causal", "padded", "two ends"):
        ranges = masks(kind, shape[0], *shape[3:5])
        ref = Ref(Q, K, V, ranges)
        O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True, num_splits=splits)
        ref.check(O, LSE)
        assert bool(((O.double() + rest.double() - ref.O).abs() <= ref.two_terms).all())
        ref.check(*sk.attn_fwd(Q, K, V, ranges=ranges, num_splits=splits))


def dirty(t, hidden, value):
    """t with `value` in the rows of [B, h, N, d] that `hidden` [B, N] marks."""
    t = t.clone()
    t.masked_fill_(hidden[:, None, :, None], value)
    return t


@gpu
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("shape", [(2, 4, 2, 700, 700, 128), (2, 3, 3, 1100, 1100, 64), (2, 8, 2, 3, 900, 128)], ids=str)
def test_what_no_row_sees_has_no_effect(shape, value):
    """Keys and values behind a sequence, and queries and output gradients of rows that see nothing."""
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape)
    dO = torch.randn((B, H, Nq, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(BF16)
    n = torch.tensor([Nk - 133, Nk // 2 + 1], dtype=torch.int32, device=DEV)
    ranges = sk.key_ranges(B, Nq, Nk, DEV, q_lengths=n.clamp(max=Nq), k_lengths=n)
    want = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    grads = sk.attn_bwd(dO, Q, K, V, *want[:2], rest=want[2], ranges=ranges)
    keys = torch.arange(Nk, device=DEV) >= n[:, None]
    rows = torch.arange(Nq, device=DEV) >= n[:, None]
    Q2, K2, V2, dO2 = dirty(Q, rows, value), dirty(K, keys, value), dirty(V, keys, value), dirty(dO, rows, value)
    got = sk.attn_fwd(Q2, K2, V2, ranges=ranges, rest=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dirty_grads = sk.attn_bwd(dO2, Q2, K2, V2, *got[:2], rest=got[2], ranges=ranges)
    assert all(torch.equal(a, b) for a, b in zip(dirty_grads[1:], grads[1:]))
    Ref(Q, K, V, ranges).check_grads(dO, *dirty_grads)


@gpu
@pytest.mark.parametrize("which", ["K", "V", "Q", "dO"])
@pytest.mark.parametrize("shape", [(1, 4, 2, 600, 600, 128), (1, 3, 1, 900, 900, 64)], ids=str)
def test_a_broken_token_reaches_those_who_see_it_alone(shape, which):
    """Causal rows: a NaN at token 333 is in the outputs of that row or of the rows from it on, and in no other."""
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape)
    dO = torch.randn((B, H, Nq, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(BF16)
    want = sk.attn_fwd(Q, K, V, causal=True, rest=True)
    clean = sk.attn_bwd(dO, Q, K, V, *want[:2], rest=want[2], causal=True)
    at = 333
    t = dict(Q=Q.clone(), K=K.clone(), V=V.clone(), dO=dO.clone())
    t[which][:, :, at, 5] = math.nan
    O, LSE, rest = sk.attn_fwd(t["Q"], t["K"], t["V"], causal=True, rest=True)
    dQ, dK, dV = sk.attn_bwd(t["dO"], t["Q"], t["K"], t["V"], O, LSE, rest=rest, causal=True)
    row = torch.arange(Nq, device=DEV)
    hit = dict(K=row >= at, V=row >= at, Q=row == at, dO=row < 0)[which]
    assert torch.equal(O.isnan().any(-1), hit.expand(B, H, Nq))
    assert torch.equal(O[:, :, ~hit], want[0][:, :, ~hit]) and torch.equal(LSE[:, :, ~hit], want[1][:, :, ~hit])
    back = hit if which != "dO" else row == at
    assert torch.equal(dQ.isnan().any(-1), back.expand(B, H, Nq))
    bound = Ref(Q, K, V, causal=True)  # rows that do not see it have their gradient, up to the order of sums
    diff = (dQ[:, :, ~back].double() - clean[0][:, :, ~back].double()).abs()
    assert bool((diff <= 2.0 ** -7 * clean[0][:, :, ~back].double().abs() + 1e-6).all()) and bound.live.all()
    # keys that a hit row sees have a term of it; keys behind every hit row (Q, dO) have none
    seen = row <= at if which in ("Q", "dO") else row >= 0
    assert bool(dK[:, :, seen].isnan().any(-1).all())
    assert torch.equal(dK[:, :, ~seen], clean[1][:, :, ~seen]) and torch.equal(dV[:, :, ~seen], clean[2][:, :, ~seen])


@gpu
@pytest.mark.parametrize("splits", [1, 2, 5])
@pytest.mark.parametrize("shape", [(1, 8, 2, 300, 300, 128), (2, 3, 1, 129, 1000, 64), (1, 2, 2, 700, 260, 128)], ids=str)
def test_gradients_with_shared_key_tiles(shape, splits):
    B, H, Hk, Nq, Nk, d = shape
    Q, K, V = inputs(*shape)
    dO = torch.randn((B, H, Nq, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(BF16)
    for kind in ("full", "two ends") + (("causal",) if Nq <= Nk else ()):
        ranges = masks(kind, B, Nq, Nk)
        O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
        Ref(Q, K, V, ranges).check_grads(dO, *sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges, num_splits=splits))


@gpu
@pytest.mark.parametrize("peak", [0.3, 2.0])
@pytest.mark.parametrize("d", [64, 128])
def test_gradients_of_keys_and_values_with_a_common_offset(d, peak):
    """What a row's keys have in common cancels in dQ, and what its values have in common in D: neither the roundings of
    probabilities nor those of dS may show there.  The bound is the outputs' own rounding (2^-8 / sqrt 3 of the norm at
    most) and a third of it for everything else."""
    Q, K, V = inputs(1, 4, 2, 500, 500, d, peak=peak)
    K[..., : d // 8] += 16.0
    V += 4.0
    dO = torch.randn((1, 4, 500, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(BF16)
    O, LSE, rest = sk.attn_fwd(Q, K, V, causal=True, rest=True)
    got = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, causal=True)
    leaves = [t.double().requires_grad_() for t in (Q, K, V)]
    s = leaves[0] @ leaves[1].repeat_interleave(2, 1).transpose(2, 3) * d ** -0.5
    s = s.masked_fill(torch.ones(500, 500, device=DEV).triu(1).bool(), -math.inf)
    out = torch.softmax(s, -1) @ leaves[2].repeat_interleave(2, 1)
    want = torch.autograd.grad((out * dO.double()).sum(), leaves)
    for name, a, b in list(zip(("dQ", "dK"), got, want)):
        err = float((a.double() - b).norm() / b.norm())
        assert err <= 2.0 ** -8 / 3 ** 0.5 * 4 / 3, (name, err)
