"""The norm with positions on several axes, the attention over prompts with its
gradients, the divergence of a student's attention from its teacher's, the 8-bit
cache and the attention over it, run together as training and serving use them.

Each stage is checked against float64 on the inputs that it really got.  An error
e in dq reaches dx as at most r max|w| |e| (2-norm of a row: the rotation keeps
norms, the projection of the norm's gradient shortens them), plus dx's rounding
of 2^-8.
"""
import math

import pytest
import torch

import test_cache8 as c8
from attention_kl_divergence_gb300 import streamkl as sk
from test_attn import Ref
from test_norm_rope import backward64
from test_rope_axes import turns_of
from test_score_pipeline_gpu import heads, projections

pytestmark = pytest.mark.gpu
BF16, DEV = torch.bfloat16, "cuda"
EPS = 1e-6


def clip(B, N, width, text, at=0):
    """Positions [3, B, N]: `text` tokens with one position on all axes, then a grid of time, rows and columns."""
    n = torch.arange(at, at + N, device=DEV)
    p = n - text
    grid = [text + p // (4 * width), text + p // width % 4, text + p % width]
    return torch.stack([torch.where(n < text, n, g) for g in grid])[:, None].expand(3, B, N).contiguous().int()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,lengths", [(128, 128, (260, 171)), (64, 32, (260, 1))])
def test_training_step(d, rot, lengths, interleaved):
    """One packed projection, normalised and turned, attended to, with a loss on the output and one on the divergence of
    the student's attention from the teacher's: every gradient from the one leaf."""
    B, N, H, Hk = 2, 260, 4, 2
    xt, xs, w = projections(B, N, H, Hk, d, seed=d + rot)
    table = sk.rope_table(N, rot, DEV)
    axes = sk.rope_axes([rot // 2 - 2 * (rot // 8)] + 2 * [rot // 8], spread=rot == 32)
    pos = clip(B, N, 9, 30)
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    ranges = sk.key_ranges(B, N, N, DEV, q_lengths=n, k_lengths=n)
    scores = sk.Scores(begin=ranges[0], end=ranges[1], offset=ranges[2])
    g = torch.rand(B, H, N, device=DEV) / N
    G = (torch.randn(B, H, N, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(6)) / N).to(BF16)

    leaf = xs.clone().requires_grad_()
    wq, wk = (t.clone().requires_grad_() for t in w[2:])
    Q, K = sk.QKNormRope.apply(*heads(leaf, H, Hk), wq, wk, table, pos, 0, EPS, interleaved, axes)
    V = leaf[:, :, H + Hk:].transpose(1, 2)
    O = sk.Attention.apply(Q, K, V, ranges)
    ref = Ref(Q.detach(), K.detach(), V.detach(), ranges)
    ref.check(O, torch.where(ref.live, ref.LSE, -math.inf).float())
    dx, dwq, dwk = torch.autograd.grad(O, (leaf, wq, wk), G, retain_graph=True)

    (dQ, dK, dV), (tQ, tK, tV) = ref.grads(G)
    err = (dx[:, :, H + Hk:].transpose(1, 2).double() - dV).abs()
    assert bool((err <= tV * 1.01 + 2.0 ** -8 * dV.abs() + 1e-30).all())
    cs = turns_of(table, pos, axes)
    q, k = heads(xs.double(), H, Hk)
    for x, u, tol, weight, got, dw in ((q, dQ, tQ, w[2], dx[:, :, :H].transpose(1, 2), dwq),
                                       (k, dK, tK, w[3], dx[:, :, H:H + Hk].transpose(1, 2), dwk)):
        tol = tol * 1.01 + 2.0 ** -8 * u.abs()  # dq and dk are bf16
        want, wdw, size, total = backward64(u, x, weight.double(), cs, rot, EPS, interleaved)
        r = torch.rsqrt(x.pow(2).mean(-1) + EPS)
        bound = r * float(weight.abs().max()) * tol.norm(dim=-1) + (2.0 ** -8 + 2.0 ** -16) * want.norm(dim=-1) + \
            2.0 ** -16 * size.norm(dim=-1) + 1e-30
        assert bool(((got.double() - want).norm(dim=-1) <= bound).all())
        unit = (x * r[..., None]).abs()
        spread = (tol.norm(dim=-1, keepdim=True) * unit).sum((0, 1, 2)) + 2.0 ** -15 * total
        assert bool(((dw.double() - wdw).abs() <= spread).all())
    for b in range(B):
        assert bool((dx[b, lengths[b]:] == 0).all())  # rows behind a sequence

    # the divergence of the same queries and keys adds its gradients
    with torch.no_grad():
        Q1, K1 = sk.qk_norm_rope(*heads(xt, H, Hk), w[0], w[1], table, pos, interleaved=interleaved, axes=axes)
    KL = sk.ScoredAttentionKL.apply(Q1, K1, Q, K, scores)
    (alone,) = torch.autograd.grad(KL, leaf, g, retain_graph=True)
    (both,) = torch.autograd.grad((O, KL), leaf, (G, g))
    assert torch.equal(both[:, :, H + Hk:], dx[:, :, H + Hk:])
    # dQ and dK are each rounded to bf16, so is their sum, and so is the norm's gradient of it: row by row
    rows = lambda t: t.double().norm(dim=-1)  # noqa: E731
    diff = rows(both.double() - dx.double() - alone.double())[:, :, :H + Hk]
    amp = max(float((w[2 + s].abs().max()) / w[2 + s].abs().min()) for s in (0, 1))
    size = torch.cat([rows(heads(t, H, Hk)[s]).transpose(1, 2) for t in (dx,) for s in (0, 1)], 2) + rows(alone)[:, :, :H + Hk]
    inner = torch.cat([(torch.rsqrt(x.pow(2).mean(-1) + EPS) * u.norm(dim=-1)).transpose(1, 2) for x, u in ((q, dQ), (k, dK))], 2)
    assert bool((diff <= 4 * 2.0 ** -8 * amp * (size + 2 * inner)).all())


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T,d,rot", [(16, 128, 64), (64, 64, 64)])
def test_serving(T, d, rot, captured):
    """Prompts of unequal length, padded: attention over them, into the cache; a second chunk, which sees the first through
    the cache; then tokens one by one, the step captured once and replayed."""
    B, N, H, Hk, M, steps = 3, 150, 8, 2, 320 // T, 4
    x, _, w = projections(B, N + 40 + steps, H, Hk, d, seed=T)
    table = sk.rope_table(N + 60, rot, DEV)
    axes = sk.rope_axes([rot // 2 - 2 * (rot // 8)] + 2 * [rot // 8])
    pages_of, pages = c8.tables(B, M, seed=3)
    cache = sk.Cache8.empty(pages, Hk, T, d, DEV)
    held = torch.zeros(B, dtype=torch.int32, device=DEV)
    first = torch.tensor([N, 97, 1], dtype=torch.int32, device=DEV)

    def turned(at, n):
        part = x[:, at:at + n]
        q, k = sk.qk_norm_rope(*heads(part, H, Hk), w[0], w[1], table, clip(B, n, 9, 30, at), axes=axes)
        return q, k, part[:, :, H + Hk:].transpose(1, 2)

    # the prompts
    Q, K, V = turned(0, N)
    ranges = sk.key_ranges(B, N, N, DEV, q_lengths=first, k_lengths=first)
    Ref(Q, K, V, ranges).check(*sk.attn_fwd(Q, K, V, ranges=ranges))
    sk.cache8_append(cache, pages_of, held, K, V, counts=first)
    held += first
    k, v = sk.cache8_read(cache, pages_of, held, tokens=N)
    live = (torch.arange(N, device=DEV) < first[:, None])[:, None, :, None]
    for got, new in ((k, K), (v, V)):
        assert bool((got.masked_select(~live) == 0).all())
        # e4m3 of a page's scale: half a step, 2^-4 of the value, or half of the smallest step, 2^-10 of the scale, which
        # is at most 2^-8 times twice the page's largest value (448 > 2^8)
        top = new.masked_fill(~live, 0).abs().amax((2, 3), keepdim=True).double()
        assert bool(((got.double() - new.double()).abs() <= (2.0 ** -4 * new.double().abs()).maximum(2.0 ** -17 * top))[live.expand_as(got)].all())
    # a second chunk of 40, 23 and 7 tokens sees the first through the cache
    more = torch.tensor([40, 23, 7], dtype=torch.int32, device=DEV)
    Q, K, V = turned(N, 40)
    sk.cache8_append(cache, pages_of, held, K, V, counts=more)
    held += more
    k, v = sk.cache8_read(cache, pages_of, held, tokens=190)
    ranges = sk.key_ranges(B, 40, 190, DEV, q_lengths=more, k_lengths=held)
    O, LSE = sk.attn_fwd(Q, k, v, ranges=ranges)
    Ref(Q, k, v, ranges).check(O, LSE)
    for b, c in enumerate((40, 23, 7)):  # its last rows, asked of the cache itself
        n = min(c, 16)
        one = c8.Ref(Q[b:b + 1, :, c - n:c], cache, pages_of[b:b + 1], held[b:b + 1])
        got = sk.attn_cache8(Q[b:b + 1, :, c - n:c], cache, pages_of[b:b + 1], held[b:b + 1])
        one.check(*got)
        # the one operator's definition is the other's: both are within their bounds of one another
        part = (*(r[b:b + 1, c - n:c].contiguous() for r in ranges[:2]), None)
        tol = one.tol + Ref(Q[b:b + 1, :, c - n:c], k[b:b + 1], v[b:b + 1], part).o_tol
        assert bool(((got[0].double() - O[b:b + 1, :, c - n:c].double()).abs() <= tol).all())
    # one token at a time
    token = x[:, :1].clone()
    where = torch.zeros(3, B, 1, dtype=torch.int32, device=DEV)

    def step():
        q, k = sk.qk_norm_rope(*heads(token, H, Hk), w[0], w[1], table, where, axes=axes)
        sk.cache8_append(cache, pages_of, held, k, token[:, :, H + Hk:].transpose(1, 2))
        held.add_(1)
        return q, *sk.attn_cache8(q, cache, pages_of, held)

    if captured:
        keep = [t.clone() for t in (*cache.tensors(), held)]
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            q, O, LSE = step()
        for t, s in zip((*cache.tensors(), held), keep):
            assert torch.equal(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t,
                               s.view(torch.uint8) if s.dtype == torch.float8_e4m3fn else s)  # nothing ran
    for s in range(steps):
        token.copy_(x[:, N + 40 + s:N + 41 + s])
        where.copy_(clip(B, 1, 9, 30, N + 40 + s))
        if captured:
            graph.replay()
        else:
            q, O, LSE = step()
        c8.Ref(q, cache, pages_of, held).check(O, LSE)
        k, v = sk.cache8_read(cache, pages_of, held)
        last = (held.long() - 1)[:, None, None, None].expand(B, Hk, 1, d)
        new = token[:, :, H + Hk:].transpose(1, 2).double()
        top = v.abs().amax((2, 3), keepdim=True).double()
        assert bool(((v.gather(2, last).double() - new).abs() <= (2.0 ** -4 * new.abs()).maximum(2.0 ** -17 * top)).all())
