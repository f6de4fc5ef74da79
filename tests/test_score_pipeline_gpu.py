"""The norm with rotation, the score-modified divergence and their gradients
run together, as a training step and as a serving step use them.

Each stage is checked against float64 on the inputs that it really got, so the
bounds are those of the stages, carried through: an error e in dq reaches dx as
at most r max|w| |e| (2-norm of a row: the rotation keeps norms, the projection
of the norm's gradient shortens them), plus dx's own rounding of 2^-8.
"""
import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk
from test_norm_rope import backward64, turns
from test_score import Ref

pytestmark = pytest.mark.gpu
BF16, DEV = torch.bfloat16, "cuda"


def projections(B, N, H, Hk, d, seed):
    """One packed projection [B, N, H + 2 Hk, d] of the teacher and one of the student, near each other."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((B, N, H + 2 * Hk, d), generator=g, device=DEV)
    y = x + 0.3 * torch.randn(x.shape, generator=g, device=DEV)
    w = [1.2 + 0.1 * torch.randn(d, generator=g, device=DEV) for _ in range(4)]
    return x.to(BF16), y.to(BF16), w


def heads(x, H, Hk):
    return x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32)])
def test_training_step(d, rot, interleaved):
    B, N, H, Hk = 2, 260, 4, 2
    xt, xs, w = projections(B, N, H, Hk, d, seed=d + rot)
    table = sk.rope_table(N + 5, rot, DEV)
    pos = (torch.arange(N, device=DEV) + torch.tensor([[0], [5]], device=DEV)).int()
    lengths = torch.tensor([N, 171], dtype=torch.int32, device=DEV)
    begin, end, offset = sk.key_ranges(B, N, N, DEV, q_lengths=lengths, k_lengths=lengths)
    sc = sk.Scores(50.0, 30.0, begin=begin, end=end, offset=offset)
    g = torch.rand(B, H, N, device=DEV) / N

    xs_leaf = xs.clone().requires_grad_()
    wq, wk = (t.clone().requires_grad_() for t in w[2:])
    with torch.no_grad():
        Q1, K1 = sk.qk_norm_rope(*heads(xt, H, Hk), w[0], w[1], table, pos, interleaved=interleaved)
    Q2, K2 = sk.QKNormRope.apply(*heads(xs_leaf, H, Hk), wq, wk, table, pos, 0, 1e-6, interleaved)
    KL = sk.ScoredAttentionKL.apply(Q1, K1, Q2, K2, sc)
    dx, dwq, dwk = torch.autograd.grad(KL, (xs_leaf, wq, wk), g)

    ref = Ref(Q1, K1, Q2.detach(), K2.detach(), begin, end, torch.arange(N, device=DEV).expand(B, N), None, 50.0, 30.0)
    assert bool(((KL.double() - ref.KL).abs() <= ref.delta_row * (4 + 4 * ref.spread_row)).all())
    (dQ, dK), (tQ, tK) = ref.grads(1, g, BF16)
    cs = turns(table, pos, B, N)
    q, k = heads(xs.double(), H, Hk)
    for x, u, tol, weight, got, dw in ((q, dQ, tQ, w[2], dx[:, :, :H].transpose(1, 2), dwq),
                                       (k, dK, tK, w[3], dx[:, :, H:H + Hk].transpose(1, 2), dwk)):
        tol = tol + 2.0 ** -8 * u.abs()  # dq and dk are bf16
        want, wdw, size, total = backward64(u, x, weight.double(), cs, rot, 1e-6, interleaved)
        r = torch.rsqrt(x.pow(2).mean(-1) + 1e-6)
        bound = r * float(weight.abs().max()) * tol.norm(dim=-1) + (2.0 ** -8 + 2.0 ** -16) * want.norm(dim=-1) + 2.0 ** -16 * size.norm(dim=-1)
        assert bool(((got.double() - want).norm(dim=-1) <= bound).all())
        n = (x * r[..., None]).abs()
        spread = (tol.norm(dim=-1, keepdim=True) * n).sum((0, 1, 2)) + 2.0 ** -15 * total  # a turned error is at most the row's
        assert bool(((dw.double() - wdw).abs() <= spread).all())
    assert bool((dx[:, :, H + Hk:] == 0).all())          # the values' part of the projection
    assert bool((dx[1, 171:] == 0).all())                # rows behind the second sequence


def test_float32_gradients_go_from_one_operator_to_the_other():
    B, N, H, Hk, d = 1, 150, 4, 2, 64
    xt, xs, w = projections(B, N, H, Hk, d, seed=1)
    table = sk.rope_table(N, d, DEV)
    q, k = heads(xs, H, Hk)
    Q1, K1 = sk.qk_norm_rope(*heads(xt, H, Hk), w[0], w[1], table)
    Q2, K2 = sk.qk_norm_rope(q, k, w[2], w[3], table)
    sc = sk.Scores(slopes1=torch.full((H,), 0.1, device=DEV), slopes2=torch.full((H,), 0.1, device=DEV))
    g = torch.rand(B, H, N, device=DEV)
    rows = sk.kl_score_fwd(sc, Q1, K1, Q2, K2, causal=True)
    dQ, dK = sk.kl_score_bwd(1, sc, g, Q1, K1, Q2, K2, *rows, causal=True)
    dq, dk, dwq, dwk = sk.qk_norm_rope_bwd(dQ, dK, q, k, w[2], w[3], table)
    cs = turns(table, None, B, N)
    for x, u, weight, got, dw in ((q, dQ, w[2], dq, dwq), (k, dK, w[3], dk, dwk)):
        want, wdw, size, total = backward64(u.double(), x.double(), weight.double(), cs, d, 1e-6, False)
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * size.amax(-1, keepdim=True)).all())
        assert bool(((dw.double() - wdw).abs() <= (B * H * N * 2.0 ** -24 + 2.0 ** -16) * total).all())


@pytest.mark.parametrize("window", [0, 40])
def test_serving_steps_agree_with_the_whole_sequence(window):
    """Tokens one by one: each one's keys go into its row of both models' caches, its queries against the caches; the
    divergences are those of the whole sequence at once."""
    B, N, H, Hk, d = 2, 150, 8, 2, 128
    xt, xs, w = projections(B, N, H, Hk, d, seed=7)
    table = sk.rope_table(N, d, DEV)
    Q1, K1 = sk.qk_norm_rope(*heads(xt, H, Hk), w[0], w[1], table)
    Q2, K2 = sk.qk_norm_rope(*heads(xs, H, Hk), w[2], w[3], table)
    begin, end, offset = sk.key_ranges(B, N, N, DEV, window=window)
    sc = sk.Scores(50.0, 50.0, begin=begin, end=end, offset=offset)
    whole = sk.kl_score_fwd(sc, Q1, K1, Q2, K2)
    ref = Ref(Q1, K1, Q2, K2, begin, end, torch.arange(N, device=DEV).expand(B, N), None, 50.0, 50.0)
    ref.check_rows(*whole)
    caches = [torch.full((B, 256, Hk, d), float("nan"), dtype=BF16, device=DEV).transpose(1, 2) for _ in range(2)]
    lengths = torch.zeros(B, dtype=torch.int32, device=DEV)
    steps = [(0, 100)] + [(n, n + 1) for n in range(100, 104)] + [(104, 120), (120, N)]
    got = [torch.empty_like(t) for t in whole]
    for lo, hi in steps:
        new = []
        for x, wq, wk, cache in ((xt, w[0], w[1], caches[0]), (xs, w[2], w[3], caches[1])):
            q, k = heads(x[:, lo:hi], H, Hk)
            out = (torch.empty((B, H, hi - lo, d), dtype=BF16, device=DEV), cache[:, :, lo:hi])
            new.append(sk.qk_norm_rope(q, k, wq, wk, table, start=lo, out=out)[0])
        lengths.fill_(hi)
        b, e, o = sk.key_ranges(B, hi - lo, 256, DEV, window=window, k_lengths=lengths)
        rows = sk.kl_score_fwd(sk.Scores(50.0, 50.0, begin=b, end=e, offset=o), new[0], caches[0], new[1], caches[1])
        for t, r in zip(got, rows):
            t[:, :, lo:hi] = r
    assert torch.equal(caches[0][:, :, :N], K1) and torch.equal(caches[1][:, :, :N], K2)
    ref.check_rows(*got)


def test_capture_beside_a_living_eager_graph_is_refused():
    x = torch.randn(1, 4, 32, 64, device=DEV).to(BF16).requires_grad_()
    k = torch.randn(1, 2, 32, 64, device=DEV).to(BF16)
    t = torch.randn(1, 4, 32, 64, device=DEV).to(BF16)
    sc = sk.Scores(20.0, 20.0)

    def step():
        q, kk = sk.QKNormRope.apply(x, k)
        return sk.ScoredAttentionKL.apply(t, k, q, kk, sc).sum()

    living = step()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="still alive"):
        with torch.cuda.graph(graph, stream=side):
            step().backward()
    torch.cuda.synchronize()
    living.backward()
    want, x.grad = x.grad, None
    del living
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step().backward()
    x.grad.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    # dQ's order of addition may differ between the two runs: one bf16 step of each value
    assert bool(((x.grad - want).abs().float() <= 2.0 ** -7 * want.abs().float() + 2.0 ** -9 * want.abs().max().float()).all())
