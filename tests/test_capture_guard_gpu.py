"""Capturing a training step while an eager graph of the same leaves is alive.

The leaves' gradient accumulators run on the stream that they were made on.  A
capture can take in another stream that can be captured itself (a warm-up's), so
such a step is captured like any other; the default stream it cannot, and the
functions refuse that before it breaks the capture.
"""
import pytest
import torch

from attention_kl_divergence_gb300 import make_qk, streamkl as sk

pytestmark = pytest.mark.gpu
BF16, DEV = torch.bfloat16, "cuda"
N, D = 64, 64


def leaves_and_step(kind):
    qk = make_qk(1, 4, N, N, D, 0.3, seed=4, device=DEV, H_kv=2)
    q, k = (t.clone().requires_grad_() for t in qk[2:])
    if kind == "unmodified":
        return (q, k), lambda: sk.AttentionKL.apply(qk[0], qk[1], q, k, True).sum()
    if kind == "views":
        x = torch.cat((qk[2], qk[3]), 1).transpose(1, 2).contiguous().requires_grad_()  # one packed projection

        def step():
            q, k = sk.QKNormRope.apply(x[:, :, :4].transpose(1, 2), x[:, :, 4:].transpose(1, 2))
            return sk.ScoredAttentionKL.apply(qk[0], qk[1], q, k, sk.Scores(20.0, 20.0), True).sum()
        return (x,), step
    if kind == "norm":
        return (q, k), lambda: sum(y.float().pow(3).sum() for y in sk.QKNormRope.apply(q, k))
    return (q, k), lambda: sk.ScoredAttentionKL.apply(qk[0], qk[1], q, k, sk.Scores(20.0, 20.0), True).sum()


KINDS = ["unmodified", "scored", "norm", "views"]


@pytest.mark.parametrize("hooked", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_step_is_captured_after_a_warm_up_whose_last_loss_lives(kind, hooked):
    leaves, step = leaves_and_step(kind)
    calls = []
    if hooked:  # a hook keeps its leaf's accumulator alive
        for t in leaves:
            t.register_post_accumulate_grad_hook(lambda t: calls.append(t))
    warm, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        for _ in range(2):
            for t in leaves:
                t.grad = None
            loss = step()
            loss.backward(retain_graph=True)
    torch.cuda.current_stream().wait_stream(warm)
    want = [t.grad.clone() for t in leaves]
    torch.cuda.synchronize()
    for t in leaves:
        t.grad = None
    with torch.cuda.graph(graph, stream=other):
        step().backward()
    for _ in range(2):
        for t in leaves:
            t.grad.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        # dQ's order of addition may differ between two runs: a bf16 step of each value
        for t, w in zip(leaves, want):
            assert bool(((t.grad - w).abs().float() <= 2.0 ** -7 * w.abs().float() + 2.0 ** -9 * w.abs().max().float()).all())
    del loss
    assert not hooked or len(calls) == 3 * len(leaves)


@pytest.mark.parametrize("kind", KINDS)
def test_capture_is_refused_while_a_graph_made_on_the_default_stream_lives(kind):
    leaves, step = leaves_and_step(kind)
    living = step()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="still alive"):
        with torch.cuda.graph(graph, stream=side):
            step().backward()
    torch.cuda.synchronize()
    living.backward()
    assert all(bool(torch.isfinite(t.grad).all()) for t in leaves)
