"""The attention's autograd function where no gradient follows: an evaluation of the module that training calls."""
import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk
from test_attn import DEV, Ref, inputs, masks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(2, 4, 2, 300, 300, 128), (1, 8, 2, 1, 3000, 64)], ids=str)
@pytest.mark.parametrize("kind", ["causal", "padded", None])
def test_without_gradients_it_is_the_forward_alone(shape, kind, monkeypatch):
    t = inputs(*shape)
    ranges = None if kind is None else masks(kind, shape[0], *shape[3:5])
    want = sk.attn_fwd(*t, ranges=ranges, scale=0.1)[0]
    trained = sk.attn_fwd(*t, ranges=ranges, scale=0.1, rest=True)[0]
    asked = []
    forward = sk.attn_fwd

    def watched(*a, rest=False, **kw):
        asked.append(rest)
        return forward(*a, rest=rest, **kw)

    monkeypatch.setattr(sk, "attn_fwd", watched)
    O = sk.Attention.apply(*t, ranges, False, 0.1)
    assert asked == [False] and torch.equal(O, want) and not O.requires_grad and O.grad_fn is None
    Ref(*t, ranges, scale=0.1).check(O, forward(*t, ranges=ranges, scale=0.1)[1])
    with torch.no_grad():  # what a module computes from its weights there requires no gradient
        assert torch.equal(sk.Attention.apply(*t, ranges, False, 0.1), want)
    for k in range(3):  # one input is enough
        leaves = [x.clone().requires_grad_(k == e) for e, x in enumerate(t)]
        asked.clear()
        O = sk.Attention.apply(*leaves, ranges, False, 0.1)
        assert asked == [True] and torch.equal(O, trained)
        O.sum().backward()
        assert leaves[k].grad is not None


def test_without_gradients_it_allocates_its_output_and_lse_alone():
    t = inputs(1, 8, 2, 4096, 4096, 128)
    sk.Attention.apply(*t, None, True)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    O = sk.Attention.apply(*t, None, True)
    lse = O.numel() // 128 * 4
    assert torch.cuda.max_memory_allocated() - before <= O.numel() * 2 + lse + (1 << 20)
