"""A rotation table of frequencies that are on the device is made without waiting
for it: the call can be captured, and follows new frequencies at every replay."""
import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk

pytestmark = pytest.mark.gpu


def test_device_frequencies_are_captured():
    freq = torch.tensor([0.5 ** e for e in range(16)], dtype=torch.float64, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        table = sk.rope_table(50, 32, "cuda", inv_freq=freq)
    for factor in (1.0, 0.25):
        freq.mul_(factor)
        table.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(table, sk.rope_table(50, 32, "cuda", inv_freq=freq.tolist()))
