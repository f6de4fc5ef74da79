"""Numbers that a call is given are read on every call, also from a tensor or an
array that a program changes in place between calls, and checked calls are known
by what the checks look at alone.

Without a device the library's calls are replaced by a recorder and the tensors
say that they are on one.
"""
import pytest
import torch

from attention_kl_divergence_gb300 import make_qk, streamkl as sk

BF16 = torch.bfloat16


class OnDevice(torch.Tensor):
    @property
    def is_cuda(self):
        return True


def fake(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def record(monkeypatch):
    calls = []
    monkeypatch.setattr(sk, "_on", lambda device, function, desc, *args: calls.append(desc) or sk.OK)
    monkeypatch.setattr(sk, "_known", {})
    return calls


def counters():
    numpy = pytest.importorskip("numpy")
    return {"tensor": torch.tensor(5), "array": numpy.array(5), "one_element": torch.tensor([5])}


@pytest.mark.parametrize("kind", ["tensor", "array", "one_element"])
def test_start_is_read_on_every_call(record, kind):
    q, k, table = fake(1, 4, 3, 64), fake(1, 2, 3, 64), fake(64, 32, 2, dtype=torch.float32)
    start = counters()[kind]
    for _ in range(3):
        sk.qk_norm_rope(q, k, table=table, start=start, out=(q, k))
        start += 1
    sk.qk_norm_rope(q, k, table=table, start=5, out=(q, k))
    assert [c.start for c in record] == [5, 6, 7, 5]


def test_eps_and_pairing_are_read_on_every_call(record):
    q, k = fake(1, 4, 3, 64), fake(1, 2, 3, 64)
    eps, neighbours = torch.tensor(0.5), torch.tensor(False)
    for _ in range(3):
        sk.qk_norm_rope(q, k, eps=eps, interleaved=neighbours, out=(q, k))
        eps *= 2
        neighbours.logical_not_()
    assert [c.eps for c in record] == [0.5, 1.0, 2.0]
    assert [c.interleaved for c in record] == [0, 1, 0]


def test_a_counter_of_positions_leaves_one_known_call(record):
    q, k = fake(1, 4, 1, 64), fake(1, 2, 1, 64)
    for n in range(600):
        sk.qk_norm_rope(q, k, start=n, out=(q, k))
    assert [c.start for c in record] == list(range(600))
    assert len(sk._known) == 1


def test_a_start_that_no_position_has_is_refused(record):
    q, k = fake(1, 4, 1, 64), fake(1, 2, 1, 64)
    for start in (2 ** 63, -2 ** 63 - 1, 2 ** 64 + 5):
        with pytest.raises(ValueError):
            sk.qk_norm_rope(q, k, start=start, out=(q, k))
    assert not record


@pytest.mark.gpu
def test_rotation_by_a_counter_on_the_device():
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, 4, 1, 64, generator=g, device="cuda").to(BF16)
    k = torch.randn(2, 2, 1, 64, generator=g, device="cuda").to(BF16)
    table = sk.rope_table(64, 64, "cuda")
    w = torch.ones(64, device="cuda")
    for at in (torch.tensor(5), torch.tensor(5, device="cuda")):
        for n in (5, 6, 7):
            want = sk.qk_norm_rope(q, k, w, w, table, start=n)
            got = sk.qk_norm_rope(q, k, w, w, table, start=at)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            want = sk.qk_norm_rope_bwd(q, k, q, k, w, w, table, start=n)
            got = sk.qk_norm_rope_bwd(q, k, q, k, w, w, table, start=at)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            at += 1


@pytest.mark.gpu
def test_split_counts_and_wait_limits_are_read_on_every_call():
    """The plan's workspace depends on the splits: a stale one would be too small."""
    qk = make_qk(1, 4, 40, 900, 64, 0.3, seed=2, device="cuda", H_kv=2)
    splits = torch.tensor(1)
    for n in (1, 2, 3):
        got = sk.kl_score_fwd(sk.Scores(), *qk, num_splits=splits)
        want = sk.kl_score_fwd(sk.Scores(), *qk, num_splits=n)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        splits += 1
    rows, g = sk.kl_score_fwd(sk.Scores(), *qk), torch.ones(1, 4, 40, device="cuda")
    setting = torch.tensor(1)
    for n in (1, 2):
        got = sk.kl_score_bwd(setting, sk.Scores(), g, *qk, *rows)
        want = sk.kl_score_bwd(n, sk.Scores(), g, *qk, *rows)
        assert torch.equal(got[1], want[1])
        setting += 1
    limit, stall = torch.tensor(10_000_000), torch.tensor(0)
    ws = sk.new_workspace(sk.score_fwd_plan(*qk[:2]).workspace_bytes, "cuda")
    for n in (0, 1, 0):
        stall.fill_(n)
        sk.kl_score_fwd(sk.Scores(), *qk, workspace=ws, wait_limit_ns=limit, debug_flags=stall)
        assert (sk.workspace_status(ws) != 0) == bool(n)


@pytest.mark.gpu
def test_the_gradients_options_are_those_of_the_forward():
    """The program moves its counter on between the forward and the backward."""
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(1, 4, 6, 64, generator=g, device="cuda").to(BF16)
    k = torch.randn(1, 2, 6, 64, generator=g, device="cuda").to(BF16)
    table, start, eps = sk.rope_table(64, 64, "cuda"), torch.tensor(5), torch.tensor(1e-3)
    leaves = [t.clone().requires_grad_() for t in (q, k)]
    y = sk.QKNormRope.apply(*leaves, None, None, table, None, start, eps)
    start += 7
    eps += 1
    got = torch.autograd.grad(y, leaves, (q, k))
    want = sk.qk_norm_rope_bwd(q, k, q, k, table=table, start=5, eps=float(torch.tensor(1e-3)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    qk = make_qk(1, 4, 40, 40, 64, 0.3, seed=2, device="cuda", H_kv=2)
    scale, causal, up = torch.tensor(0.5), torch.tensor(True), torch.ones(1, 4, 40, device="cuda")
    leaves = [t.clone().requires_grad_() for t in qk]
    KL = sk.ScoredAttentionKL.apply(*leaves, sk.Scores(), causal, scale)
    scale *= 3
    causal.logical_not_()
    (got,) = torch.autograd.grad(KL, leaves[3], up)
    rows = sk.kl_score_fwd(sk.Scores(), *qk, causal=True, scale=0.5)
    want = sk.kl_score_bwd(1, sk.Scores(), up, *qk, *rows, causal=True, scale=0.5, grad_dtype=BF16)[1]
    assert torch.equal(got, want)
