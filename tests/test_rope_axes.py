"""The norm of query and key heads with a rotation whose pairs follow positions
on several axes, and its gradient, against the definition in float64.  The
tolerances are those of one axis (derived in test_norm_rope.py): an axis only
says which row of the table turns a pair."""
import ctypes
import random

import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk
from test_norm_rope import BF16, F64, STEP, backward64, case, check_bwd, check_fwd, table64

gpu = pytest.mark.gpu


def turns_of(table, pos, axes):
    """[B, N, rot/2, 2]: pair e at the position on its axis."""
    pair = torch.arange(len(axes), device=table.device)
    at = pos.long()[torch.tensor(axes, device=table.device)].permute(1, 2, 0)
    return table.double()[at, pair]


def axes_for(kind, pairs, n):
    if kind == "sections":  # multiples of four pairs
        a = pairs // 4 // n * 4
        return sk.rope_axes([pairs - a * (n - 1)] + [a] * (n - 1))
    if kind == "odd sections":
        a = max(1, pairs // n - 1)
        return sk.rope_axes([pairs - a * (n - 1)] + [a] * (n - 1))
    if kind == "spread":
        return sk.rope_axes([pairs - pairs // n * (n - 1)] + [pairs // n] * (n - 1), spread=True)
    r = random.Random(pairs)
    return tuple(r.randrange(n) for _ in range(pairs))


CASES = [  # B, Hq, Hk, N, d, rot, axes of positions
    (1, 2, 1, 1, 64, 64, 3), (2, 4, 2, 37, 128, 128, 3), (3, 12, 4, 50, 64, 32, 2), (1, 9, 3, 130, 128, 64, 4), (2, 3, 3, 9, 128, 8, 1),
]


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["sections", "odd sections", "spread", "any"])
@pytest.mark.parametrize("shape", CASES, ids=str)
def test_forward_and_gradients(shape, kind, interleaved):
    B, Hq, Hk, N, d, rot, A = shape
    q, k, wq, wk, table, _, gq, gk = case(B, Hq, Hk, N, d, rot, seed=N, packed=N % 2 == 1)
    axes = axes_for(kind, rot // 2, A)
    for kind_of in (torch.int32, torch.int64):
        pos = torch.randint(0, 64, (A, B, N), generator=torch.Generator(device="cuda").manual_seed(N), device="cuda").to(kind_of)
        cs = turns_of(table, pos, axes)
        got = sk.qk_norm_rope(q, k, wq, wk, table, pos, interleaved=interleaved, axes=axes)
        for y, x, w in zip(got, (q, k), (wq, wk)):
            check_fwd(y, x, w, cs, rot, 1e-6, interleaved)
    for g in ((gq, gk), (gq.float(), gk.float())):
        dq, dk, dwq, dwk = sk.qk_norm_rope_bwd(*g, q, k, wq, wk, table, pos, interleaved=interleaved, axes=axes)
        check_bwd(dq, dwq, g[0], q, wq, cs, rot, 1e-6, interleaved)
        check_bwd(dk, dwk, g[1], k, wk, cs, rot, 1e-6, interleaved)


@gpu
def test_one_position_on_every_axis_is_the_rotation_without_axes():
    q, k, wq, wk, table, pos, gq, gk = case(2, 4, 2, 21, 128, 128, positions=torch.int32)
    same = pos.expand(3, 2, 21).contiguous()
    for axes in (sk.rope_axes((16, 24, 24)), sk.rope_axes((24, 20, 20), spread=True)):
        assert all(torch.equal(a, b) for a, b in zip(sk.qk_norm_rope(q, k, wq, wk, table, pos),
                                                     sk.qk_norm_rope(q, k, wq, wk, table, same, axes=axes)))
        assert all(torch.equal(a, b) for a, b in zip(sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos),
                                                     sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, same, axes=axes)))


@gpu
def test_positions_outside_the_table_give_nan_in_their_pairs_alone():
    q, k, wq, wk, table, _, _, _ = case(1, 2, 1, 5, 128, 128)
    pos = torch.zeros((3, 1, 5), dtype=torch.int64, device="cuda")
    pos[1, 0, 2], pos[2, 0, 3] = 64, -1
    for axes in (sk.rope_axes((16, 24, 24)), sk.rope_axes((22, 21, 21), spread=True)):
        y, _ = sk.qk_norm_rope(q, k, wq, wk, table, pos, axes=axes)
        of = torch.tensor(axes + axes, device="cuda")  # the axis of each value (halves)
        for n, axis in ((2, 1), (3, 2)):
            assert torch.equal(y[0, :, n].isnan(), (of == axis).expand(2, 128))
        assert not bool(y[0, :, [0, 1, 4]].isnan().any())


@gpu
def test_autograd_function_and_replay_of_a_graph():
    q, k, wq, wk, table, _, gq, gk = case(1, 4, 2, 33, 128, 128, packed=True)
    pos = torch.randint(0, 64, (3, 1, 33), device="cuda", dtype=torch.int32)
    axes = sk.rope_axes((16, 24, 24))
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, wq, wk)]
    y = sk.QKNormRope.apply(*leaves, table, pos, 0, 1e-6, False, axes)
    grads = torch.autograd.grad(y, leaves, (gq, gk))
    want = sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos, axes=axes)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    ref, _, _, _ = backward64(gq.double(), q.double(), wq.double(), turns_of(table, pos, axes), 128, 1e-6, False)
    assert bool(((grads[0].double() - ref).abs() <= STEP * ref.abs() + 2.0 ** -14 * ref.abs().max()).all())
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = sk.qk_norm_rope(q, k, wq, wk, table, pos, axes=axes)
    pos.copy_(torch.randint(0, 64, (3, 1, 33), device="cuda", dtype=torch.int32))  # read on every replay
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, sk.qk_norm_rope(q, k, wq, wk, table, pos, axes=axes)))


@gpu
def test_axes_given_as_a_list_are_read_on_every_call():
    q, k, wq, wk, table, _, _, _ = case(1, 2, 1, 5, 64, 16)
    pos = torch.randint(0, 64, (2, 1, 5), device="cuda")
    axes = [0] * 8
    first = sk.qk_norm_rope(q, k, wq, wk, table, pos, axes=axes)
    axes[3] = 1
    assert not torch.equal(first[0], sk.qk_norm_rope(q, k, wq, wk, table, pos, axes=axes)[0])
    assert torch.equal(first[0], sk.qk_norm_rope(q, k, wq, wk, table, pos, axes=torch.zeros(8, dtype=torch.int32))[0])


def test_sections():
    assert sk.rope_axes((2, 1, 3)) == (0, 0, 1, 2, 2, 2)
    assert sk.rope_axes((2, 1, 3), spread=True) == (0, 1, 2, 0, 2, 2)
    for bad in ((), (3, -1)):
        with pytest.raises(ValueError):
            sk.rope_axes(bad)


@gpu
def test_refusals():
    q, k, wq, wk, table, pos, _, _ = case(2, 4, 2, 10, 128, 128, positions=torch.int32)
    three = pos.expand(3, 2, 10).contiguous()
    axes = sk.rope_axes((16, 24, 24))

    def bad(positions=three, axes=axes, table=table):
        with pytest.raises((ValueError, sk.StreamKLError)):
            sk.qk_norm_rope(q, k, wq, wk, table, positions, axes=axes)

    bad(axes=axes[:-1])
    bad(axes=axes[:-1] + (3,))
    bad(axes=axes[:-1] + (-1,))
    bad(axes=None)  # [3, B, N] without axes
    bad(positions=pos)
    bad(positions=None)
    bad(positions=three[:, :1])
    bad(positions=three.float())
    bad(positions=three.transpose(1, 2))
    bad(positions=pos.expand(5, 2, 10).contiguous())
    bad(table=None)


def test_abi_rejects_bad_axes_without_a_device():
    from test_norm_rope import _desc

    P, lib = ctypes.c_void_p, sk.load()

    def fwd(axes, positions=256, **kw):
        return lib.streamkl_norm_rope_axes_fwd(ctypes.byref(_desc(**kw)), None if axes is None else ctypes.byref(axes),
                                               P(256), P(256), P(256), P(256), P(256), P(positions), P(256), P(256), P(0))

    def bwd(axes):
        return lib.streamkl_norm_rope_axes_bwd(ctypes.byref(_desc()), None if axes is None else ctypes.byref(axes),
                                               *[P(256)] * 12, P(256), 1 << 20, P(0))

    bad = sk.RopeAxes(3)
    bad.axis_of[1] = 3
    for call in (fwd, bwd):
        assert call(None) == sk.ERR_INVALID_ARG
        assert call(sk.RopeAxes(0)) == sk.ERR_INVALID_ARG
        assert call(sk.RopeAxes(5)) == sk.ERR_INVALID_ARG
        assert call(bad) == sk.ERR_INVALID_ARG
    assert fwd(sk.RopeAxes(3), positions=0) == sk.ERR_INVALID_ARG
    assert fwd(sk.RopeAxes(3), rot=0) == sk.ERR_INVALID_ARG
