"""Calls of the attention over whole prompts that its users make around the plain
one: views and strided tensors, outputs of their own, autograd, graphs, streams,
threads, waits that give up, large offsets, and what it refuses."""
import ctypes
import math
import threading

import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk
from test_attn import BF16, DEV, F64, Ref, inputs, masks

gpu = pytest.mark.gpu
STALL = dict(wait_limit_ns=20_000_000, debug_flags=sk.DEBUG_INJECT_STALL)
STALE = 7.0


def grad_like(Q, seed=5):
    return torch.randn(Q.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)).to(BF16)


def spread(t, how):
    """The values of t [B, h, N, d] in memory of another layout."""
    B, h, N, d = t.shape
    if how == "rows by token":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if how == "padded rows":
        big = torch.full((B, h, N, d + 8), math.nan, dtype=t.dtype, device=DEV)
        big[..., :d] = t
        return big[..., :d]
    if how == "heads first":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    assert how == "every second token"
    big = torch.full((B, h, 2 * N, d), math.nan, dtype=t.dtype, device=DEV)
    big[:, :, ::2] = t
    return big[:, :, ::2]


@gpu
@pytest.mark.parametrize("how", ["rows by token", "padded rows", "heads first", "every second token"])
@pytest.mark.parametrize("shape", [(2, 4, 2, 200, 333, 128), (2, 6, 2, 3, 700, 64), (1, 1, 1, 150, 150, 64)], ids=str)
def test_layouts_give_the_same_bits(shape, how):
    Q, K, V = inputs(*shape)
    dO = grad_like(Q)
    want = sk.attn_fwd(Q, K, V, causal=True, rest=True)
    grads = sk.attn_bwd(dO, Q, K, V, *want[:2], rest=want[2], causal=True)
    views = [spread(t, how) for t in (Q, K, V)]
    out = spread(torch.full_like(Q, STALE), how)
    guard = out._base.clone()
    O, LSE, rest = sk.attn_fwd(*views, causal=True, rest=True, out=out)
    assert O is out and all(torch.equal(a, b) for a, b in zip((O, LSE, rest), want))
    got = sk.attn_bwd(spread(dO, how), *views, O, LSE, rest=rest, causal=True)
    assert torch.equal(got[1], grads[1]) and torch.equal(got[2], grads[2])
    Ref(Q, K, V, causal=True).check_grads(dO, *got)
    if how in ("padded rows", "every second token"):  # what lies between the rows stays
        out.copy_(torch.full_like(Q, STALE))
        assert torch.equal(out._base.isnan(), guard.isnan()) and torch.equal(out._base[~guard.isnan()], guard[~guard.isnan()])
    own = tuple(torch.full_like(t, STALE) for t in grads)
    again = sk.attn_bwd(dO, Q, K, V, *want[:2], rest=want[2], causal=True, out=own)
    assert all(a is b for a, b in zip(again, own)) and torch.equal(own[1], grads[1]) and torch.equal(own[2], grads[2])


@gpu
@pytest.mark.parametrize("Nq,Nk", [(5, 300), (300, 5), (300, 300), (130, 400), (400, 130)])
@pytest.mark.parametrize("d", [64, 128])
def test_causal_and_offset(Nq, Nk, d):
    """Without ranges the last row sees every key; rows that stand before the first key see none."""
    Q, K, V = inputs(2, 4, 2, Nq, Nk, d)
    dO = grad_like(Q)
    off = torch.tensor([3, Nk + 7], dtype=torch.int32, device=DEV)
    for ranges in (None, (None, None, None), (None, None, off), (None, None, off - 200)):
        given = None if ranges is None or ranges[2] is None else ranges
        ref = Ref(Q, K, V, given, causal=True)
        O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, causal=True, rest=True)
        ref.check(O, LSE)
        ref.check_grads(dO, *sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges, causal=True))


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_ranges_beyond_the_keys_are_clamped(d):
    Q, K, V = inputs(1, 2, 1, 140, 200, d)
    begin = torch.randint(-500, 500, (1, 140), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).int()
    end = torch.randint(-500, 500, (1, 140), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)).int()
    begin[0, :4] = torch.tensor([-2 ** 31, 2 ** 31 - 1, -2 ** 31, 0], device=DEV)
    end[0, :4] = torch.tensor([2 ** 31 - 1, -2 ** 31, -2 ** 31, 2 ** 31 - 1], device=DEV)
    for ranges in ((begin, end, None), (begin, None, None), (None, end, None)):
        ref = Ref(Q, K, V, ranges)
        O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
        ref.check(O, LSE)
        ref.check_grads(grad_like(Q), *sk.attn_bwd(grad_like(Q), Q, K, V, O, LSE, rest=rest, ranges=ranges))


@gpu
@pytest.mark.parametrize("scale", [0.0, 1e-3, -0.3, 3.0])
def test_scales(scale):
    """As in every call of the library, what is not above 0 stands for 1 / sqrt d."""
    Q, K, V = inputs(1, 4, 2, 150, 260, 64)
    ref = Ref(Q, K, V, causal=True, scale=scale if scale > 0 else 64 ** -0.5)
    O, LSE, rest = sk.attn_fwd(Q, K, V, causal=True, scale=scale, rest=True)
    ref.check(O, LSE)
    ref.check_grads(grad_like(Q), *sk.attn_bwd(grad_like(Q), Q, K, V, O, LSE, rest=rest, causal=True, scale=scale))


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_directional_derivatives_are_the_differences(d):
    """<grad, U> of each input against the difference quotient of the definition, steps of 2^-12 along U of unit entries.
    Its own error is the third derivative's, 2^-24 / 6 of it: below 1e-5 of the sums of magnitudes here."""
    Q, K, V = inputs(1, 4, 2, 70, 90, d)
    dO = grad_like(Q)
    O, LSE, rest = sk.attn_fwd(Q, K, V, causal=True, rest=True)
    got = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, causal=True)
    ref = Ref(Q, K, V, causal=True)
    want, tol = ref.grads(dO)
    hide = ~ref.vis

    def loss(q, k, v):
        s = (q @ k.repeat_interleave(2, 1).transpose(2, 3) * d ** -0.5).masked_fill(hide, -math.inf)
        return float(((torch.softmax(s, -1) @ v.repeat_interleave(2, 1)) * dO.double()).sum())

    g = torch.Generator(device=DEV).manual_seed(9)
    for i in range(3):
        U = torch.randint(0, 2, got[i].shape, generator=g, device=DEV).double() * 2 - 1
        at = [t.double() for t in (Q, K, V)]
        h = 2.0 ** -12
        ends = [loss(*[x + (sign * h * U if j == i else 0) for j, x in enumerate(at)]) for sign in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * h)
        bound = float((tol[i] * 1.01 + (2.0 ** -8 + 1e-5) * want[i].abs()).sum())
        assert abs(float((got[i].double() * U).sum()) - slope) <= bound, i


@gpu
@pytest.mark.parametrize("shape", [(2, 4, 2, 150, 150, 128), (1, 3, 1, 2, 80, 64)], ids=str)
def test_autograd(shape):
    Q, K, V = inputs(*shape)
    ranges = masks("padded", shape[0], *shape[3:5])
    leaves = [t.clone().requires_grad_() for t in (Q, K, V)]
    O = sk.Attention.apply(*leaves, ranges, False, 0.1)
    want = sk.attn_fwd(Q, K, V, ranges=ranges, scale=0.1, rest=True)
    assert torch.equal(O, want[0])
    ref = Ref(Q, K, V, ranges, scale=0.1)
    # a gradient that is broadcast, one with d outside, one that starts at an odd address, one of another layout
    one = torch.ones((), dtype=BF16, device=DEV)
    odd = torch.zeros(Q.numel() + 1, dtype=BF16, device=DEV)
    odd[1:] = grad_like(Q).flatten()
    for dO in (one.expand(Q.shape), grad_like(Q)[..., :1].expand(Q.shape), grad_like(Q.transpose(2, 3)).transpose(2, 3),
               odd[1:].view(Q.shape), spread(grad_like(Q), "rows by token"), grad_like(Q)[:, :1].expand(Q.shape)):
        ref.check_grads(dO, *torch.autograd.grad(O, leaves, dO, retain_graph=True))
    O.sum().backward()
    ref.check_grads(one.expand(Q.shape), *[t.grad for t in leaves])
    # gradients of some inputs alone
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        some = [t.clone().requires_grad_(bool(n)) for t, n in zip((Q, K, V), need)]
        sk.Attention.apply(*some, ranges, False, 0.1).sum().backward()
        assert [t.grad is not None for t in some] == [bool(n) for n in need]


@gpu
def test_autograd_takes_the_heads_of_one_projection_and_one_leaf_three_times():
    """One packed leaf, whose views the three inputs are; and one tensor that is query, key and value at once."""
    B, N, H, Hk, d = 2, 131, 4, 2, 64
    x = torch.randn(B, N, H + 2 * Hk, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).to(BF16).requires_grad_()
    parts = [t.transpose(1, 2) for t in x.split((H, Hk, Hk), 2)]
    O = sk.Attention.apply(*parts, None, True)
    dO = grad_like(O)
    O.backward(dO)
    Ref(*[p.detach() for p in parts], causal=True).check_grads(dO, *[t.transpose(1, 2) for t in x.grad.split((H, Hk, Hk), 2)])
    y = torch.randn(1, 2, 90, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(4)).to(BF16).requires_grad_()
    O = sk.Attention.apply(y, y, y, None, True)
    O.backward(grad_like(O))
    want, tol = Ref(y.detach(), y.detach(), y.detach(), causal=True).grads(grad_like(O))
    # each of the three and their two sums are rounded to bf16: half a step of each
    bound = sum(t * 1.01 + 3 * 2.0 ** -8 * w.abs() for w, t in zip(want, tol))
    assert bool(((y.grad.double() - sum(want)).abs() <= bound).all())


@gpu
def test_a_changed_input_is_noticed_by_the_backward():
    Q, K, V = (t.requires_grad_() for t in inputs(1, 2, 1, 64, 64, 64))
    begin = torch.zeros(1, 64, dtype=torch.int32, device=DEV)
    for change in (lambda: K.detach().add_(1), lambda: begin.add_(1)):
        O = sk.Attention.apply(Q, K, V, (begin, None, None))
        change()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            O.sum().backward()


@gpu
@pytest.mark.parametrize("living", ["a warm-up's", "the default stream's"])
def test_a_training_step_is_captured_or_refused(living):
    leaves = [t.requires_grad_() for t in inputs(2, 4, 2, 200, 200, 64)]
    dO = grad_like(leaves[0])
    step = lambda: sk.Attention.apply(*leaves, None, True)  # noqa: E731
    ref = Ref(*[t.detach() for t in leaves], causal=True)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    if living == "the default stream's":
        held = step()
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="still alive"):
            with torch.cuda.graph(graph, stream=side):
                step().backward(dO)
        torch.cuda.synchronize()
        held.backward(dO)
        ref.check_grads(dO, *[t.grad for t in leaves])
        return
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        held = step()
        held.backward(dO, retain_graph=True)
    torch.cuda.synchronize()
    for t in leaves:
        t.grad = None
    with torch.cuda.graph(graph, stream=side):
        step().backward(dO)
    for _ in range(2):
        for t in leaves:
            t.grad.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        ref.check_grads(dO, *[t.grad for t in leaves])
    del held


@gpu
@pytest.mark.parametrize("shape", [(1, 8, 2, 1, 5000, 128), (2, 4, 2, 300, 300, 64)], ids=str)
def test_two_graphs_and_an_eager_call_do_not_share_memory(shape):
    """Each graph's inputs are changed in place between replays; replays of both on two streams, beside eager calls."""
    sets = [inputs(*shape, seed=s) for s in (1, 2)]
    want = [sk.attn_fwd(*t, causal=True) for t in sets]
    graphs, outs = [], []
    held = [[torch.zeros_like(x) for x in t] for t in sets]
    for h in held:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=torch.cuda.Stream()):
            outs.append(sk.attn_fwd(*h, causal=True))
    for h, t in zip(held, sets):
        for a, b in zip(h, t):
            a.copy_(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = sk.attn_fwd(*sets[0], causal=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, want[0]))
    for out, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))


@gpu
def test_calls_of_several_threads():
    sets = [inputs(2, 4, 2, n, n, 64, seed=n) for n in (1, 65, 200, 500)]
    want = [sk.attn_fwd(*t, causal=True, rest=True) for t in sets]
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = sk.attn_fwd(*sets[i], causal=True, rest=True)
                grads = sk.attn_bwd(sets[i][0], *sets[i], *got[:2], rest=got[2], causal=True)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])) or not all(bool(g.isfinite().all()) for g in grads):
                    bad.append(i)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@gpu
def test_offsets_beyond_32_bits():
    """Rows 2^24 elements apart, heads and batches further; the same bits as packed tensors."""
    Q, K, V = inputs(2, 2, 1, 150, 150, 64)
    far = torch.empty(2 ** 24 * 310, dtype=BF16, device=DEV)  # 10 GB
    place = lambda t, at: far.as_strided(t.shape, (2 ** 24 * 150 + 192, 2 ** 23, 2 ** 24, 1), at).copy_(t)  # noqa: E731
    q, k, v = place(Q, 0), place(K, 64), place(V, 128)
    out = far.as_strided(Q.shape, (2 ** 24 * 150 + 192, 2 ** 23, 2 ** 24, 1), 1024)
    want = sk.attn_fwd(Q, K, V, causal=True, rest=True)
    got = sk.attn_fwd(q, k, v, causal=True, rest=True, out=out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dO = grad_like(Q)
    grads = sk.attn_bwd(place(dO, 2048), q, k, v, *got[:2], rest=got[2], causal=True)
    clean = sk.attn_bwd(dO, Q, K, V, *want[:2], rest=want[2], causal=True)
    assert torch.equal(grads[1], clean[1]) and torch.equal(grads[2], clean[2])
    Ref(Q, K, V, causal=True).check_grads(dO, *grads)


@gpu
def test_more_output_elements_than_32_bits_count():
    """33 M rows of 64: the last rows and some in the middle against the definition."""
    B, H, N, d = 1, 33 * 64, 16384, 64
    Q = torch.empty(B, H, N, d, dtype=BF16, device=DEV)
    Q.view(-1, 64 * N * d).copy_(torch.randn(1, 64 * N * d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF16).expand(33, -1))
    K, V = (torch.randn(B, 1, 128, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(s)).to(BF16) for s in (2, 3))
    O, LSE = sk.attn_fwd(Q, K, V)
    for h in (0, 32 * 64, H - 1):
        Ref(Q[:, h:h + 1, -300:], K, V).check(O[:, h:h + 1, -300:], LSE[:, h:h + 1, -300:])
    first = O.view(33, -1)[0]
    assert all(torch.equal(o, first) for o in O.view(33, -1))


def stale_workspace(nbytes):
    ws = torch.full(((nbytes + 255) // 256 * 64,), STALE, dtype=torch.float32, device=DEV).view(torch.uint8)
    ws[:256] = 0
    return ws


def right_or_nan(got, want):
    lost = torch.isnan(got)
    assert bool((lost | (got == want)).all())
    return lost


# one tile; two tiles of a unit; few rows with one tile and many keys; parts of rows; several waves of units
@gpu
@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("shape", [(1, 1, 1, 9, 100, 64), (1, 4, 2, 300, 600, 128), (2, 8, 2, 1, 3000, 128), (1, 2, 2, 40, 1500, 64),
                                   (4, 64, 8, 300, 300, 64)], ids=str)
def test_a_forward_wait_that_gives_up_leaves_right_rows_and_nan(shape, splits):
    t = inputs(*shape)
    for rest in (False, True):
        want = sk.attn_fwd(*t, causal=True, num_splits=splits, rest=rest)
        ws = stale_workspace(sk.attn_fwd_plan(*t, num_splits=splits).workspace_bytes)
        out = torch.full_like(t[0], STALE)
        got = sk.attn_fwd(*t, causal=True, num_splits=splits, rest=rest, workspace=ws, out=out, **STALL)
        assert sk.workspace_status(ws) != 0
        lost = [right_or_nan(a, b) for a, b in zip(got, want)]
        assert bool(lost[0].any()) and torch.equal(lost[0].all(-1), lost[1]) and torch.equal(lost[0].any(-1), lost[1])
        alone = sk.attn_fwd(*t, causal=True, num_splits=splits, rest=rest, **STALL)  # without the caller's status word
        assert torch.equal(alone[1].isnan(), lost[1])
        again = sk.attn_fwd(*t, causal=True, num_splits=splits, rest=rest, workspace=ws, out=out)
        assert sk.workspace_status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(again, want))


@gpu
@pytest.mark.parametrize("shape,splits", [((1, 4, 2, 8, 600, 64), 1), ((1, 4, 2, 300, 600, 64), 1), ((1, 4, 2, 300, 600, 128), 3),
                                          ((1, 4, 2, 600, 600, 128), 2)], ids=str)
def test_a_backward_wait_that_gives_up_leaves_right_rows_and_nan(shape, splits):
    t = inputs(*shape)
    dO = grad_like(t[0])
    O, LSE, rest = sk.attn_fwd(*t, rest=True)
    want = sk.attn_bwd(dO, *t, O, LSE, rest=rest, num_splits=splits)
    ws = stale_workspace(sk.attn_bwd_plan(*t, num_splits=splits).workspace_bytes)
    out = tuple(torch.full_like(x, STALE) for x in want)
    sk.attn_bwd(dO, *t, O, LSE, rest=rest, num_splits=splits, workspace=ws, out=out, **STALL)
    assert sk.workspace_status(ws) != 0
    lost = [right_or_nan(a, b) for a, b in zip(out[1:], want[1:])]
    # the first CTA: one key tile of one key head, and rows of that head's queries
    assert bool(lost[0].any()) and torch.equal(lost[0], lost[1]) and int(lost[0][..., 0].sum()) <= 128
    rows = torch.isnan(out[0])
    assert bool(rows.any()) and bool(rows.eq(rows[..., :1]).all()) and int(rows.any(-1).any(-1).sum()) <= shape[1] // shape[2]
    near = (out[0].double() - want[0].double()).abs() <= 1e-5 * want[0].double().abs().max() + 2.0 ** -7 * want[0].double().abs()
    assert bool((rows | near).all())
    got = sk.attn_bwd(dO, *t, O, LSE, rest=rest, num_splits=splits, workspace=ws, out=out)
    assert sk.workspace_status(ws) == 0 and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    Ref(*t).check_grads(dO, *got)


@gpu
def test_refusals():
    Q, K, V = inputs(2, 4, 2, 10, 30, 64)
    dO = grad_like(Q)
    O, LSE, rest = sk.attn_fwd(Q, K, V, rest=True)
    b32 = torch.zeros(2, 10, dtype=torch.int32, device=DEV)

    def bad(call, *a, **kw):
        for _ in range(2):  # also when it was refused before
            with pytest.raises((ValueError, sk.StreamKLError)):
                call(*a, **kw)

    def all_calls(q=Q, k=K, v=V, **kw):
        bad(sk.attn_fwd, q, k, v, **kw)
        bad(sk.attn_bwd, dO, q, k, v, O, LSE, **kw)
        if "num_splits" not in kw:
            bad(sk.Attention.apply, q, k, v, kw.get("ranges"))

    for wrong in (Q.float(), Q.half(), Q.cpu(), Q[..., :32], Q[0], Q[:1], Q[:, :3], Q[:, :, :0], Q.transpose(2, 3), None,
                  Q[:, :, :1].expand_as(Q), Q[..., ::2], Q[:, :, :, 1:]):
        all_calls(q=wrong)
    for wrong in (K.float(), K.cpu(), K[..., :32], K[:1], K[:, :, :0], K[:, :, :20], K[:, :1], K.transpose(1, 2), K[:, :1].expand_as(K)):
        all_calls(k=wrong)
        all_calls(v=wrong)
    all_calls(k=K[:, :0], v=V[:, :0])
    odd = torch.zeros(K.numel() + 1, dtype=BF16, device=DEV)[1:].view(K.shape)
    all_calls(k=odd)
    for wrong in (b32, (b32, b32), (b32, b32, None, None), (b32.long(), None, None), (b32[:1], None, None), (b32.T.contiguous(), None, None),
                  (None, b32.float(), None), (None, None, b32), (b32.cpu(), None, None), (torch.zeros(2, 20, dtype=torch.int32, device=DEV)[:, ::2], None, None),
                  (None,), 3):
        all_calls(ranges=wrong)
    all_calls(num_splits=-1)
    bad(sk.attn_fwd, Q, K, V, out=O.float())
    bad(sk.attn_fwd, Q, K, V, out=O[:, :, :5])
    bad(sk.attn_fwd, Q, K, V, out=O[:, :, :1].expand_as(O))
    bad(sk.attn_fwd, Q, K, V, out=O.cpu())
    bad(sk.attn_bwd, dO.float(), Q, K, V, O, LSE)
    bad(sk.attn_bwd, dO[:, :, :5], Q, K, V, O, LSE)
    bad(sk.attn_bwd, dO, Q, K, V, O[:1], LSE)
    bad(sk.attn_bwd, dO, Q, K, V, O, LSE[:1])
    bad(sk.attn_bwd, dO, Q, K, V, O, LSE.double())
    bad(sk.attn_bwd, dO, Q, K, V, O, None)
    bad(sk.attn_bwd, dO, Q, K, V, O, LSE, rest=rest.float())
    bad(sk.attn_bwd, dO, Q, K, V, O, LSE, rest=rest[:1])
    bad(sk.attn_bwd, dO, Q, K, V, O, LSE, out=(Q, K))
    bad(sk.attn_bwd, dO, Q, K, V, O, LSE, out=(Q.float(), K, V))
    bad(sk.attn_bwd, dO, Q, K, V, O, LSE, out=(Q, K, V.transpose(0, 1)))
    small = torch.zeros(256, dtype=torch.uint8, device=DEV)
    bad(sk.attn_bwd, dO, Q, K, V, O, LSE, workspace=small)
    long = torch.zeros(2, 2, 3000, 64, dtype=BF16, device=DEV)
    bad(sk.attn_fwd, Q, long, long, num_splits=3, workspace=small)
    bad(sk.attn_fwd, Q, K, V, workspace=small.cpu())
    bad(sk.attn_fwd, Q, K, V, workspace=small[1:])
    bad(sk.attn_fwd, Q, K, V, debug_flags=1 << 20)
    sk.attn_fwd(Q, K, V, ranges=[b32, b32, None])  # a list will do


def test_abi_rejects_bad_descriptions_and_pointers_without_a_device():
    P, lib = ctypes.c_void_p, sk.load()

    def desc(**kw):
        s = dict(B=2, H=4, H_kv=2, Nq=8, Nk=8, d=64)
        s.update({k: v for k, v in kw.items() if k in s})
        out = sk.Attn(*s.values())
        for name, heads in (("q", 4), ("k", 2), ("v", 2), ("o", 4), ("d_o", 4)):
            setattr(out, name, kw.get(name, sk.Strides(heads * 512, 512, 64)))
        return out

    def fwd(d, ptrs=(256,) * 9, ws=256, nbytes=1 << 24, opts=None):
        return lib.streamkl_attn_fwd(None if d is None else ctypes.byref(d), *[P(p) for p in ptrs[:6]], ctypes.c_float(0.0), 0,
                                     *[P(p) for p in ptrs[6:]], P(ws), nbytes, opts, P(0))

    def bwd(d, ptrs=(256,) * 13, ws=256, nbytes=1 << 24, opts=None):
        return lib.streamkl_attn_bwd(None if d is None else ctypes.byref(d), *[P(p) for p in ptrs[:10]], ctypes.c_float(0.0), 0,
                                     *[P(p) for p in ptrs[10:]], P(ws), nbytes, opts, P(0))

    wrong = [(None, sk.ERR_INVALID_ARG), (desc(d=96), sk.ERR_UNSUPPORTED), (desc(H=3), sk.ERR_INVALID_ARG),
             (desc(H=1 << 24, H_kv=1 << 24), sk.ERR_UNSUPPORTED), (desc(Nq=2 ** 31 - 1), sk.ERR_UNSUPPORTED),
             (desc(Nk=2 ** 31 - 1), sk.ERR_UNSUPPORTED)]
    wrong += [(desc(**{n: v}), sk.ERR_INVALID_ARG) for n in ("B", "H", "H_kv", "Nq", "Nk") for v in (0, -1)]
    for name in ("q", "k", "v", "o"):
        for st in ((56, 512, 64), (2048, 512, 0), (2048, 516, 64), (-2048, 512, 64), (2048, 512, 1 << 39), (0, 512, 64), (2048, 0, 64)):
            wrong.append((desc(**{name: sk.Strides(*st)}), sk.ERR_INVALID_ARG))
    for call in (fwd, bwd):
        for d, code in wrong:
            assert call(d) == code
    assert bwd(desc(d_o=sk.Strides(2048, 512, 0))) == sk.ERR_INVALID_ARG
    plan = sk.Plan()
    for call in (lib.streamkl_attn_fwd_plan, lib.streamkl_attn_bwd_plan):
        assert call(ctypes.byref(desc()), None, None) == sk.ERR_INVALID_ARG
        for d, code in wrong:
            assert call(None if d is None else ctypes.byref(d), None, ctypes.byref(plan)) == code
    # Q, K, V, begin, end, offset, O, rest, LSE: what may be absent, what takes 4 bytes
    for call, count, absent, small in ((fwd, 9, (3, 4, 5, 7), (3, 4, 5, 8)), (bwd, 13, (5, 7, 8, 9), (6, 7, 8, 9))):
        for k in range(count):
            if k not in absent:
                assert call(desc(), tuple(0 if k == e else 256 for e in range(count))) == sk.ERR_INVALID_ARG, k
            assert call(desc(), tuple((258 if k in small else 264) if k == e else 256 for e in range(count))) == sk.ERR_INVALID_ARG, k
    for ws in (0, 8):
        assert bwd(desc(), ws=ws) == sk.ERR_WORKSPACE


def test_a_cpu_tensor_is_refused_without_a_device():
    t = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: sk.attn_fwd(t, t, t), lambda: sk.attn_bwd(t, t, t, t, t, t[..., 0].float()), lambda: sk.Attention.apply(t, t, t),
                 lambda: sk.attn_fwd_plan(t, t, t)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
