"""Norm of query and key heads with the position rotation, and its gradient,
against the definition in float64.

Tolerances.  An output y is rounded once to bf16: off by at most 2^-8 |y|.
Before that, float32 arithmetic: the mean square is a sum of d products (any
order: relative error at most d 2^-24 of a sum of positive terms, half of it in
r), rsqrt a few units, then four more roundings per product and two products per
turned value.  With d <= 128 that is below 80 * 2^-24 < 2^-17 relative to the
pair's size |a| + |b|.  dx adds a dot product of d terms: the same bound on
r (|w u| + |n| mean|w u n|).  dw sums T rows in float32: T 2^-24 of the sum of
magnitudes at most, on top of the relative 2^-17 of each term.
"""
import ctypes

import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk

gpu = pytest.mark.gpu
F64, BF16 = torch.float64, torch.bfloat16
STEP = 2.0 ** -8


def table64(rows, rot, base=10000.0):
    freq = torch.tensor([base ** (-2.0 * e / rot) for e in range(rot // 2)], dtype=F64)
    a = torch.arange(rows, dtype=F64)[:, None] * freq
    return torch.stack((a.cos(), a.sin()), -1)


def turn64(x, cs, rot, interleaved):
    c, s = cs[..., 0], cs[..., 1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rot:]), -1)


def forward64(x, w, cs, rot, eps, interleaved):
    """y for x [B, H, N, d] and cs [B, N, rot/2, 2], float64."""
    n = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    n = n if w is None else n * w
    return turn64(n, cs[:, None], rot, interleaved) if rot else n


def backward64(dy, x, w, cs, rot, eps, interleaved):
    """(dx, dw, bound of |dx| terms, sum of |u n|) by the formula."""
    u = turn64(dy, cs[:, None] * torch.tensor([1.0, -1.0], dtype=F64, device=x.device), rot, interleaved) if rot else dy
    r = torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    n = x * r
    wu = u if w is None else u * w
    dx = r * (wu - n * (wu * n).mean(-1, keepdim=True))
    size = r * (wu.abs() + n.abs() * (wu * n).abs().mean(-1, keepdim=True))
    return dx, (u * n).sum((0, 1, 2)), size, (u * n).abs().sum((0, 1, 2))


def pair_size(y, w, x, rot, eps, interleaved):
    """|a| + |b| of each output's pair before the turn."""
    n = (x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps)).abs()
    n = n if w is None else n * w.abs()
    if not rot:
        return n
    if interleaved:
        s = n[..., :rot].unflatten(-1, (rot // 2, 2)).sum(-1, keepdim=True).expand(*n.shape[:-1], rot // 2, 2).flatten(-2)
    else:
        s = n[..., :rot // 2] + n[..., rot // 2:rot]
        s = torch.cat((s, s), -1)
    return torch.cat((s, n[..., rot:]), -1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 8, 16])
def test_formula_of_the_gradient_against_autograd_and_differences(rot, interleaved):
    g = torch.Generator().manual_seed(rot + interleaved)
    x = torch.randn(2, 3, 4, 16, generator=g, dtype=F64, requires_grad=True)
    w = torch.randn(16, generator=g, dtype=F64, requires_grad=True)
    dy = torch.randn(2, 3, 4, 16, generator=g, dtype=F64)
    cs = table64(64, rot)[torch.randint(0, 64, (2, 4), generator=g)] if rot else None
    f = lambda x, w: (forward64(x, w, cs, rot, 1e-6, interleaved) * dy).sum()  # noqa: E731
    dx, dw, _, _ = backward64(dy, x.detach(), w.detach(), cs, rot, 1e-6, interleaved)
    ax, aw = torch.autograd.grad(f(x, w), (x, w))
    assert torch.allclose(dx, ax, rtol=1e-10, atol=1e-12) and torch.allclose(dw, aw, rtol=1e-10, atol=1e-12)
    with torch.no_grad():
        for i in range(0, 384, 41):
            h = torch.zeros(384, dtype=F64)
            h[i] = 1e-5
            d = (f(x + h.view_as(x), w) - f(x - h.view_as(x), w)) / 2e-5
            assert abs(d - dx.flatten()[i]) < 1e-7 * (1 + abs(d))


def case(B, Hq, Hk, N, d, rot, weights=torch.float32, positions=None, seed=0, grad=BF16, packed=False, rows=64, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if packed:
        x = (n(B, N, Hq + 2 * Hk, d) * scale).to(BF16)
        q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    else:
        q, k = (n(B, Hq, N, d) * scale).to(BF16), (n(B, Hk, N, d) * scale).to(BF16)
    wq, wk = (None, None) if weights is None else ((1 + 0.2 * n(d)).to(weights), (1 + 0.2 * n(d)).to(weights))
    table = table64(rows, rot).float().cuda() if rot else None
    pos = None if positions is None else torch.randint(0, rows, (B, N), generator=g, device="cuda").to(positions)
    return q, k, wq, wk, table, pos, n(B, Hq, N, d).to(grad), n(B, Hk, N, d).to(grad)


def turns(table, pos, B, N, start=0):
    if table is None:
        return None
    at = pos.long() if pos is not None else (start + torch.arange(N, device=table.device)).expand(B, N)
    return table.double()[at]


def check_fwd(got, x, w, cs, rot, eps, interleaved):
    x, w = x.double(), None if w is None else w.double()
    want = forward64(x, w, cs, rot, eps, interleaved)
    bound = STEP * want.abs() + 2.0 ** -17 * pair_size(want, w, x, rot, eps, interleaved) + 1e-30
    assert got.dtype == BF16 and bool(((got.double() - want).abs() <= bound).all())


def check_bwd(dx, dw, dy, x, w, cs, rot, eps, interleaved):
    T = x.shape[0] * x.shape[1] * x.shape[2]
    wdx, wdw, size, total = backward64(dy.double(), x.double(), None if w is None else w.double(), cs, rot, eps, interleaved)
    # the turned gradient carries its pair's rounding: the bound takes the row's largest term
    bound = STEP * wdx.abs() + 2.0 ** -17 * size.amax(-1, keepdim=True) * 2
    assert dx.dtype == BF16 and bool(((dx.double() - wdx).abs() <= bound).all())
    if w is not None:
        tol = (T * 2.0 ** -24 + 2.0 ** -17) * total * 2 + (STEP * wdw.abs() if w.dtype == BF16 else 0)
        assert dw.dtype == w.dtype and bool(((dw.double() - wdw).abs() <= tol).all())
    else:
        assert dw is None


SHAPES = [  # B, Hq, Hk, N, d, rot, interleaved
    (1, 1, 1, 1, 64, 64, False),
    (2, 3, 1, 7, 128, 128, False),
    (1, 12, 4, 33, 128, 64, True),
    (3, 8, 8, 9, 64, 8, False),
    (2, 17, 5, 65, 64, 64, True),
    (1, 32, 8, 300, 128, 128, False),
    (4, 32, 8, 1, 128, 128, True),
    (2, 4, 2, 5, 128, 120, False),
    (2, 4, 2, 5, 64, 56, True),
    (1, 9, 9, 13, 128, 0, False),
]


@gpu
@pytest.mark.parametrize("weights", [torch.float32, BF16, None])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, packed, weights):
    B, Hq, Hk, N, d, rot, il = shape
    q, k, wq, wk, table, pos, _, _ = case(B, Hq, Hk, N, d, rot, weights, torch.int32, packed=packed, seed=N + rot)
    yq, yk = sk.qk_norm_rope(q, k, wq, wk, table, pos, eps=1e-6, interleaved=il)
    cs = turns(table, pos, B, N)
    check_fwd(yq, q, wq, cs, rot, 1e-6, il)
    check_fwd(yk, k, wk, cs, rot, 1e-6, il)


@gpu
@pytest.mark.parametrize("grad", [BF16, torch.float32])
@pytest.mark.parametrize("weights", [torch.float32, BF16, None])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, weights, grad):
    B, Hq, Hk, N, d, rot, il = shape
    q, k, wq, wk, table, pos, gq, gk = case(B, Hq, Hk, N, d, rot, weights, torch.int64, packed=True, seed=N + d, grad=grad)
    gq = gq.transpose(1, 2).contiguous().transpose(1, 2)  # gradients in another order than the inputs'
    dq, dk, dwq, dwk = sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos, interleaved=il)
    cs = turns(table, pos, B, N)
    check_bwd(dq, dwq, gq, q, wq, cs, rot, 1e-6, il)
    check_bwd(dk, dwk, gk, k, wk, cs, rot, 1e-6, il)
    again = sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos, interleaved=il)
    for a, b in zip((dq, dk, dwq, dwk), again):  # every sum in a fixed order
        assert a is b is None or torch.equal(a, b)


@gpu
def test_backward_more_rows_than_one_wave_of_ctas():
    q, k, wq, wk, table, pos, gq, gk = case(1, 16, 2, 9001, 64, 64, positions=torch.int32, rows=9001, seed=4)
    dq, dk, dwq, dwk = sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos)
    cs = turns(table, pos, 1, 9001)
    check_bwd(dq, dwq, gq, q, wq, cs, 64, 1e-6, False)
    check_bwd(dk, dwk, gk, k, wk, cs, 64, 1e-6, False)
    # dw of many rows: float32 sums of blocks stay within a few 2^-24 of the magnitudes' root sum square
    _, want, _, total = backward64(gq.double(), q.double(), wq.double(), cs, 64, 1e-6, False)
    assert bool(((dwq.double() - want).abs() <= 2.0 ** -17 * total).all())


@gpu
def test_start_scale_eps_and_large_or_zero_rows():
    q, k, wq, wk, table, _, gq, gk = case(1, 2, 1, 40, 128, 128, seed=9)
    q[:, 0, 3] = 0.0          # a zero row: y = 0, dx = w u / sqrt(eps)
    q[:, 1, 5] *= 2.0 ** 50   # squares up to 2^110
    q[:, 1, 6] *= 2.0 ** -40  # far below eps
    yq, yk = sk.qk_norm_rope(q, k, wq, wk, table, start=20, eps=1e-5)
    cs = turns(table, None, 1, 40, 20)
    check_fwd(yq, q, wq, cs, 128, 1e-5, False)
    check_fwd(yk, k, wk, cs, 128, 1e-5, False)
    dq, dk, dwq, dwk = sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, start=20, eps=1e-5)
    check_bwd(dq, dwq, gq, q, wq, cs, 128, 1e-5, False)
    check_bwd(dk, dwk, gk, k, wk, cs, 128, 1e-5, False)


@gpu
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_positions_outside_the_table_give_nan_there_alone(kind):
    q, k, wq, wk, table, pos, gq, gk = case(2, 3, 1, 6, 128, 64, positions=kind, seed=2)
    pos[0, 1], pos[1, 4] = -1, 64
    if kind == torch.int64:
        pos[0, 3] = 2 ** 62
    bad = (pos < 0) | (pos >= 64)
    ok = torch.where(bad, 0, pos)
    for y, z in zip(sk.qk_norm_rope(q, k, wq, wk, table, pos), sk.qk_norm_rope(q, k, wq, wk, table, ok)):
        rows = bad[:, None, :, None].expand(*y.shape[:3], 1)
        assert bool(torch.isnan(y[..., :64]).eq(rows).all())
        assert torch.equal(y[..., 64:], z[..., 64:]) and torch.equal(torch.where(rows, z, y), z)
    dq, _, dwq, _ = sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos)
    assert bool(torch.isnan(dq).any(-1).eq(bad[:, None].expand(2, 3, 6)).all()) and bool(torch.isnan(dwq[:64]).all())


@gpu
def test_outputs_in_place_in_a_cache_and_of_broadcast_inputs():
    q, k, wq, wk, table, pos, gq, gk = case(2, 8, 2, 3, 128, 128, positions=torch.int32, seed=6)
    yq, yk = sk.qk_norm_rope(q, k, wq, wk, table, pos)
    cache = torch.full((2, 50, 2, 128), 7.0, dtype=BF16, device="cuda")
    buf = q.clone()
    sk.qk_norm_rope(buf, k, wq, wk, table, pos, out=(buf, cache[:, 21:24].transpose(1, 2)))
    assert torch.equal(buf, yq) and torch.equal(cache[:, 21:24].transpose(1, 2), yk)
    assert bool((cache[:, :21] == 7).all()) and bool((cache[:, 24:] == 7).all())
    one = k[:, :1].expand(2, 8, 3, 128)  # one head seen as eight
    a, _ = sk.qk_norm_rope(one, k, wk, wk, table, pos)
    assert torch.equal(a, yk[:, :1].expand(2, 8, 3, 128))
    dy = gq.clone()
    want = sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos)
    got = sk.qk_norm_rope_bwd(dy, gk, q, k, wq, wk, table, pos, out=(dy, torch.empty_like(k)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


@gpu
def test_no_tokens():
    q, k, wq, wk, table, pos, gq, gk = case(2, 4, 2, 0, 64, 64, positions=torch.int32)
    yq, yk = sk.qk_norm_rope(q, k, wq, wk, table, pos)
    assert yq.shape == q.shape and yk.shape == k.shape
    _, _, dwq, dwk = sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos)
    assert bool((dwq == 0).all()) and bool((dwk == 0).all())


@gpu
def test_offsets_beyond_32_bits():
    """Batch stride of 2^31 + 64 elements: the second item lies past 4 GiB."""
    B, Hq, Hk, N, d = 2, 2, 1, 4, 64
    step = 2 ** 31 + 64
    buf = torch.empty(step + 4 * Hq * N * d, dtype=BF16, device="cuda")
    q0, k0, wq, wk, table, pos, gq, gk = case(B, Hq, Hk, N, d, 64, positions=torch.int32)
    q = buf.as_strided((B, Hq, N, d), (step, N * d, d, 1))
    y = buf.as_strided((B, Hq, N, d), (step, N * d, d, 1), 2 * Hq * N * d)
    q.copy_(q0)
    want = sk.qk_norm_rope(q0, k0, wq, wk, table, pos)
    sk.qk_norm_rope(q, k0, wq, wk, table, pos, out=(y, torch.empty_like(k0)))
    assert torch.equal(y, want[0])
    a = sk.qk_norm_rope_bwd(gq, gk, q0, k0, wq, wk, table, pos)
    b = sk.qk_norm_rope_bwd(gq, gk, q, k0, wq, wk, table, pos, out=(y, torch.empty_like(k0)))
    assert torch.equal(a[0], b[0]) and torch.equal(y, a[0])


@gpu
def test_table_of_far_positions():
    """cos and sin of angles in float64: within a float32 rounding (2^-24 of values up to 1, and the
    frequencies' own rounding in float64) at every position up to 2^20."""
    t = sk.rope_table(2 ** 20 + 3, 128, "cuda")
    want = table64(2 ** 20 + 3, 128)
    assert t.shape == want.shape and float((t.cpu().double() - want).abs().max()) <= 2.0 ** -24 + 1e-9
    f = [0.5 ** e for e in range(4)]
    a = torch.arange(9, dtype=F64)[:, None] * torch.tensor(f, dtype=F64)
    assert float((sk.rope_table(9, 8, "cuda", inv_freq=f).cpu().double() - torch.stack((a.cos(), a.sin()), -1)).abs().max()) <= 2.0 ** -24


@gpu
def test_autograd_function():
    q, k, wq, wk, table, pos, gq, gk = case(2, 4, 2, 10, 128, 128, positions=torch.int32, packed=True, seed=3)
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, wq, wk)]
    yq, yk = sk.QKNormRope.apply(*leaves, table, pos)
    grads = torch.autograd.grad((yq, yk), leaves, (gq, gk))
    want = sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    # one output only, a broadcast upstream gradient, and an input that needs none
    x = q.detach().clone().requires_grad_()
    y, _ = sk.QKNormRope.apply(x, k, wq, wk, table, pos)
    (dx,) = torch.autograd.grad(y.float().sum(), x)
    ref, _, _, _ = backward64(torch.ones_like(q, dtype=F64), q.double(), wq.double(), turns(table, pos, 2, 10), 128, 1e-6, False)
    assert float((dx.double() - ref).abs().max()) <= STEP * float(ref.abs().max()) * 1.01


@gpu
def test_replays_from_a_graph_on_another_stream():
    q, k, wq, wk, table, pos, gq, gk = case(1, 8, 2, 50, 128, 128, positions=torch.int32, seed=5)
    want = sk.qk_norm_rope(q, k, wq, wk, table, pos) + sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = sk.qk_norm_rope(q, k, wq, wk, table, pos) + sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos)
    for _ in range(2):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_refusals():
    q, k, wq, wk, table, pos, gq, gk = case(2, 4, 2, 10, 128, 128, positions=torch.int32)
    ok = dict(q=q, k=k, wq=wq, wk=wk, table=table, positions=pos)

    def bad(**kw):
        with pytest.raises((ValueError, sk.StreamKLError)):
            sk.qk_norm_rope(**{**ok, **kw})

    bad(q=q.float())
    bad(q=q.cpu())
    bad(k=k[:1])
    bad(k=k[:, :, :9])
    bad(q=q[..., ::2])
    bad(q=q[..., :96], k=k[..., :96])
    bad(wq=wq[:64])
    bad(wq=wq.to(BF16))
    bad(wq=wq.half(), wk=wk.half())
    bad(wk=wk.cpu())
    bad(table=table.double())
    bad(table=table[:, :31])
    bad(table=torch.zeros(64, 128, 2, device="cuda"))
    bad(table=table[:0])
    bad(positions=pos.float())
    bad(positions=pos[:1])
    bad(eps=float("nan"))
    bad(eps=-1.0)
    bad(out=(q.float(), k))
    bad(out=(torch.empty_like(q)[:, :1].expand_as(q), torch.empty_like(k)))
    bad(out=(torch.empty(2, 4, 10, 129, dtype=BF16, device="cuda")[..., 1:], torch.empty_like(k)))  # rows off 16 bytes
    with pytest.raises(ValueError):
        sk.qk_norm_rope_bwd(gq, gk.float(), q, k, wq, wk, table, pos)
    with pytest.raises(ValueError):
        sk.qk_norm_rope_bwd(gq[:, :1], gk, q, k, wq, wk, table, pos)
    with pytest.raises(ValueError):
        sk.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, table, pos, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    for kw in (dict(rot=12), dict(rot=0), dict(rows=0), dict(rot=256)):
        with pytest.raises(ValueError):
            sk.rope_table(**{**dict(rows=8, rot=64, device="cuda"), **kw})


def _desc(**kw):
    d = sk.NormRope()
    v = dict(B=1, Hq=2, Hk=1, N=4, d=64, rot=64, interleaved=0, weight_bf16=0, grad_bf16=0, pos_int64=0, eps=1e-6,
             table_rows=8, start=0)
    v.update({a: b for a, b in kw.items() if a in v})
    for a, b in v.items():
        setattr(d, a, b)
    for name, heads in (("q", 2), ("k", 1), ("yq", 2), ("yk", 1), ("dq", 2), ("dk", 1)):
        setattr(d, name, sk.Strides(*kw.get(name, (heads * 4 * 64, 4 * 64, 64))))
    return d


def test_abi_rejects_bad_descriptions_and_pointers_without_a_device():
    lib, P = sk.load(), ctypes.c_void_p

    def fwd(desc, ptrs=(256,) * 8):
        return lib.streamkl_norm_rope_fwd(ctypes.byref(desc) if desc is not None else None, *[P(p) for p in ptrs], P(0))

    def bwd(desc, ptrs=(256,) * 12, ws=256, nbytes=1 << 20):
        return lib.streamkl_norm_rope_bwd(ctypes.byref(desc) if desc is not None else None, *[P(p) for p in ptrs], P(ws),
                                          nbytes, P(0))

    for call in (fwd, bwd):
        assert call(None) == sk.ERR_INVALID_ARG
        for kw in (dict(B=0), dict(Hq=0), dict(Hk=0), dict(N=-1), dict(rot=12), dict(rot=72), dict(rot=-8), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(table_rows=0), dict(interleaved=2), dict(weight_bf16=-1), dict(pos_int64=7),
                   dict(q=(512, 256, 60)), dict(k=(512, -256, 64))):
            assert call(_desc(**kw)) == sk.ERR_INVALID_ARG, kw
        assert call(_desc(d=96)) == sk.ERR_UNSUPPORTED
        assert call(_desc(B=1 << 14, N=1 << 14)) == sk.ERR_UNSUPPORTED
    assert fwd(_desc(yq=(512, 0, 64))) == sk.ERR_INVALID_ARG   # heads written over one another
    assert bwd(_desc(dq=(512, 256, 32))) == sk.ERR_INVALID_ARG
    for i in (0, 1, 4, 6, 7):  # q, k, table, yq, yk
        for v in (0, 264):
            assert fwd(_desc(), tuple(v if j == i else 256 for j in range(8))) == sk.ERR_INVALID_ARG
    assert fwd(_desc(pos_int64=1), (256, 256, 256, 256, 256, 260, 256, 256)) == sk.ERR_INVALID_ARG
    for i in (0, 1, 2, 3, 6, 8, 9):  # dyq, dyk, q, k, table, dq, dk
        assert bwd(_desc(), tuple(0 if j == i else 256 for j in range(12))) == sk.ERR_INVALID_ARG
    assert bwd(_desc(), (256,) * 4 + (0,) + (256,) * 7) == sk.ERR_INVALID_ARG  # dwq without wq
    assert bwd(_desc(), ws=0) == sk.ERR_WORKSPACE
    assert lib.streamkl_norm_rope_workspace_bytes(ctypes.byref(_desc(d=96))) == 0
    assert lib.streamkl_rope_table(P(0), 8, 32, P(256), P(0)) == sk.ERR_INVALID_ARG
    assert lib.streamkl_rope_table(P(256), 0, 32, P(256), P(0)) == sk.ERR_INVALID_ARG
    assert lib.streamkl_rope_table(P(256), 8, 65, P(256), P(0)) == sk.ERR_INVALID_ARG
