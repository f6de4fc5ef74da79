"""The paged 8-bit cache, written, read back and attended to, against the
definitions in float64.

Writing and reading are exact statements: a stored value is the nearest e4m3
number (ties to even) to x 2^-e, and what is read is that number times 2^e,
which bf16 holds.  Tests compare bits.

Attention.  The stored values enter the products exactly, q as f16 after a
power of two (exact but for values 2^-25 below the row's largest, off by 2^-35
of it), so a score is off by  del = (d + 32) 2^-24 A + 2^-32 A' + 2^-20 (M + 1),
A the largest scale |q|.|k|, A' the largest scale max|q| sum|k|, M the largest
|S|.  LSE is off by at most del + N 2^-24 and its rounding.  A probability p is
off by a factor 1 +- 2 del and is rounded to f16: 2^-11 of it, or for small ones
2^-25 in units in which the row's largest p s_V is at least 2^7 / 2^2.  The
product accumulates in float32, O is rounded once:
(2^-11 + 4 del + (N + 128) 2^-24) sum p |v| + 2^-30 max(p s_V) sum |v / s_V| + 2^-8 |O|.
"""
import ctypes
import math

import pytest
import torch

from attention_kl_divergence_gb300 import streamkl as sk

gpu = pytest.mark.gpu
F64, F32, BF16, E4M3 = torch.float64, torch.float32, torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda"


def nearest(x):
    """The nearest e4m3 numbers to finite x (ties to even) as float64."""
    _, e = torch.frexp(x)
    step = torch.tensor(2.0, dtype=F64) ** (e.double() - 4).clamp_min(-9)  # on the CPU: exact powers
    return torch.round(x / step) * step


def power_for(top):
    """The smallest 2^e, e >= -100, with top <= 448 2^e."""
    e = -100
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append_reference(values, scales, table, lengths, new, counts, T):
    """Sequence by sequence on the CPU; values float64 [pages, Hk, T, d] (NaN for NaN), scales float64 [pages, Hk]."""
    pages, Hk = scales.shape
    for b in range(table.shape[0]):
        held = max(int(lengths[b]), 0)
        n = min(max(int(counts[b]), 0), new.shape[2])
        for m in range(held // T, table.shape[1]):
            lo, hi = max(held, m * T), min(held + n, (m + 1) * T)
            page = int(table[b, m])
            if lo >= hi or not 0 <= page < pages:
                continue
            for h in range(Hk):
                x = new[b, h, lo - held:hi - held].double()
                finite = x.abs() < math.inf
                want = power_for(float(x[finite].abs().max()) if bool(finite.any()) else 0.0)
                now = max(float(scales[page, h]), want) if lo > m * T else want
                old = values[page, h, :lo - m * T] * (float(scales[page, h]) / now)
                values[page, h, :lo - m * T] = torch.where(old.isnan(), old, nearest(torch.nan_to_num(old)))
                q = nearest(torch.where(finite, x, 0.0) / now)
                values[page, h, lo - m * T:hi - m * T] = torch.where(finite, q, math.nan)
                scales[page, h] = now


def pool(pages, Hk, T, d, seed=0):
    """A cache whose pages hold values of many sizes, as e4m3 bytes with power-of-two scales."""
    g = torch.Generator().manual_seed(seed)
    v = [(torch.randn(pages, Hk, T, d, generator=g) * 40).clamp(-448, 448).to(E4M3).to(DEV) for _ in range(2)]
    s = [(2.0 ** torch.randint(-9, 0, (pages, Hk), generator=g).double()).float().to(DEV) for _ in range(2)]
    return sk.Cache8(v[0], v[1], s[0], s[1])


def tables(B, M, seed=0):
    """Pages of a shuffled pool that has one page more than the sequences need."""
    order = torch.randperm(B * M + 1, generator=torch.Generator().manual_seed(seed))[:B * M]
    return order.reshape(B, M).int().to(DEV), B * M + 1


def same(got, want):
    got = got.double().cpu()
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


APPENDS = [  # B, Hk, T, d, M, lengths, N, counts
    (1, 1, 16, 64, 1, [0], 1, None), (3, 2, 16, 128, 5, [0, 15, 16], 1, None), (2, 4, 64, 128, 4, [63, 100], 130, [130, 7]),
    (3, 1, 128, 64, 3, [127, 0, 5], 200, [0, 200, 1]), (2, 3, 32, 128, 3, [80, 90], 40, [40, 3]), (1, 2, 64, 64, 9, [1], 513, [513]),
]


@gpu
@pytest.mark.parametrize("shape", APPENDS, ids=str)
def test_append_and_read(shape):
    B, Hk, T, d, M, lengths, N, counts = shape
    table, pages = tables(B, M)
    cache = pool(pages, Hk, T, d)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    g = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randn(B, N, 4 * Hk, d, generator=g, device=DEV) * 2.0 ** torch.randint(-6, 12, (B, N, 1, 1), generator=g, device=DEV)
    x = x.to(BF16)
    k, v = x[:, :, :Hk].transpose(1, 2), x[:, :, 3 * Hk:].transpose(1, 2)  # views of one projection
    ref = [t.double().cpu() for t in cache.tensors()]
    sk.cache8_append(cache, table, i32(lengths), k, v, None if counts is None else i32(counts))
    for values, scales, new in ((ref[0], ref[2], k), (ref[1], ref[3], v)):
        append_reference(values, scales, table.cpu(), lengths, new.cpu(), counts or [N] * B, T)
    for got, want in zip(cache.tensors(), ref):
        assert same(got, want)
    after = [min(n + c, M * T) for n, c in zip(lengths, counts or [N] * B)]
    K, V = sk.cache8_read(cache, table, i32(after))
    for got, values, scales in ((K, ref[0], ref[2]), (V, ref[1], ref[3])):
        want = (values * scales[..., None, None])[table.cpu().long()].transpose(1, 2).reshape(B, Hk, M * T, d).clone()
        for b in range(B):
            want[b, :, after[b]:] = 0
        assert same(got, want)
    out = [torch.full((B, M * T + 3, Hk, d), 7.0, dtype=BF16, device=DEV) for _ in range(2)]
    sk.cache8_read(cache, table, i32(after), tokens=M * T, out=[t[:, :M * T].transpose(1, 2) for t in out])
    assert same(out[0][:, :M * T].transpose(1, 2), K.double().cpu()) and bool((out[1][:, M * T:] == 7).all())
    short = sk.cache8_read(cache, table, i32(after), tokens=5)
    assert same(short[0], torch.nn.functional.pad(K.double().cpu(), (0, 0, 0, 8))[:, :, :5])


@gpu
def test_tokens_one_by_one_give_the_same_cache_as_all_at_once():
    """The scale is the same; values are, where they are not among the least ones (rounded twice)."""
    T, d, Hk = 32, 64, 2
    table, pages = tables(1, 2)
    one, all_ = sk.Cache8.empty(pages, Hk, T, d, DEV), sk.Cache8.empty(pages, Hk, T, d, DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = (torch.randn(1, Hk, 50, d, generator=g, device=DEV) * torch.arange(1, 51, device=DEV)[:, None]).to(BF16)
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    sk.cache8_append(all_, table, n, x, x)
    for i in range(50):
        sk.cache8_append(one, table, n, x[:, :, i:i + 1], x[:, :, i:i + 1])
        n += 1
    assert torch.equal(one.k_scale, all_.k_scale)
    a, b = sk.cache8_read(one, table, n)[0], sk.cache8_read(all_, table, n)[0]
    scale = all_.k_scale[table[0].long()].transpose(0, 1).repeat_interleave(T, 1)[None, ..., None]
    least = b.abs() < 2.0 ** -6 * scale
    assert torch.equal(a[~least], b[~least]) and bool(((a - b).abs() <= 2.0 ** -9 * scale).all())


@gpu
def test_nan_infinities_zeros_and_ends_of_the_range():
    T, d = 16, 64
    x = torch.zeros(6, 1, 2, d, dtype=BF16, device=DEV)
    x[0, 0, 0, 3], x[0, 0, 1, 5], x[0, 0, 1, 6] = math.nan, math.inf, 3.0
    x[1] = 0.0
    x[2, 0, 0, 0] = torch.finfo(BF16).max
    x[3, 0, 0, 0] = 1e-38
    x[4] = 448.0
    x[5, 0, 0], x[5, 0, 1] = 450.0, -math.inf
    cache = sk.Cache8.empty(6, 1, T, d, DEV)
    table = torch.arange(6, dtype=torch.int32, device=DEV)[:, None].contiguous()
    ref = [t.double().cpu() for t in cache.tensors()]
    zero = torch.zeros(6, dtype=torch.int32, device=DEV)
    sk.cache8_append(cache, table, zero, x, x)
    append_reference(ref[0], ref[2], table.cpu(), [0] * 6, x.cpu(), [2] * 6, T)
    assert same(cache.k, ref[0]) and same(cache.k_scale, ref[2]) and same(cache.v, ref[0])
    assert cache.k_scale.flatten().tolist()[4:] == [1.0, 2.0]


@gpu
def test_missing_pages_and_rows_behind_the_tokens_stay_as_they_are():
    T, d, Hk = 16, 64, 1
    cache = pool(4, Hk, T, d)
    before = [t.clone() for t in cache.tensors()]
    x = torch.ones(5, Hk, 40, d, dtype=BF16, device=DEV)
    # a page below and above the pool, no room left in the table, nothing to write, and one good token
    table = torch.tensor([[-1, 9], [4, 2 ** 30], [0, 1], [2, 3], [3, 0]], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([0, 3, 32, 20, -5], dtype=torch.int32, device=DEV)
    counts = torch.tensor([40, 40, 40, -3, 1], dtype=torch.int32, device=DEV)
    sk.cache8_append(cache, table, lengths, x, x, counts)
    bits = [t.view(torch.uint8) if t.dtype == E4M3 else t for t in cache.tensors()]
    was = [t.view(torch.uint8) if t.dtype == E4M3 else t for t in before]
    for k in range(2):
        assert torch.equal(bits[k][:3], was[k][:3]) and torch.equal(bits[k][3, :, 1:], was[k][3, :, 1:])
        assert bool((cache.tensors()[k][3, :, 0].float() == 256).all())
        assert torch.equal(bits[2 + k][:3], was[2 + k][:3]) and bits[2 + k][3].item() == 2.0 ** -8
    K, _ = sk.cache8_read(cache, table, torch.tensor([3, 0, 33, 1, 1], dtype=torch.int32, device=DEV), tokens=40)
    assert bool(K[0, :, :3].isnan().all()) and bool((K[0, :, 3:] == 0).all()) and bool((K[1] == 0).all())
    assert bool(K[2, :, 32:33].isnan().all()) and not bool(K[2, :, :32].isnan().any())


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Ref:
    def __init__(self, Q, cache, table, lengths, scale=None):
        B, H, Nq, d = Q.shape
        T, Hk = cache.k.shape[2], cache.k.shape[1]
        N = table.shape[1] * T
        scale = d ** -0.5 if scale is None else scale
        at = table.long().clamp(0, cache.k.shape[0] - 1)
        seq = lambda v, s: (v.double() * s)[at].transpose(1, 2).reshape(B, Hk, N, d).repeat_interleave(H // Hk, 1)  # noqa: E731
        ks, vs = cache.k_scale.double()[..., None, None], cache.v_scale.double()[..., None, None]
        j = torch.arange(N, device=DEV)
        self.vis = (j < (lengths.long()[:, None] - Nq + 1 + torch.arange(Nq, device=DEV))[..., None])[:, None]
        live_keys = (j < lengths.long()[:, None])[:, None, :, None]
        k, v = seq(cache.k, ks).masked_fill(~live_keys, 0.0), seq(cache.v, vs).masked_fill(~live_keys, 0.0)
        v8 = seq(cache.v, torch.ones_like(vs)).masked_fill(~live_keys, 0.0)
        sv = vs.expand(-1, -1, T, 1)[at].transpose(1, 2).reshape(B, Hk, N, 1).repeat_interleave(H // Hk, 1)
        sv = sv.masked_fill(~live_keys, 0.0)
        q = Q.double()
        s = (q @ k.transpose(2, 3) * scale).masked_fill(~self.vis, -math.inf)
        self.LSE = torch.logsumexp(s, -1)
        self.live = self.vis.any(-1).expand_as(self.LSE)
        p = torch.exp(s - torch.where(self.live, self.LSE, 0.0)[..., None]).masked_fill(~self.vis, 0.0)
        self.O = p @ v
        big = lambda t: float(t.masked_fill(~self.vis, 0.0).abs().max())  # noqa: E731
        A = big(q.abs() @ k.abs().transpose(2, 3)) * scale
        A2 = big(q.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[:, :, None]) * scale
        self.delta = (d + 32) * 2.0 ** -24 * A + 2.0 ** -32 * A2 + 2.0 ** -20 * (big(s) + 1)
        self.acc = (N + 128) * 2.0 ** -24
        self.tol = (2.0 ** -11 + 4 * self.delta + self.acc) * (p @ v.abs()) + 2.0 ** -8 * self.O.abs() + 1e-30 + \
            2.0 ** -30 * (p * sv.transpose(2, 3)).amax(-1, keepdim=True) * v8.abs().sum(2)[:, :, None]

    def check(self, O, LSE):
        assert torch.equal(LSE == -math.inf, ~self.live)
        err = (LSE.double() - self.LSE)[self.live].abs()
        tol = self.delta + self.acc + 2.0 ** -23 * self.LSE[self.live].abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        assert bool((O[~self.live] == 0).all())
        err = (O.double() - self.O).abs()
        assert bool((err <= self.tol).all()), float((err / self.tol).max())


ATTENTION = [  # B, H, Hk, Nq, T, d, M, lengths
    (1, 1, 1, 1, 16, 64, 1, [1]), (2, 8, 2, 1, 16, 128, 9, [144, 3]), (3, 6, 2, 5, 64, 64, 5, [300, 4, 0]),
    (1, 16, 2, 16, 128, 128, 3, [384]), (2, 4, 4, 2, 32, 128, 40, [1279, 17]), (4, 8, 1, 1, 64, 128, 70, [4480, 1, 4097, 2000]),
    (2, 24, 8, 7, 16, 64, 20, [319, 6]), (1, 2, 1, 1, 64, 128, 700, [44003]),
    (2, 8, 2, 9, 16, 128, 60, [900, 33]), (1, 24, 2, 16, 32, 64, 30, [960]), (1, 40, 1, 16, 64, 128, 21, [1300]), (40, 4, 2, 1, 16, 64, 70, list(range(0, 1120, 28))),
]


@gpu
@pytest.mark.parametrize("splits", [0, 1, 3, 40])
@pytest.mark.parametrize("shape", ATTENTION, ids=str)
def test_attention(shape, splits):
    B, H, Hk, Nq, T, d, M, lengths = shape
    table, pages = tables(B, M, seed=M)
    cache = pool(pages, Hk, T, d, seed=M)
    Q = torch.randn(B, Nq, H, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF16).transpose(1, 2)
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    O, LSE = sk.attn_cache8(Q, cache, table, n, scale=0.02, num_splits=splits)
    Ref(Q, cache, table, n, 0.02).check(O, LSE)
    again = sk.attn_cache8(Q, cache, table, n, scale=0.02, num_splits=splits)
    assert torch.equal(O, again[0]) and torch.equal(LSE, again[1])


@gpu
@pytest.mark.parametrize("size", [2.0 ** -20, 1.0, 2.0 ** 20])
def test_attention_with_scales_far_apart(size):
    B, H, Hk, Nq, T, d, M = 2, 4, 2, 2, 16, 64, 12
    table, pages = tables(B, M)
    cache = pool(pages, Hk, T, d)
    g = torch.Generator().manual_seed(3)
    cache.v_scale.copy_(size * 2.0 ** torch.randint(-30, 31, (pages, Hk), generator=g).double())
    cache.v_scale[::5] = 2.0 ** -100
    cache.v[::5] = 0
    cache.k_scale.copy_(0.004 * (1 + torch.rand(pages, Hk, generator=g)))  # no powers of two
    Q = torch.randn(B, H, Nq, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF16)
    Q[0] *= 2.0 ** 20  # rows of sizes that f16 does not hold
    n = torch.tensor([M * T, 100], dtype=torch.int32, device=DEV)
    scale = torch.tensor([1.0])
    for b, scale in ((0, 2.0 ** -22), (1, 0.25)):
        O, LSE = sk.attn_cache8(Q[b:b + 1], cache, table[b:b + 1], n[b:b + 1], scale=scale)
        Ref(Q[b:b + 1], cache, table[b:b + 1], n[b:b + 1], scale).check(O, LSE)


@gpu
def test_what_a_row_does_not_see_has_no_effect():
    B, H, Hk, Nq, T, d, M = 2, 4, 2, 3, 16, 128, 6
    table, pages = tables(B, M)
    cache = pool(pages, Hk, T, d)
    Q = torch.randn(B, H, Nq, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF16)
    n = torch.tensor([50, 20], dtype=torch.int32, device=DEV)
    want = sk.attn_cache8(Q, cache, table, n)
    for b in range(B):
        for m in range(M):
            dead = max(0, int(n[b]) - m * T)
            page = int(table[b, m])
            if dead < T:
                cache.k.view(torch.uint8)[page, :, dead:] = 0x7f  # NaN
                cache.v.view(torch.uint8)[page, :, dead:] = 0xff
            if dead == 0:
                cache.k_scale[page], cache.v_scale[page] = math.nan, math.inf
                table[b, m] = -7
    got = sk.attn_cache8(Q, cache, table, n)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the last token is NaN: the rows before it do not see it
    cache.v.view(torch.uint8)[int(table[1, 1]), :, 3] = 0x7f
    got = sk.attn_cache8(Q, cache, table, n)
    assert torch.equal(got[0][0], want[0][0]) and bool(got[0][1, :, 2].isnan().all())
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0][1, :, :2], want[0][1, :, :2])


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,Nq,T", [(1, 3, 16), (4, 16, 64), (5, 7, 16)])  # rows in one 8-row tile, in teams of 16-row tiles
def test_a_broken_new_token_reaches_the_rows_that_see_it_alone(group, Nq, T, d):
    """The token at distance `back` from the last: NaN in its key, in a byte of its value, or a page of its own that has a
    scale which is no number."""
    B, Hk, M = 2, 2, 8
    table, pages = tables(B, M)
    Q = torch.randn(B, group * Hk, Nq, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF16)
    rows = torch.arange(Nq, device=DEV)
    for length in (2 * T + 1, 3 * T, 5 * T - 2):
        n = torch.tensor([length, length - 1], dtype=torch.int32, device=DEV)
        for back in sorted({0, 1, Nq - 2, Nq - 1}):
            for which in ("key", "value", "scale"):
                cache = pool(pages, Hk, T, d)
                want = sk.attn_cache8(Q, cache, table, n)
                at = length - 1 - back
                page = int(table[0, at // T])
                if which == "scale":  # the whole page: every token of it
                    cache.v_scale[page] = math.inf
                    at = at // T * T
                else:
                    (cache.k if which == "key" else cache.v).view(torch.uint8)[page, 1, at % T, d - 3] = 0x7f
                O, LSE = sk.attn_cache8(Q, cache, table, n)
                hit = (length - Nq + rows >= at) & torch.ones(B, Hk, group, Nq, dtype=torch.bool, device=DEV)
                hit[1] = False
                if which != "scale":
                    hit[:, 0] = False
                hit = hit.view(B, Hk * group, Nq)
                assert torch.equal(O.isnan().any(-1), hit), (length, back, which)
                assert torch.equal(O[~hit], want[0][~hit])
                clean = ~hit if which == "key" else torch.ones_like(hit)
                assert torch.equal(LSE[clean], want[1][clean])


@gpu
def test_missing_pages_and_lengths_behind_the_table_give_nan():
    B, H, Hk, Nq, T, d, M = 5, 2, 1, 1, 16, 64, 3
    table, pages = tables(B, M)
    cache = pool(pages, Hk, T, d)
    Q = torch.randn(B, H, Nq, d, device=DEV).to(BF16)
    table[0, 1], table[1, 2], table[2, 2] = -1, pages, 2 ** 31 - 1
    n = torch.tensor([48, 40, 32, 49, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    for splits in (0, 1):
        O, LSE = sk.attn_cache8(Q, cache, table, n, num_splits=splits)
        nan = torch.tensor([True, True, False, True, True], device=DEV)
        assert torch.equal(O.isnan().all(-1).all(-1).all(-1), nan) and torch.equal(LSE.isnan().all(-1).all(-1), nan)
        assert not bool(O[2].isnan().any())


@gpu
def test_outputs_streams_graphs_and_in_place_changes():
    B, H, Hk, Nq, T, d, M = 2, 8, 2, 1, 32, 128, 8
    table, pages = tables(B, M)
    cache = pool(pages, Hk, T, d)
    Q, k, v = (torch.randn(B, h, 1, d, device=DEV).to(BF16) for h in (H, Hk, Hk))
    n = torch.tensor([100, 31], dtype=torch.int32, device=DEV)
    out = torch.zeros(B, 1, H, d, dtype=BF16, device=DEV)
    start = [t.clone() for t in cache.tensors()]

    def reset():
        for t, s in zip(cache.tensors(), start):
            t.copy_(s)
        n.copy_(torch.tensor([100, 31], dtype=torch.int32))

    def step():
        sk.cache8_append(cache, table, n, k, v)
        n.add_(1)
        return sk.attn_cache8(Q, cache, table, n, out=out.transpose(1, 2))

    want = []
    for _ in range(3):
        O, LSE = step()
        want.append((O.clone(), LSE.clone()))
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    reset()
    for k_ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[k_][0]) and torch.equal(got[1], want[k_][1])


@gpu
@pytest.mark.parametrize("splits", [0, 3])
def test_lengths_below_zero_are_zero(splits):
    B, H, Hk, Nq, T, d, M = 4, 4, 2, 5, 16, 64, 100
    table, pages = tables(B, M)
    cache = pool(pages, Hk, T, d)
    Q = torch.randn(B, H, Nq, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF16)
    n = torch.tensor([-2 ** 31, -1, 1000, 0], dtype=torch.int32, device=DEV)
    O, LSE = sk.attn_cache8(Q, cache, table, n, num_splits=splits)
    Ref(Q, cache, table, n.clamp(min=0)).check(O, LSE)
    assert all(bool((t[[0, 1, 3]] == 0).all()) for t in sk.cache8_read(cache, table, n))


@gpu
def test_pages_beyond_32_bits_of_bytes():
    """The last pages of a cache of 4.4 GB each for keys and values, and the same pages of a small one."""
    B, H, Hk, T, d, M = 2, 8, 2, 128, 128, 5
    far = 2 ** 32 // (Hk * T * d) + 700
    big = sk.Cache8(*(torch.empty(far, Hk, T, d, dtype=torch.uint8, device=DEV) for _ in range(2)),
                    *(torch.empty(far, Hk, device=DEV) for _ in range(2)))
    small = sk.Cache8.empty(B * M, Hk, T, d, DEV)
    for a, s in zip(big.tensors(), small.tensors()):
        a[-B * M:] = s.view(torch.uint8) if s.dtype == E4M3 else s
    table = torch.arange(B * M, dtype=torch.int32, device=DEV).flip(0).reshape(B, M).contiguous()
    held = torch.zeros(B, dtype=torch.int32, device=DEV)
    k, v = (torch.randn(B, Hk, 500, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(s)).to(BF16) for s in (1, 2))
    Q = torch.randn(B, H, 3, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).to(BF16)
    got = []
    for cache, at in ((big, table + (far - B * M)), (small, table)):
        n = held.clone()
        for part in ((0, 499), (499, 500)):
            sk.cache8_append(cache, at, n, k[:, :, slice(*part)], v[:, :, slice(*part)])
            n += part[1] - part[0]
        got.append((*sk.attn_cache8(Q, cache, at, n), *sk.cache8_read(cache, at, n)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    Ref(Q, small, table, n).check(*got[0][:2])


@gpu
@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("Nq", [1, 9])
def test_a_wait_that_gives_up_leaves_nan_and_a_status(Nq, splits):
    B, H, Hk, T, d, M = 2, 8, 2, 16, 128, 64
    table, pages = tables(B, M)
    cache = pool(pages, Hk, T, d)
    Q = torch.randn(B, H, Nq, d, device=DEV).to(BF16)
    n = torch.tensor([1000, 300], dtype=torch.int32, device=DEV)
    work = sk.new_workspace(sk.attn_cache8_plan(Q, cache, table, n, num_splits=splits).workspace_bytes, DEV)
    O, LSE = sk.attn_cache8(Q, cache, table, n, num_splits=splits, workspace=work, wait_limit_ns=10 ** 7, debug_flags=sk.DEBUG_INJECT_STALL)
    assert sk.workspace_status(work) != 0
    assert bool(O[0, :H // Hk].isnan().all()) and bool(LSE[0, :H // Hk].isnan().all())  # the first segment's rows
    want = sk.attn_cache8(Q, cache, table, n, num_splits=splits, workspace=work)
    assert sk.workspace_status(work) == 0 and not bool(want[0].isnan().any())
    good = ~O.isnan()
    assert torch.equal(O[good], want[0][good])


@gpu
def test_refusals():
    table, pages = tables(2, 3)
    cache = pool(pages, 2, 16, 64)
    Q, k = torch.zeros(2, 4, 1, 64, dtype=BF16, device=DEV), torch.zeros(2, 2, 5, 64, dtype=BF16, device=DEV)
    n = torch.zeros(2, dtype=torch.int32, device=DEV)

    def bad(call, *a, **kw):
        with pytest.raises((ValueError, sk.StreamKLError)):
            call(*a, **kw)

    for call, args in ((sk.cache8_append, (k, k)), (sk.cache8_read, ())):
        bad(call, (cache.k, cache.v), table, n, *args)
        bad(call, cache, table.long(), n, *args)
        bad(call, cache, table[:1], n, *args)
        bad(call, cache, table, n.cpu(), *args)
        bad(call, cache, table, n.float(), *args)
        for k_, t in enumerate(cache.tensors()):
            for wrong in (t.float() if k_ < 2 else t.half(), t[:2], t.cpu(), t.transpose(0, 1)):
                other = list(cache.tensors())
                other[k_] = wrong
                bad(call, sk.Cache8(*other), table, n, *args)
    bad(sk.cache8_append, cache, table, n, k.float(), k)
    bad(sk.cache8_append, cache, table, n, k, k[:, :, :4])
    bad(sk.cache8_append, cache, table, n, k[:, :1], k[:, :1])
    bad(sk.cache8_append, cache, table, n, k[..., :32], k[..., :32])
    bad(sk.cache8_append, cache, table, n, k, k, counts=n[:1])
    bad(sk.cache8_append, cache, table, n, k, k, counts=n.long())
    bad(sk.cache8_append, sk.Cache8.empty(4, 2, 24, 64, DEV), table, n, k, k)
    bad(sk.cache8_append, sk.Cache8.empty(4, 2, 16, 96, DEV), table, n, k, k)
    bad(sk.cache8_read, cache, table, n, tokens=-1)
    bad(sk.cache8_read, cache, table, n, tokens=5, out=(k, k[:, :, :4]))
    bad(sk.cache8_read, cache, table, n, tokens=5, out=(k, k[:, :1].expand_as(k)))
    bad(sk.attn_cache8, Q.float(), cache, table, n)
    bad(sk.attn_cache8, Q[:1], cache, table, n)
    bad(sk.attn_cache8, Q[:, :3], cache, table, n)
    bad(sk.attn_cache8, Q[..., :32], cache, table, n)
    bad(sk.attn_cache8, torch.zeros(2, 4, 17, 64, dtype=BF16, device=DEV), cache, table, n)
    bad(sk.attn_cache8, Q[:, :, :0], cache, table, n)
    bad(sk.attn_cache8, Q, cache, table, n, out=Q.float())
    bad(sk.attn_cache8, Q, cache, table, n, num_splits=-1)
    assert sk.attn_cache8_plan(Q, cache, table, n, num_splits=2).workspace_bytes > 256
    bad(sk.attn_cache8, Q, cache, table, n, num_splits=2, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
    sk.cache8_append(cache, table, n, k[:, :, :0], k[:, :, :0])  # no tokens is allowed
    assert sk.cache8_read(cache, table, n, tokens=0)[0].shape == (2, 2, 0, 64)


def test_abi_rejects_bad_descriptions_and_pointers_without_a_device():
    P, lib = ctypes.c_void_p, sk.load()

    def desc(**kw):
        s = dict(pages=4, H_kv=2, T=16, d=64, B=2, M=2, H=4, N=1)
        s.update({k: v for k, v in kw.items() if k not in ("x", "y")})
        out = sk.CacheDesc(*[s[k] for k in ("pages", "H_kv", "T", "d", "B", "M", "H", "N")])
        out.x = kw.get("x", sk.Strides(256, 64, 64))
        out.y = kw.get("y", sk.Strides(256, 64, 64))
        return out

    def append(d, ptrs=(256,) * 9):
        return lib.streamkl_cache8_append(None if d is None else ctypes.byref(d), *[P(p) for p in ptrs], P(0))

    def read(d, ptrs=(256,) * 8):
        return lib.streamkl_cache8_read(None if d is None else ctypes.byref(d), *[P(p) for p in ptrs], P(0))

    def attn(d, ptrs=(256,) * 9, ws=256, nbytes=1 << 20):
        return lib.streamkl_attn_cache8(None if d is None else ctypes.byref(d), *[P(p) for p in ptrs[:7]], ctypes.c_float(0.0),
                                        *[P(p) for p in ptrs[7:]], P(ws), nbytes, None, P(0))

    wrong = [(None, sk.ERR_INVALID_ARG), (desc(pages=0), sk.ERR_INVALID_ARG), (desc(H_kv=0), sk.ERR_INVALID_ARG),
             (desc(B=0), sk.ERR_INVALID_ARG), (desc(M=0), sk.ERR_INVALID_ARG), (desc(T=48), sk.ERR_UNSUPPORTED),
             (desc(d=96), sk.ERR_UNSUPPORTED), (desc(M=1 << 27), sk.ERR_UNSUPPORTED)]
    strided = [(desc(N=-1), sk.ERR_INVALID_ARG), (desc(x=sk.Strides(60, 64, 64)), sk.ERR_INVALID_ARG),
               (desc(y=sk.Strides(-64, 64, 64)), sk.ERR_INVALID_ARG)]
    for call in (append, read):
        for d, code in wrong + strided:
            assert call(d) == code
    for d, code in wrong + [(desc(H=3), sk.ERR_INVALID_ARG), (desc(N=0), sk.ERR_INVALID_ARG), (desc(N=17), sk.ERR_UNSUPPORTED)] + strided[1:]:
        assert attn(d) == code
    assert read(desc(x=sk.Strides(0, 64, 64))) == sk.ERR_INVALID_ARG  # outputs must not overlap
    for call, count, small in ((append, 9, (2, 3, 4, 5, 8)), (read, 8, (2, 3, 4, 5))):
        for k in range(count):
            if not (call is append and k == 8):  # counts may be absent
                assert call(desc(), tuple(0 if k == e else 256 for e in range(count))) == sk.ERR_INVALID_ARG
            assert call(desc(), tuple((258 if k in small else 264) if k == e else 256 for e in range(count))) == sk.ERR_INVALID_ARG
    for k in range(9):
        assert attn(desc(), tuple(0 if k == e else 256 for e in range(9))) == sk.ERR_INVALID_ARG
