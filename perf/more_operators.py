"""Timed cases of the operators that make and serve an attention's output.

``attn``: attention over whole prompts with a key range for each query row
(causal, packed documents, padded batches, windows) and keys shared by groups
of query heads: forward, training step, and few rows against a long cache.

``append``: new tokens written into a paged cache of 8-bit values with one
power-of-two scale for each page and head, and the cache read back.

``cache``: attention of a few new tokens over that cache.

``rope``: the norm of query and key heads with a rotation whose pairs follow
the positions on several axes (time, height, width), and its gradient.

The plain forms are elementary torch operations in 32 bits, rounded once at the
end; ``exact`` restates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
E4M3_MAX, LEAST_EXPONENT = 448.0, -100


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def attn_case(name, form, B, H, Hk, Nq, Nk, d, mask, layout=0, peak=1.0):
    """form: fwd or train (forward and the gradients of queries, keys and values)."""
    return dict(name=name, op="attn", form=form, B=B, H=H, Hk=Hk, Nq=Nq, Nk=Nk, d=d, mask=mask, layout=layout, peak=peak)


def append_case(name, B, Hk, d, page, held, new, layout=0):
    """Up to `new` tokens for each sequence, behind up to `held` tokens that are there."""
    return dict(name=name, op="append", B=B, Hk=Hk, d=d, page=page, held=held, new=new, layout=layout)


def cache_case(name, B, H, Hk, Nq, Nk, d, page, layout=0):
    """Nq new tokens of each sequence, the last of up to Nk tokens in the cache."""
    return dict(name=name, op="cache", B=B, H=H, Hk=Hk, Nq=Nq, Nk=Nk, d=d, page=page, layout=layout)


def rope_case(name, form, B, H, Hk, frames, height, width, d, sections, spread, pairs, grad="bf16"):
    """Tokens of `frames` pictures of height x width patches; sections: pairs for time, height and width."""
    return dict(name=name, op="rope", form=form, B=B, H=H, Hk=Hk, frames=frames, height=height, width=width, d=d,
                s0=sections[0], s1=sections[1], s2=sections[2], spread=spread, pairs=pairs, grad=grad)


def listed():
    return [
        # a unit-sized prompt: what one call costs in latency
        attn_case("attn_fwd_tiny", "fwd", 1, 4, 2, 128, 128, 64, "causal"),
        # documents of uneven lengths packed in one 8K sequence, evaluated
        attn_case("attn_fwd_docs_8k", "fwd", 1, 32, 8, 8192, 8192, 128, "docs", layout=1),
        # one long prompt
        attn_case("attn_fwd_32k", "fwd", 1, 8, 2, 32768, 32768, 128, "causal", peak=1.6),
        # one new token of four sequences with unequal caches in 16 bits
        attn_case("attn_decode_64k", "fwd", 4, 32, 8, 1, 65536, 128, "padded", layout=2),
        # the training step on 8K causal tokens
        attn_case("attn_train_8k", "train", 1, 32, 8, 8192, 8192, 128, "causal", peak=1.3),
        # a padded batch of odd length (rows behind each sequence see nothing), small heads
        attn_case("attn_train_pad", "train", 3, 12, 4, 1001, 1001, 64, "padded", layout=3),
        # prompts of four sequences go into the cache and are read back for a chunk that follows
        append_case("append_prompt_4k", 4, 8, 128, 64, 700, 4096, layout=4),
        # one new token of each of 32 short sequences, most pages begun already
        append_case("append_token", 32, 8, 128, 16, 120, 1, layout=5),
        # one new token of four sequences with unequal caches of up to 128K tokens
        cache_case("cache_128k", 4, 32, 8, 1, 131072, 128, 64, layout=6),
        # five drafted tokens of a few short sequences
        cache_case("cache_draft_1k", 3, 16, 4, 5, 1000, 128, 16, layout=7),
        # one new token of four sequences, positions on three axes
        rope_case("rope_decode", "fwd", 4, 32, 8, 1, 1, 1, 128, (16, 24, 24), False, "halves"),
        # a training step on the patches of a clip
        rope_case("rope_train_clip", "train", 1, 32, 8, 16, 34, 60, 128, (24, 20, 20), True, "halves"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    layout = rng.randrange(1, 1 << 20)
    op = rng.choice(("attn", "attn", "append", "cache", "rope"))
    d = rng.choice((64, 128))
    Hk = rng.choice((1, 2, 4, 8))
    H = Hk * rng.choice((1, 2, 3, 4, 8))
    if op == "attn":
        form = rng.choice(("fwd", "train"))
        B = rng.choice((1, 2, 3))
        if form == "fwd" and rng.random() < 0.35:  # a few rows against a long cache
            Nq, Nk = rng.choice((1, 1, 2, 5, 16, 40)), log_int(rng, 100, 65536)
            return attn_case("", form, B, H, Hk, Nq, max(Nk, Nq), d, rng.choice(("causal", "padded", "full")), layout)
        most = min(8192, int(math.sqrt(32 * 8192 * 8192 / (2 * B * H))))
        Nk = log_int(rng, 17, most)
        mask = rng.choice(("causal", "docs", "padded", "window", "full"))
        # a chunk of new rows against a longer prefix, where the mask is made for it
        Nq = log_int(rng, 17, Nk) if mask in ("causal", "full") and rng.random() < 0.4 else Nk
        return attn_case("", form, B, H, Hk, Nq, Nk, d, mask, layout, rng.choice((1.0, 1.6)))
    if op == "append":
        new = rng.choice((1, log_int(rng, 2, 4096)))
        return append_case("", rng.choice((1, 2, 3, 4)) if new > 64 else log_int(rng, 1, 64), Hk, d, rng.choice((16, 32, 64, 128)),
                           log_int(rng, 1, 700), new, layout)
    if op == "cache":
        B = rng.choice((1, 2, 4))
        return cache_case("", B, H, Hk, rng.choice((1, 1, 2, 5, 16)), log_int(rng, 20, 131072), d, rng.choice((16, 32, 64, 128)), layout)
    half = d // 2
    s1 = 4 * rng.randrange(1, half // 12 + 1) if rng.random() < 0.7 else rng.randrange(1, half // 3)
    rot_half = rng.choice((half, half // 2)) if 2 * s1 < half // 2 else half
    return rope_case("", rng.choice(("fwd", "train")), rng.choice((1, 2)), H, Hk, log_int(rng, 1, 8), log_int(rng, 1, 40),
                     log_int(rng, 1, 60), d, (rot_half - 2 * s1, s1, s1), rng.random() < 0.5, rng.choice(("halves", "neighbours")),
                     rng.choice(("bf16", "f32")))


# ---------------------------------------------------------------------------
# what a case's layout says
# ---------------------------------------------------------------------------
def key_ranges(case):
    """(begin, end) as int32 [B, Nq] and offset as int32 [B] on the CPU: row i of batch b stands at key position i + offset."""
    B, Nq, Nk, mask = case["B"], case["Nq"], case["Nk"], case["mask"]
    r = random.Random(case["layout"])
    begin = torch.zeros((B, Nq), dtype=torch.int64)
    end = torch.full((B, Nq), Nk, dtype=torch.int64)
    offset = torch.full((B,), Nk - Nq, dtype=torch.int64)
    rows = torch.arange(Nq)
    if mask == "padded":  # lengths of 55 to 100 percent; one item of a larger batch is whole
        for b in range(B):
            n = Nk if b == 0 and B > 1 else max(1, int(Nk * r.uniform(0.55, 1.0)))
            if Nq == Nk:  # rows behind the sequence see nothing
                offset[b] = 0
                end[b] = torch.where(rows < n, rows + 1, torch.zeros_like(rows))
            else:  # the new tokens are the last of a cache of n keys
                n = max(n, Nq)
                offset[b] = n - Nq
                end[b] = rows + offset[b] + 1
    elif mask != "full":
        at = rows + Nk - Nq
        end = (at + 1).repeat(B, 1)
        if mask == "docs":  # documents of log-normal length
            for b in range(B):
                start = 0
                while start < Nk:
                    n = max(1, min(Nk - start, int(r.lognormvariate(math.log(max(2, Nk / 8)), 0.8))))
                    begin[b, start:start + n] = start
                    start += n
        elif mask == "window":
            w = max(1, Nk // r.choice((8, 16, 30)))
            begin = (at - w + 1).clamp_min(0).repeat(B, 1)
    return begin.int(), end.int(), offset.int()


def cache_layout(case):
    """(lengths, new tokens, page table, pages) as lists of numbers: what the sequences hold, in pages of a shuffled pool."""
    r = random.Random(case["layout"])
    B, page = case["B"], case["page"]
    if case["op"] == "append":
        held = [r.randrange(0, case["held"] + 1) for _ in range(B)]
        new = [case["new"]] + [case["new"] if case["new"] == 1 else r.randrange(0, case["new"] + 1) for _ in range(B - 1)]
        most = case["held"] + case["new"]
    else:
        most, new = max(case["Nk"], case["Nq"]), [0] * B
        held = [most] + [max(case["Nq"], int(most * r.uniform(0.4, 1.0))) for _ in range(B - 1)]
    per = -(-most // page)
    order = list(range(B * per + 1))
    r.shuffle(order)
    return held, new, [order[b * per:(b + 1) * per] for b in range(B)], B * per + 1


def axes_of_pairs(case):
    """The axis that turns each pair: sections one after the other, or spread (in turn, as long as an axis has pairs left)."""
    left = [case["s0"], case["s1"], case["s2"]]
    if not case["spread"]:
        return [a for a in range(3) for _ in range(left[a])]
    axes = []
    while sum(left):
        for a in range(3):
            if left[a]:
                axes.append(a)
                left[a] -= 1
    return axes


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def power_of_two(e):
    """2^e of whole numbers in -126 .. 127, in 32 bits (exp2 may be off by a rounding)."""
    return ((e.int() + 127) << 23).view(F32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=F32)

    s = dict(case)
    if case["op"] == "attn":
        B, H, Hk, Nq, Nk, d = (case[k] for k in ("B", "H", "Hk", "Nq", "Nk", "d"))
        # heads lie beside one another in a token, as projections leave them; `peak` makes the attention peaked
        s["q"] = (normal(B, Nq, H, d) * case["peak"]).to(BF16).transpose(1, 2)
        s["k"], s["v"] = ((normal(B, Nk, Hk, d) * p).to(BF16).transpose(1, 2) for p in (case["peak"], 1.0))
        s["ranges"] = tuple(t.cuda() for t in key_ranges(case))
        if case["form"] == "train":
            s["do"] = normal(B, H, Nq, d).to(BF16)
        return s
    if case["op"] in ("append", "cache"):
        held, new, table, pages = cache_layout(case)
        Hk, d, T = case["Hk"], case["d"], case["page"]
        s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
        s["lengths"] = torch.tensor(held, dtype=torch.int32, device="cuda")
        values = []
        for _ in range(2):  # pages hold heads of different sizes, each with the scale that a cache gives it
            x = normal(pages, Hk, T, d) * power_of_two(torch.randint(-2, 3, (pages, Hk, 1, 1), generator=g, device="cuda"))
            top = x.abs().amax((2, 3), keepdim=True)
            scale = power_of_two(torch.ceil(torch.log2(top / E4M3_MAX)))
            values.append(((x / scale).to(E4M3), scale.reshape(pages, Hk)))
        (s["k"], s["ks"]), (s["v"], s["vs"]) = values
        if case["op"] == "append":
            s["counts"] = torch.tensor(new, dtype=torch.int32, device="cuda")
            s["after"] = s["lengths"] + s["counts"]
            size = power_of_two(torch.randint(-1, 4, (case["B"], Hk, 1, 1), generator=g, device="cuda"))
            s["nk"], s["nv"] = ((normal(case["B"], Hk, case["new"], d) * size).to(BF16) for _ in range(2))
        else:
            s["q"] = normal(case["B"], case["H"], case["Nq"], d).to(BF16)
        return s
    B, H, Hk, d = (case[k] for k in ("B", "H", "Hk", "d"))
    t, y, x = torch.meshgrid(*(torch.arange(case[k], device="cuda") for k in ("frames", "height", "width")), indexing="ij")
    N, rot = t.numel(), 2 * (case["s0"] + case["s1"] + case["s2"])
    packed = normal(B, N, H + 2 * Hk, d).to(BF16)  # one projection's output, the values behind the keys
    s["q"], s["k"] = packed[:, :, :H].transpose(1, 2), packed[:, :, H:H + Hk].transpose(1, 2)
    s["wq"], s["wk"] = (1 + 0.1 * normal(d) for _ in range(2))
    first = torch.randint(0, 50, (B, 1), generator=g, device="cuda")  # text stands before the pictures
    s["positions"] = torch.stack([first + a.reshape(1, -1) for a in (t, y, x)]).to(torch.int32)  # [3, B, N]
    at = torch.arange(50 + max(case["frames"], case["height"], case["width"]), device="cuda", dtype=F64)
    angle = at[:, None] * torch.tensor([10000.0 ** (-2.0 * e / rot) for e in range(rot // 2)], device="cuda", dtype=F64)
    s["table"] = torch.stack((angle.cos(), angle.sin()), -1).to(F32)  # [positions, rot / 2, 2]
    s["axes"] = tuple(axes_of_pairs(case))
    if case["form"] == "train":
        kind = BF16 if case["grad"] == "bf16" else F32
        s["gq"], s["gk"] = normal(B, H, N, d).to(kind), normal(B, Hk, N, d).to(kind)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (OWN if own else PLAIN)[s["op"]](s)


def own_attn(s):
    from attention_kl_divergence_gb300 import streamkl

    if s["form"] != "train":
        return streamkl.attn_fwd(s["q"], s["k"], s["v"], ranges=s["ranges"])
    O, LSE, rest = streamkl.attn_fwd(s["q"], s["k"], s["v"], ranges=s["ranges"], rest=True)
    return (O, LSE) + streamkl.attn_bwd(s["do"], s["q"], s["k"], s["v"], O, LSE, rest=rest, ranges=s["ranges"])


def own_append(s):
    from attention_kl_divergence_gb300 import streamkl

    cache = streamkl.Cache8(s["k"], s["v"], s["ks"], s["vs"])
    streamkl.cache8_append(cache, s["table"], s["lengths"], s["nk"], s["nv"], counts=s["counts"])
    return streamkl.cache8_read(cache, s["table"], s["after"]) + (cache.k_scale, cache.v_scale)


def own_cache(s):
    from attention_kl_divergence_gb300 import streamkl

    return streamkl.attn_cache8(s["q"], streamkl.Cache8(s["k"], s["v"], s["ks"], s["vs"]), s["table"], s["lengths"])


def own_rope(s):
    from attention_kl_divergence_gb300 import streamkl

    how = dict(positions=s["positions"], axes=s["axes"], interleaved=s["pairs"] == "neighbours")
    out = streamkl.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["table"], **how)
    if s["form"] == "train":
        out += streamkl.qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["table"], **how)
    return out


def plain_softmax(z, hidden):
    """(probabilities, log-sum-exp [..., 1]) of the visible scores; a row that sees nothing has zeros and -inf."""
    z = z.masked_fill_(hidden, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(total.masked_fill(total == 0, 1.0)), top + torch.log(total)


def plain_attn(s):
    B, H, Hk, Nq, Nk, d = (s[k] for k in ("B", "H", "Hk", "Nq", "Nk", "d"))
    G, scale, train = H // Hk, d ** -0.5, s["form"] == "train"
    begin, end, _ = s["ranges"]
    j = torch.arange(Nk, device="cuda")
    hidden = ((j < begin[..., None]) | (j >= end[..., None]))[:, None, None]  # [B, 1, 1, Nq, Nk]
    step = max(1, min(Hk, (1 << 31) // (B * G * Nq * Nk)))  # key heads at a time
    parts = []
    for h in range(0, Hk, step):
        k, v = s["k"][:, h:h + step, None].float(), s["v"][:, h:h + step, None].float()
        q = s["q"][:, h * G:(h + step) * G].float().reshape(B, -1, G, Nq, d)
        p, lse = plain_softmax(torch.matmul(q, k.transpose(-1, -2)).mul_(scale), hidden)
        o = torch.matmul(p, v)
        part = [o.reshape(B, -1, Nq, d).to(BF16), lse.reshape(B, -1, Nq)]
        if train:
            do = s["do"][:, h * G:(h + step) * G].float().reshape(q.shape)
            dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
            ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
            grads = torch.matmul(ds, k).reshape(B, -1, Nq, d), torch.matmul(ds.transpose(-1, -2), q).sum(2), dv
            part += [x.to(BF16) for x in grads]
            del ds
        del p
        parts.append(part)
    return tuple(torch.cat(x, 1) for x in zip(*parts))


def plain_append(s):
    """Pages are gathered into the sequences' order, changed there and scattered back."""
    B, Hk, d, T = (s[k] for k in ("B", "Hk", "d", "page"))
    table = s["table"].long()
    M = table.shape[1]
    at = torch.arange(M * T, device="cuda")[None]
    first, last = s["lengths"].long()[:, None], s["after"].long()[:, None]
    fresh = ((at >= first) & (at < last))[:, None, :, None]                  # new tokens
    valid = (at < last)[:, None, :, None]
    source = (at - first).clamp(0, s["new"] - 1)[:, None, :, None].expand(B, Hk, M * T, d)
    starts = torch.arange(M, device="cuda")[None] * T
    touched = ((starts < last) & (starts + T > first))[:, None]              # [B, 1, M]
    begun = (starts < first)[:, None]                                        # the page held tokens before
    out = []
    for name, scale, new in (("k", "ks", "nk"), ("v", "vs", "nv")):
        x = torch.gather(s[new], 2, source).float()
        old_scale = s[scale][table].transpose(1, 2)                          # [B, Hk, M]
        top = (x.abs() * fresh).reshape(B, Hk, M, T * d).amax(-1)
        e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(LEAST_EXPONENT, 120)
        e = torch.where(top > E4M3_MAX * power_of_two(e), e + 1, e)          # the logarithm may be off by a rounding
        e = torch.where((top <= E4M3_MAX * power_of_two(e - 1)) & (e > LEAST_EXPONENT), e - 1, e)
        want = power_of_two(e)
        now = torch.where(touched, torch.where(begun, torch.maximum(old_scale, want), want), old_scale)
        held = s[name][table].transpose(1, 2).float()                        # [B, Hk, M, T, d]
        held = held * (old_scale / now)[..., None, None]
        values = torch.where(fresh.reshape(B, 1, M, T, 1), x.reshape(held.shape) / now[..., None, None], held)
        keep = valid.reshape(B, 1, M, T, 1)
        bits = torch.where(keep & touched[..., None, None], values, s[name][table].transpose(1, 2).float()).to(E4M3)
        s[name][table.reshape(-1)] = bits.transpose(1, 2).reshape(B * M, Hk, T, d)
        s[scale][table.reshape(-1)] = now.transpose(1, 2).reshape(B * M, Hk)
        out.append((bits.float() * now[..., None, None]).reshape(B, Hk, M * T, d).masked_fill(~valid, 0.0).to(BF16))
    return tuple(out) + (s["ks"], s["vs"])


def plain_cache(s):
    B, H, Hk, Nq, d, T = (s[k] for k in ("B", "H", "Hk", "Nq", "d", "page"))
    table = s["table"].long()
    Nk = table.shape[1] * T
    j = torch.arange(Nk, device="cuda")
    rows = torch.arange(Nq, device="cuda")[None, :, None] - Nq + 1
    outs, logs = [], []
    for b in range(B):
        k, v = (((s[n][table[b]].float() * s[c][table[b]][..., None, None]).transpose(0, 1).reshape(Hk, 1, Nk, d))
                for n, c in (("k", "ks"), ("v", "vs")))
        q = s["q"][b].float().reshape(Hk, H // Hk, Nq, d)
        p, lse = plain_softmax(torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5), j >= rows + s["lengths"][b])
        outs.append(torch.matmul(p, v.masked_fill((j >= s["lengths"][b])[:, None], 0.0)).reshape(H, Nq, d))
        logs.append(lse.reshape(H, Nq))
    return torch.stack(outs).to(BF16), torch.stack(logs)


def plain_turn(x, c, s, rot, neighbours):
    """The first `rot` values of every head turned by the angles of its position."""
    if neighbours:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).reshape(*x.shape[:-1], rot)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rot:]), -1)


def plain_rope(s):
    nb, rot = s["pairs"] == "neighbours", 2 * len(s["axes"])
    pair = torch.arange(rot // 2, device="cuda")
    at = s["positions"].long()[torch.tensor(s["axes"], device="cuda")].permute(1, 2, 0)  # [B, N, rot / 2]
    turn = s["table"][at, pair][:, None]
    c, sn = turn[..., 0], turn[..., 1]
    out, more, dw = [], [], []
    for x, w, g in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
        n = xf * r
        out.append(plain_turn(n * w, c, sn, rot, nb).to(BF16))
        if g is not None:
            back = plain_turn(g.float(), c, -sn, rot, nb)
            gw = back * w
            more.append((r * (gw - n * (gw * n).mean(-1, keepdim=True))).to(BF16))
            dw.append((back * n).sum((0, 1, 2)))
    return tuple(out + more + dw)


OWN = dict(attn=own_attn, append=own_append, cache=own_cache, rope=own_rope)
PLAIN = dict(attn=plain_attn, append=plain_append, cache=plain_cache, rope=plain_rope)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    train = case.get("form") == "train"
    if case["op"] == "attn":
        B, H, Hk, Nq, Nk, d = (case[k] for k in ("B", "H", "Hk", "Nq", "Nk", "d"))
        begin, end, _ = key_ranges(case)
        pairs = H * int((end - begin).clamp_min(0).sum())
        q, rows = B * H * Nq * d, B * H * Nq
        # keys that some row sees (a cache behind its length is not read)
        seen = Hk * d * int((end.amax(1) - torch.where(end > begin, begin, torch.full_like(begin, Nk)).amin(1)).clamp_min(0).sum())
        size, products = 4 * q + 4 * seen + 4 * rows, 2
        if train:  # inputs, output and its gradient again, three gradients
            size += 6 * q + 4 * seen + 4 * rows + 2 * (q + 2 * B * Hk * Nk * d)
            products += 5
        return {"bytes": size, "flops": 2 * products * pairs * d}
    if case["op"] == "append":
        held, new, table, _ = cache_layout(case)
        row, T = case["Hk"] * case["d"], case["page"]
        begun = sum(h % T for h, n in zip(held, new) if n)  # read with the page that goes on
        # new tokens in and out, then the cache in, its values out (zeros behind a sequence among them)
        size = 2 * row * (3 * sum(new) + begun + sum(held) + sum(new) + 2 * len(table) * len(table[0]) * T)
        return {"bytes": size, "flops": 4 * row * sum(new)}
    if case["op"] == "cache":
        held, _, table, _ = cache_layout(case)
        B, H, Hk, Nq, d = (case[k] for k in ("B", "H", "Hk", "Nq", "d"))
        seen = sum(held)
        return {"bytes": 2 * seen * Hk * d + 8 * Hk * sum(-(-n // case["page"]) for n in held) + 4 * B * H * Nq * d + 4 * B * H * Nq,
                "flops": 4 * H * d * sum(Nq * n - Nq * (Nq - 1) // 2 for n in held)}
    B, H, Hk, d = (case[k] for k in ("B", "H", "Hk", "d"))
    tokens = B * case["frames"] * case["height"] * case["width"]
    n = tokens * (H + Hk) * d
    size, flops = 4 * n + 12 * tokens, 8 * n
    if train:
        size += n * (4 + (2 if case["grad"] == "bf16" else 4)) + 12 * tokens
        flops += 16 * n
    return {"bytes": size, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    return dict(attn=exact_attn, append=exact_append, cache=exact_cache, rope=exact_rope)[case["op"]](state)


def exact_rows(q, k, v, sees):
    """Softmax attention of one head in 64 bits: (output, log-sum-exp, rows that see a key)."""
    live = sees.any(1)
    sees = sees.clone()
    sees[:, 0] |= ~live  # an empty row gets one key here, and none of what follows from it below
    z = (q @ k.T / math.sqrt(q.shape[1])).masked_fill(~sees, -math.inf)
    return torch.softmax(z, 1) @ v, torch.logsumexp(z.detach(), 1).masked_fill(~live, -math.inf), live


def exact_attn(s):
    B, H, Hk, Nq, Nk, d = (s[k] for k in ("B", "H", "Hk", "Nq", "Nk", "d"))
    O, LSE = torch.zeros((B, H, Nq, d), dtype=F64, device="cuda"), torch.zeros((B, H, Nq), dtype=F64, device="cuda")
    train = s["form"] == "train"
    grads = [torch.zeros(x.shape, dtype=F64, device="cuda") for x in (s["q"], s["k"], s["v"])] if train else []
    key = torch.arange(Nk, device="cuda")[None]
    for b in range(B):
        sees = (key >= s["ranges"][0][b][:, None]) & (key < s["ranges"][1][b][:, None])
        for h in range(H):
            hk = h * Hk // H
            leaves = [x.double().requires_grad_(train) for x in (s["q"][b, h], s["k"][b, hk], s["v"][b, hk])]
            o, lse, live = exact_rows(*leaves, sees)
            O[b, h], LSE[b, h] = torch.where(live[:, None], o.detach(), torch.zeros_like(o)), lse
            if train:
                g = torch.where(live[:, None], s["do"][b, h].double(), torch.zeros_like(o))
                dq, dk, dv = torch.autograd.grad((o * g).sum(), leaves)
                grads[0][b, h] = dq
                grads[1][b, hk] += dk
                grads[2][b, hk] += dv
            del o, leaves
    return (O, LSE, *grads)


def nearest_e4m3(x):
    """Nearest multiple of the step at x (ties to the even one): 2^-3 of its power of two, 2^-9 at the least."""
    _, e = torch.frexp(x)
    step = ((e.long() - 4).clamp_min(-9) + 1023 << 52).view(F64)
    return torch.round(x / step) * step


def exact_append(s):
    """Sequence by sequence, page by page."""
    B, Hk, d, T = (s[k] for k in ("B", "Hk", "d", "page"))
    M = s["table"].shape[1]
    out, scales = [], []
    for name, scale, new in (("k", "ks", "nk"), ("v", "vs", "nv")):
        values, sc = s[name].double(), s[scale].double()
        res = torch.zeros((B, Hk, M * T, d), dtype=F64, device="cuda")
        for b in range(B):
            held, last = int(s["lengths"][b]), int(s["after"][b])
            for m in range(-(-last // T)):
                page, lo, hi = int(s["table"][b, m]), max(held, m * T), min(last, (m + 1) * T)
                if hi > lo:
                    x = s[new][b, :, lo - held:hi - held].double()
                    tops = [math.frexp(a / E4M3_MAX) for a in x.abs().amax((1, 2)).tolist()]
                    # the smallest power of two that is not less
                    want = [2.0 ** max(LEAST_EXPONENT, e - 1 if f == 0.5 else e if f else LEAST_EXPONENT) for f, e in tops]
                    want = torch.tensor(want, dtype=F64, device="cuda")
                    was = sc[page].clone()
                    now = torch.maximum(was, want) if lo > m * T else want
                    values[page, :, :lo - m * T] = nearest_e4m3(values[page, :, :lo - m * T] * (was / now)[:, None, None])
                    values[page, :, lo - m * T:hi - m * T] = nearest_e4m3(x / now[:, None, None])
                    sc[page] = now
                n = min(last, (m + 1) * T) - m * T
                res[b, :, m * T:m * T + n] = values[page, :, :n] * sc[page][:, None, None]
        out.append(res)
        scales.append(sc)
    return tuple(out + scales)


def exact_cache(s):
    B, H, Hk, Nq, d, T = (s[k] for k in ("B", "H", "Hk", "Nq", "d", "page"))
    O, LSE = torch.zeros((B, H, Nq, d), dtype=F64, device="cuda"), torch.zeros((B, H, Nq), dtype=F64, device="cuda")
    for b in range(B):
        n = int(s["lengths"][b])
        pages = s["table"][b, :-(-n // T)].long()
        sees = torch.arange(n, device="cuda")[None] <= torch.arange(n - Nq, n, device="cuda")[:, None]
        for hk in range(Hk):
            k, v = ((s[x][pages, hk].double() * s[c][pages, hk].double()[:, None, None]).reshape(-1, d)[:n]
                    for x, c in (("k", "ks"), ("v", "vs")))
            for h in range(hk * H // Hk, (hk + 1) * H // Hk):
                O[b, h], LSE[b, h], _ = exact_rows(s["q"][b, h].double(), k, v, sees)
    return O, LSE


def exact_rope(s):
    """Rotation as a product of complex numbers, gradients by autograd, heads in groups."""
    d, rot = s["d"], 2 * len(s["axes"])
    turn = torch.view_as_complex(s["table"].double())
    out, dx, dw = [], [], []
    for x, w, g in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        y, gx, gw = [], [], torch.zeros(d, dtype=F64, device="cuda")
        for b in range(s["B"]):
            c = torch.stack([turn[s["positions"][a, b].long(), e] for e, a in enumerate(s["axes"])], -1)
            for heads in torch.arange(x.shape[1], device="cuda").split(4):
                xi, wi = x[b, heads].double().requires_grad_(), w.double().requires_grad_()
                n = xi / torch.sqrt(xi.pow(2).mean(-1, keepdim=True) + 1e-6) * wi
                part = n[..., :rot]
                near = s["pairs"] == "neighbours"
                part = part.unflatten(-1, (rot // 2, 2)) if near else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
                part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * c)
                part = part.flatten(-2) if near else part.transpose(-1, -2).flatten(-2)
                yi = torch.cat((part, n[..., rot:]), -1)
                y.append(yi.detach())
                if g is not None:
                    a, v = torch.autograd.grad((yi * g[b, heads].double()).sum(), (xi, wi))
                    gx.append(a)
                    gw += v
        out.append(torch.cat(y).reshape(x.shape))
        if g is not None:
            dx.append(torch.cat(gx).reshape(x.shape))
            dw.append(gw)
    return tuple(out + dx + dw)
