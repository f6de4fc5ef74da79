"""Timed cases of two operators beside the attention KL divergence.

``score``: the KL divergence of two attentions whose scores are capped by a
tanh, get a bias that falls with distance, and are masked by a key range of
each query row (causal, document, window, prefix and padding masks), with its
gradient to one side and its form for single new tokens.

``norm_rope``: the norm of every query and key head with the position rotation
in the same pass, and its gradient.

The plain forms are elementary torch operations in 32 bits, rounded once at the
end; ``exact`` restates the definitions in 64 bits through autograd.
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def score_case(name, form, B, H, Hk, Nq, Nk, d, mask, layout=0, cap1=0.0, cap2=0.0, bias=False, setting=0, peak=1.0):
    """form: fwd, train (forward and the gradient of one side) or decode."""
    return dict(name=name, op="score", form=form, B=B, H=H, Hk=Hk, Nq=Nq, Nk=Nk, d=d, mask=mask, layout=layout, cap1=cap1,
                cap2=cap2, bias=bias, setting=setting, peak=peak)


def norm_case(name, form, B, H, Hk, N, d, rot, pairs, grad="bf16", weights="f32", packed=True, far=0):
    """form: fwd or train; pairs: halves (e, e + rot/2) or neighbours (2e, 2e + 1); far: first position."""
    return dict(name=name, op="norm_rope", form=form, B=B, H=H, Hk=Hk, N=N, d=d, rot=rot, pairs=pairs, grad=grad, weights=weights,
                packed=packed, far=far)


def listed():
    return [
        # a unit-sized problem: what one call costs in latency
        score_case("score_fwd_tiny", "fwd", 1, 2, 2, 256, 256, 64, "causal", cap1=50.0, cap2=50.0),
        # packed documents of uneven lengths in one 8K sequence, plain scores: the loss alone, as an evaluation runs it
        score_case("score_fwd_docs_8k", "fwd", 1, 32, 8, 8192, 8192, 128, "docs", layout=1),
        # 8K causal training step of the student against a teacher with capped scores, keys shared by four heads
        score_case("score_train_cap_8k", "train", 1, 32, 8, 8192, 8192, 128, "causal", cap1=50.0, cap2=50.0, setting=1, peak=1.6),
        # packed documents, both sides capped differently, the teacher trains
        score_case("score_train_docs_4k", "train", 1, 16, 16, 4096, 4096, 128, "docs", layout=2, cap1=50.0, cap2=30.0, setting=2, peak=1.6),
        # a padded batch (rows behind each sequence see nothing) with distance biases, odd length, small heads
        score_case("score_train_bias_pad", "train", 3, 8, 8, 1001, 1001, 64, "padded", layout=3, bias=True, setting=1),
        # a prefix seen by every row, distance bias and cap at once
        score_case("score_train_prefix", "train", 2, 8, 2, 2048, 2048, 128, "prefix", layout=4, cap1=30.0, cap2=30.0, bias=True, setting=2),
        # a sliding window over a long sequence
        score_case("score_fwd_window_16k", "fwd", 1, 8, 8, 16384, 16384, 128, "window", layout=5, cap1=50.0),
        # one new token of four sequences with unequal caches, keys shared by four heads, capped
        score_case("score_decode_128k", "decode", 4, 32, 8, 1, 131072, 128, "padded", layout=6, cap1=50.0, cap2=50.0),
        # one new token of four sequences
        norm_case("norm_rope_decode", "fwd", 4, 32, 8, 1, 128, 128, "halves", far=131071),
        # a prompt of 8K tokens out of one packed projection
        norm_case("norm_rope_fwd_8k", "fwd", 1, 32, 8, 8192, 128, 128, "halves"),
        # the training step of the same width at 64K tokens
        norm_case("norm_rope_train_64k", "train", 1, 32, 8, 65536, 128, 128, "halves"),
        # small heads, part of each head rotated, neighbouring pairs, odd length, gradients in 32 bits
        norm_case("norm_rope_train_part", "train", 3, 12, 4, 4097, 64, 32, "neighbours", grad="f32", weights="bf16", packed=False, far=100000),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    layout = rng.randrange(1, 1 << 20)
    if rng.random() < 0.35:
        d = rng.choice((64, 128))
        form = rng.choice(("fwd", "train"))
        heads = rng.choice(((8, 8), (16, 4), (32, 8), (12, 4), (32, 32)))
        most = 65536 * 40 // (heads[0] + heads[1])
        tokens = log_int(rng, 1, most)
        B = rng.choice([b for b in (1, 2, 3, 4) if b <= tokens])
        rot = rng.choice((d, d // 2))
        return norm_case("", form, B, *heads, max(1, tokens // B), d, rot, rng.choice(("halves", "neighbours")),
                         rng.choice(("bf16", "f32")), rng.choice(("bf16", "f32")), rng.random() < 0.5, rng.choice((0, 77, 500000)))
    d = rng.choice((64, 128))
    Hk = rng.choice((2, 4, 8))
    H = Hk * rng.choice((1, 2, 4))
    form = rng.choice(("fwd", "train", "train", "decode"))
    cap1, cap2 = rng.choice(((0.0, 0.0), (50.0, 50.0), (30.0, 0.0), (50.0, 20.0)))
    setting = 0 if form != "train" else rng.choice((1, 2))
    if form == "decode":
        B, Nq, Nk = rng.choice((1, 2, 4)), rng.choice((1, 1, 2, 7, 16)), log_int(rng, 100, 131072)
        if Nq > Nk:
            Nq = 1
        mask = rng.choice(("causal", "padded", "full"))
    else:
        B = rng.choice((1, 2, 3))
        most = min(8192, int(math.sqrt(32 * 8192 * 8192 / (2 * B * H))))
        Nk = log_int(rng, 33, most)
        mask = rng.choice(("causal", "docs", "padded", "prefix", "window", "full"))
        # a chunk of new rows against a longer prefix, where the mask is made for it
        Nq = log_int(rng, 17, Nk) if mask in ("causal", "full") and rng.random() < 0.4 else Nk
    return score_case("", form, B, H, Hk, Nq, Nk, d, mask, layout, cap1, cap2, rng.random() < 0.4, setting, rng.choice((1.0, 1.6)))


# ---------------------------------------------------------------------------
# masks: the key range [begin, end) of each row, and the position of row 0
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
        elif mask == "prefix":
            for b in range(B):
                end[b] = end[b].clamp_min(int(Nk * r.uniform(0.1, 0.6)))
    return begin.int(), end.int(), offset.int()


def bias_slopes(H):
    """Slopes of the distance bias, 2^(-8 (h + 1) / H)."""
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=F32)

    s = dict(case)
    if case["op"] == "score":
        B, H, Hk, Nq, Nk, d = (case[k] for k in ("B", "H", "Hk", "Nq", "Nk", "d"))
        # a student near its teacher; `peak` makes the attention of both peaked, where caps matter
        q1, k1 = normal(B, H, Nq, d) * case["peak"], normal(B, Hk, Nk, d) * case["peak"]
        q2, k2 = q1 + 0.3 * normal(B, H, Nq, d), k1 + 0.3 * normal(B, Hk, Nk, d)
        s["qk"] = tuple(t.to(BF16) for t in (q1, k1, q2, k2))
        s["begin"], s["end"], s["offset"] = (t.cuda() for t in key_ranges(case))
        s["slopes"] = torch.tensor(bias_slopes(H), dtype=F32, device="cuda") if case["bias"] else None
        if case["form"] == "train":
            s["g"] = normal(B, H, Nq).abs() / Nq
        return s
    B, H, Hk, N, d, rot = (case[k] for k in ("B", "H", "Hk", "N", "d", "rot"))
    if case["packed"]:  # one projection's output, [B, N, H + 2 Hk, d] with the values behind the keys
        x = normal(B, N, H + 2 * Hk, d).to(BF16)
        s["q"], s["k"] = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
    else:
        s["q"], s["k"] = normal(B, H, N, d).to(BF16), normal(B, Hk, N, d).to(BF16)
    w = BF16 if case["weights"] == "bf16" else F32
    s["wq"], s["wk"] = ((1 + 0.1 * normal(d)).to(w) for _ in range(2))
    # cosines and sines of every position that the program may meet, made once from angles in 64 bits
    last = case["far"] + N + 1
    at = torch.arange(last, device="cuda", dtype=F64)
    freq = torch.tensor([10000.0 ** (-2.0 * e / rot) for e in range(rot // 2)], device="cuda", dtype=F64)
    angle = at[:, None] * freq
    s["table"] = torch.stack((angle.cos(), angle.sin()), -1).to(F32)  # [positions, rot / 2, 2]
    first = torch.randint(0, 2, (B, 1), generator=g, device="cuda")  # each sequence has a start of its own
    s["positions"] = (case["far"] + first + torch.arange(N, device="cuda")).to(torch.int32)
    if case["form"] == "train":
        t = BF16 if case["grad"] == "bf16" else F32
        s["gq"], s["gk"] = normal(B, H, N, d).to(t), normal(B, Hk, N, d).to(t)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if s["op"] == "score":
        return own_score(s) if own else plain_score(s)
    return own_norm_rope(s) if own else plain_norm_rope(s)


def own_score(s):
    from attention_kl_divergence_gb300 import streamkl

    Q1, K1, Q2, K2 = s["qk"]
    scores = streamkl.Scores(cap1=s["cap1"], cap2=s["cap2"], slopes1=s["slopes"], slopes2=s["slopes"], begin=s["begin"],
                             end=s["end"], offset=s["offset"])
    KL, L1, L2 = streamkl.kl_score_fwd(scores, Q1, K1, Q2, K2)
    if s["form"] != "train":
        return KL, L1, L2
    dQ, dK = streamkl.kl_score_bwd(s["setting"], scores, s["g"], Q1, K1, Q2, K2, KL, L1, L2, grad_dtype=BF16)
    return KL, L1, L2, dQ, dK


def own_norm_rope(s):
    from attention_kl_divergence_gb300 import streamkl

    how = dict(positions=s["positions"], eps=1e-6, interleaved=s["pairs"] == "neighbours")
    q, k = streamkl.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["table"], **how)
    if s["form"] != "train":
        return q, k
    return (q, k) + tuple(streamkl.qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["table"], **how))


def plain_side(Q, K, cap, slopes, distance, hidden):
    """(scores of the visible pairs, tanh or None, log-sum-exp, probabilities) of one side, [B, Hk, G, Nq, Nk]."""
    B, H, Nq, d = Q.shape
    Hk, Nk = K.shape[1], K.shape[2]
    s = torch.matmul(Q.float().reshape(B, Hk, -1, d), K.float().transpose(2, 3)).mul_(d ** -0.5)
    s = s.reshape(B, Hk, H // Hk, Nq, Nk)
    t = None
    if cap > 0:
        t = torch.tanh(s / cap)
        s = cap * t
    if slopes is not None:
        s = s - slopes.reshape(1, Hk, H // Hk, 1, 1) * distance
    top = s.masked_fill(hidden, -math.inf).amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top)).masked_fill_(hidden, 0.0)
    total = e.sum(-1, keepdim=True)
    p = e.div_(torch.where(total == 0, torch.ones_like(total), total))
    return s, t, top + torch.log(total), p


def plain_score(s):
    Q1, K1, Q2, K2 = s["qk"]
    B, H, Nq, d = Q1.shape
    Hk, Nk = K1.shape[1], K1.shape[2]
    j = torch.arange(Nk, device="cuda")
    hidden = ((j < s["begin"][..., None]) | (j >= s["end"][..., None])).reshape(B, 1, 1, Nq, Nk)
    at = torch.arange(Nq, device="cuda") + s["offset"][:, None]
    distance = (at[..., None] - j).abs().float().reshape(B, 1, 1, Nq, Nk) if s["slopes"] is not None else None
    s1, t1, l1, p1 = plain_side(Q1, K1, s["cap1"], s["slopes"], distance, hidden)
    s2, t2, l2, p2 = plain_side(Q2, K2, s["cap2"], s["slopes"], distance, hidden)
    empty = l1 == -math.inf
    zero = torch.zeros_like(l1)
    ratio = (s1 - torch.where(empty, zero, l1)) - (s2 - torch.where(empty, zero, l2))
    del s1, s2
    KL = (p1 * ratio).sum(-1, keepdim=True)
    rows = tuple(x.reshape(B, H, Nq) for x in (KL, l1, l2))
    if s["form"] != "train":
        return rows
    g = s["g"].reshape(KL.shape)
    if s["setting"] == 1:
        ds, t, cap, Q, K = g * (p2 - p1), t2, s["cap2"], Q2, K2
    else:
        ds, t, cap, Q, K = g * p1 * (ratio - KL), t1, s["cap1"], Q1, K1
    del ratio, p1, p2
    if cap > 0:
        ds = ds * (1 - t * t)
    ds = ds.mul_(d ** -0.5).reshape(B, Hk, -1, Nk)
    dQ = torch.matmul(ds, K.float()).reshape(B, H, Nq, d).to(BF16)
    dK = torch.matmul(ds.transpose(2, 3), Q.float().reshape(B, Hk, -1, d)).to(BF16)
    return rows + (dQ, dK)


def plain_turn(x, c, s, rot, neighbours):
    """The first `rot` values of every head turned by the angles of its position."""
    if neighbours:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).reshape(*x.shape[:-1], rot)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rot:]), -1)


def plain_norm_rope(s):
    rot, nb = s["rot"], s["pairs"] == "neighbours"
    turn = s["table"][s["positions"].long()][:, None]  # [B, 1, N, rot / 2, 2]
    c, sn = turn[..., 0], turn[..., 1]
    out, more, dw = [], [], []
    for x, w, g in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        xf, wf = x.float(), w.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
        n = xf * r
        out.append(plain_turn(n * wf, c, sn, rot, nb).to(BF16))
        if g is not None:
            back = plain_turn(g.float(), c, -sn, rot, nb)
            gw = back * wf
            more.append((r * (gw - n * (gw * n).mean(-1, keepdim=True))).to(BF16))
            dw.append((back * n).sum((0, 1, 2)).to(w.dtype))
    return tuple(out + more + dw)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    train = case["form"] == "train"
    if case["op"] == "score":
        B, H, Hk, Nq, Nk, d = (case[k] for k in ("B", "H", "Hk", "Nq", "Nk", "d"))
        begin, end, _ = key_ranges(case)
        pairs = H * int((end - begin).clamp_min(0).sum())
        q, rows = B * H * Nq * d, B * H * Nq
        # keys that some row sees (a cache behind its length is not read)
        seen = Hk * d * int((end.amax(1) - torch.where(end > begin, begin, torch.full_like(begin, Nk)).amin(1)).clamp_min(0).sum())
        size = 4 * (q + seen) + 12 * rows
        products = 2  # the scores of both sides
        if train:  # scores again, the gradients of the queries and of the keys of one side
            size += 4 * (q + seen) + 16 * rows + 2 * (q + B * Hk * Nk * d)
            products += 4
        return {"bytes": size, "flops": 2 * products * pairs * d}
    B, H, Hk, N, d = (case[k] for k in ("B", "H", "Hk", "N", "d"))
    n = B * N * (H + Hk) * d
    size = 4 * n + 4 * B * N + 4 * B * N * case["rot"]
    flops = 8 * n
    if train:
        size += n * (4 + (2 if case["grad"] == "bf16" else 4)) + 4 * B * N + 4 * B * N * case["rot"]
        flops += 16 * n
    return {"bytes": size, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    return exact_score(state) if case["op"] == "score" else exact_norm_rope(state)


def exact_score(s):
    """Head by head: the divergence of two masked softmaxes and autograd's gradient of it to one side."""
    B, H, Hk, Nq, Nk, d = (s[k] for k in ("B", "H", "Hk", "Nq", "Nk", "d"))
    new = lambda *shape: torch.zeros(shape, dtype=F64, device="cuda")  # noqa: E731
    KL, L1, L2 = new(B, H, Nq), new(B, H, Nq), new(B, H, Nq)
    train = s["form"] == "train"
    dQ, dK = (new(B, H, Nq, d), new(B, Hk, Nk, d)) if train else (None, None)
    slopes = [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]
    if s["bias"]:
        slopes = torch.tensor(slopes, dtype=F32).double().tolist()  # the operator is given slopes in 32 bits
    key = torch.arange(Nk, device="cuda", dtype=torch.int64)[None]
    for b in range(B):
        lo, hi = s["begin"][b].long()[:, None], s["end"][b].long()[:, None]
        live = (hi > lo).reshape(-1)
        sees = (key >= lo) & (key < hi)
        sees[:, 0] |= ~live  # an empty row gets one key here, and none of what follows from it below
        away = (torch.arange(Nq, device="cuda")[:, None] + int(s["offset"][b]) - key).abs().double() if s["bias"] else None
        for h in range(H):
            hk = h * Hk // H
            side, logs = [], []
            for n, cap in ((0, s["cap1"]), (2, s["cap2"])):
                q, k = s["qk"][n][b, h].double(), s["qk"][n + 1][b, hk].double()
                if train and n == (2 if s["setting"] == 1 else 0):
                    q.requires_grad_(), k.requires_grad_()
                    side = [q, k]
                z = q @ k.T / math.sqrt(d)
                if cap > 0:
                    z = torch.tanh(z / cap) * cap
                if s["bias"]:
                    z = z - slopes[h] * away
                z = z.masked_fill(~sees, -math.inf)
                logs.append((z, torch.logsumexp(z, 1)))
                del z
            (z1, n1), (z2, n2) = logs
            lp1 = (z1 - n1[:, None]).masked_fill(~sees, 0.0)
            lp2 = (z2 - n2[:, None]).masked_fill(~sees, 0.0)
            p1 = lp1.exp().masked_fill(~sees, 0.0)
            kl = (p1 * (lp1 - lp2)).sum(1)
            KL[b, h] = torch.where(live, kl.detach(), torch.zeros_like(kl))
            for out, n in ((L1, n1), (L2, n2)):
                out[b, h] = n.detach().masked_fill(~live, -math.inf)
            if train:
                g = torch.where(live, s["g"][b, h].double(), torch.zeros_like(n1))
                gq, gk = torch.autograd.grad((kl * g).sum(), side)
                dQ[b, h] = gq
                dK[b, hk] += gk
            del logs, z1, z2, n1, n2, lp1, lp2, p1, kl, side
    return (KL, L1, L2, dQ, dK) if train else (KL, L1, L2)


def exact_norm_rope(s):
    """Rotation as a product of complex numbers, gradients by autograd, a sequence's heads in groups."""
    rot, d = s["rot"], s["d"]
    turn = torch.view_as_complex(s["table"].double())
    out, dx, dw = [], [], []
    for x, w, g in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        y, gx, gw = [], [], torch.zeros(d, dtype=F64, device="cuda")
        for b in range(s["B"]):
            c = turn[s["positions"][b].long()]
            for heads in torch.arange(x.shape[1], device="cuda").split(4):
                xi = x[b, heads].double().requires_grad_()
                wi = w.double().requires_grad_()
                n = xi / torch.sqrt(xi.pow(2).mean(-1, keepdim=True) + 1e-6) * wi
                part = n[..., :rot]
                part = part.unflatten(-1, (rot // 2, 2)) if s["pairs"] == "neighbours" else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
                part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * c)
                part = part.flatten(-2) if s["pairs"] == "neighbours" else part.transpose(-1, -2).flatten(-2)
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
