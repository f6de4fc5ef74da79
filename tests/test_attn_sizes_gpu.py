"""Attention at the sizes that training and serving have: whole key heads, or the last rows, against float64."""
import pytest
import torch

import test_cache8 as c8
from attention_kl_divergence_gb300 import streamkl as sk
from test_attn import BF16, DEV, Ref, inputs, masks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["causal", "docs"])
def test_training_8k(kind, d):
    N = 8192
    Q, K, V = inputs(1, 32, 8, N, N, d, seed=d)
    dO = torch.randn(Q.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(BF16)
    ranges = masks(kind, 1, N, N)
    O, LSE, rest = sk.attn_fwd(Q, K, V, ranges=ranges, rest=True)
    dQ, dK, dV = sk.attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges)
    for h in (0, 7):
        q, k = slice(4 * h, 4 * h + 4), slice(h, h + 1)
        ref = Ref(Q[:, q], K[:, k], V[:, k], ranges)
        ref.check(O[:, q], LSE[:, q])
        ref.check_grads(dO[:, q], dQ[:, q], dK[:, k], dV[:, k])
        del ref
        torch.cuda.empty_cache()


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_32k(d):
    Q, K, V = inputs(1, 8, 8, 32768, 32768, d, seed=d)
    O, LSE = sk.attn_fwd(Q, K, V, causal=True)
    for h in (0, 7):
        for end in (256, 20000, 32768):
            rows, one = slice(end - 256, end), slice(h, h + 1)
            Ref(Q[:, one, rows], K[:, one, :end], V[:, one, :end], causal=True).check(O[:, one, rows], LSE[:, one, rows])


@pytest.mark.parametrize("Nq", [1, 5])
def test_few_tokens_over_long_caches(Nq):
    """Four caches of up to 128K tokens in 8 bits, and what they hold as bf16."""
    B, H, Hk, T, d, M = 4, 32, 8, 64, 128, 2048
    table, pages = c8.tables(B, M)
    cache = c8.pool(64, Hk, T, d)
    cache = sk.Cache8(*(t.repeat(-(-pages // 64), *[1] * (t.dim() - 1))[:pages].contiguous() for t in
                        (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)))
    cache = sk.Cache8(cache.k.view(c8.E4M3), cache.v.view(c8.E4M3), cache.k_scale, cache.v_scale)
    Q = torch.randn(B, H, Nq, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF16)
    n = torch.tensor([131072, 100003, 64, 70000], dtype=torch.int32, device=DEV)
    O, LSE = sk.attn_cache8(Q, cache, table, n, scale=0.02)
    K, V = sk.cache8_read(cache, table, n)
    ranges = sk.key_ranges(B, Nq, M * T, DEV, q_lengths=torch.full_like(n, Nq), k_lengths=n)
    wide = sk.attn_fwd(Q, K, V, ranges=ranges, scale=0.02)
    for b in range(B):
        one, heads, m = slice(b, b + 1), slice(0, 4), -(-int(n[b]) // T)
        few = sk.Cache8(*(t[:, :1].contiguous() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)))
        few = sk.Cache8(few.k.view(c8.E4M3), few.v.view(c8.E4M3), few.k_scale, few.v_scale)
        c8.Ref(Q[one, heads], few, table[one, :m], n[one], 0.02).check(O[one, heads], LSE[one, heads])
        at = int(n[b])
        Ref(Q[one, heads], K[one, :1, :at], V[one, :1, :at], causal=True, scale=0.02).check(wide[0][one, heads], wide[1][one, heads])
