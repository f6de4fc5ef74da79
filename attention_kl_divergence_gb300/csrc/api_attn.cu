// api_attn.cu -- C ABI of the attention over whole prompts: argument validation,
// launch planning and launches on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"

using namespace streamkl;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Element strides of a [B, heads, N, d] tensor: multiples of 8 (16 bytes), rows
// that do not overlap; an axis with one entry has a stride that is never used.
bool strides_ok(const streamkl_strides& s, int B, int heads, int N, int d) {
    const int64_t st[3] = {s.b, s.h, s.n};
    const int n[3] = {B, heads, N};
    for (int k = 0; k < 3; ++k)
        if (n[k] > 1 && (st[k] < d || st[k] % 8 != 0 || st[k] > (int64_t(1) << 38))) return false;
    return true;
}

// The strides that a tensor map gets: those of unused axes are any valid ones.
streamkl_strides used(const streamkl_strides& s, int B, int heads, int N, int d) {
    return {B > 1 ? s.b : d, heads > 1 ? s.h : d, N > 1 ? s.n : d};
}

streamkl_status check_desc(const streamkl_attn* s, bool backward) {
    if (!s) return STREAMKL_ERR_INVALID_ARG;
    if (s->B < 1 || s->H < 1 || s->H_kv < 1 || s->Nq < 1 || s->Nk < 1 || s->H % s->H_kv != 0) return STREAMKL_ERR_INVALID_ARG;
    if (s->d != 64 && s->d != 128) return STREAMKL_ERR_UNSUPPORTED;
    if (!strides_ok(s->q, s->B, s->H, s->Nq, s->d) || !strides_ok(s->k, s->B, s->H_kv, s->Nk, s->d) ||
        !strides_ok(s->v, s->B, s->H_kv, s->Nk, s->d) || !strides_ok(s->o, s->B, s->H, s->Nq, s->d) ||
        (backward && !strides_ok(s->d_o, s->B, s->H, s->Nq, s->d)))
        return STREAMKL_ERR_INVALID_ARG;
    // rows and keys are counted in 32 bits, up to the end of their tiles
    if (s->Nq > INT32_MAX - 2 * kBlockQ || s->Nk > INT32_MAX - 2 * kBlockK) return STREAMKL_ERR_UNSUPPORTED;
    if (int64_t(s->B) * s->H > (int64_t(1) << 24) || int64_t(s->B) * s->H * s->Nq > (int64_t(1) << 38))
        return STREAMKL_ERR_UNSUPPORTED;
    return STREAMKL_OK;
}

bool options_ok(const streamkl_options* opt) {
    return !opt || (opt->num_splits >= 0 && opt->grad_bf16 == 0 && opt->bwd_mode == 0 &&
                    !(opt->debug_flags & ~STREAMKL_DEBUG_INJECT_STALL));
}

struct AttnFwdPlan {
    AttnFwdParams p;  // the layout of the work
    int ctas;
    size_t ws_bytes;
};

streamkl_status plan_attn_fwd(const streamkl_attn* s, const streamkl_options* opt, AttnFwdPlan* pl) {
    streamkl_status st = check_desc(s, false);
    if (st != STREAMKL_OK) return st;
    if (!options_ok(opt)) return STREAMKL_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != STREAMKL_OK) return st;
    AttnFwdParams& p = pl->p;
    p = AttnFwdParams{};
    p.B = s->B;
    p.H = s->H;
    p.H_kv = s->H_kv;
    p.Nq = s->Nq;
    p.Nk = s->Nk;
    p.group = s->H / s->H_kv;
    // few rows: as many heads of a key head in a tile as fit (a divisor of the group, so that no tile is ragged)
    p.heads = 1;
    p.rows = std::min(s->Nq, kBlockQ);
    for (int c = p.group; c > 1; --c)
        if (p.group % c == 0 && int64_t(c) * s->Nq <= kBlockQ) {
            p.heads = c;
            break;
        }
    p.blocks = p.group / p.heads;
    p.q_tiles = (s->Nq - 1) / kBlockQ + 1;
    // two head blocks have the same keys to see; where they do not pair up, neighbouring query tiles do
    p.pair_heads = p.blocks > 1 && (p.blocks % 2 == 0 || p.q_tiles == 1);
    p.units_h = p.pair_heads ? (p.blocks + 1) / 2 : p.blocks;
    p.units_q = p.pair_heads ? p.q_tiles : (p.q_tiles + 1) / 2;
    const int64_t heads = int64_t(s->B) * s->H_kv * p.units_h, units = heads * p.units_q;
    if (units > INT32_MAX) return STREAMKL_ERR_UNSUPPORTED;
    const int k_tiles = (s->Nk - 1) / kBlockK + 1;
    // One tile with no other to pair with stands twice from 8 key tiles on.  One token (us, in a graph; with twice, without): 4
    // caches, 32 heads on 8, of 896 keys 18.5 / 14.4, 1024 16.4 / 16.4, 1536 16.5 / 16.6, 4096 20.5 / 24.6, 8192 36.9 / 36.9;
    // one cache, 8 heads on 2, 896 keys 16.9 / 14.4, 1024 16.0 / 13.7, 2048 16.4 / 14.4, 4096 18.5 / 18.5.
    p.dual = p.blocks == 1 && p.q_tiles == 1 && k_tiles >= 8;
    int splits = 1;
    if (opt && opt->num_splits > 0) {
        splits = std::min({opt->num_splits, k_tiles, kMaxSplits});
    } else if (p.dual) {
        // Bound by HBM: one wave of CTAs, which saturates it from about two thirds of the SMs on; more waves start and
        // end more often than unequal lengths cost (4 caches of up to 65536 keys, 8 key heads: 3 splits 186 us, 4 160,
        // 5 167, 9 168, 19 185; one cache: 8 splits 77, 14 62, 19 62, 28 83).
        splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms / units, k_tiles / 4)));
    } else {
        // Splits that leave a CTA fewer key tiles by 4 at least: they cost a second kernel.  300 rows, 8 heads (1 split, chosen ones):
        // 512 keys 18.5 / 18.5 us, 640 18.5 / 18.0, 1024 24.6 / 18.5; 256 rows, 4 heads, d = 64: 640 16.4 / 14.4, 1536 28.7 / 16.4; one
        // token, 8 heads on 2: 384 12.3 / 12.3, 512 14.4 / 12.3.
        const int n = choose_splits(units, k_tiles, sms);
        if ((k_tiles + n - 1) / n + 3 < k_tiles) splits = n;
    }
    splits = std::min(splits, kMaxSplits);
    if (units * splits > INT32_MAX) return STREAMKL_ERR_UNSUPPORTED;
    p.num_splits = splits;
    p.parts = p.dual ? 2 * splits : splits;
    pl->ctas = static_cast<int>(units * splits);
    const int group = order_group(heads, p.units_q, sms), last = static_cast<int>(heads % group);
    if (int64_t(group) * p.units_q > INT32_MAX) return STREAMKL_ERR_UNSUPPORTED;
    p.order_group = FastDiv::by(group);
    p.order_last = FastDiv::by(last ? last : group);
    p.order_units = FastDiv::by(int64_t(group) * p.units_q);
    p.by_splits = FastDiv::by(splits);
    p.by_units_h = FastDiv::by(p.units_h);
    p.by_H_kv = FastDiv::by(p.H_kv);
    p.by_rows = FastDiv::by(p.rows);
    pl->ws_bytes = kStatusBytes;
    if (p.parts > 1) pl->ws_bytes += size_t(p.parts) * s->B * s->H * s->Nq * (size_t(s->d) + 2) * sizeof(float);
    return STREAMKL_OK;
}

struct AttnBwdPlan {
    int ctas, num_q_tiles, num_k_tiles, group, splits, sms;
    size_t row_bytes, key_bytes, part_bytes, ws_bytes;
};

streamkl_status plan_attn_bwd(const streamkl_attn* s, const streamkl_options* opt, AttnBwdPlan* pl) {
    streamkl_status st = check_desc(s, true);
    if (st != STREAMKL_OK) return st;
    if (!options_ok(opt)) return STREAMKL_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != STREAMKL_OK) return st;
    pl->sms = sms;
    pl->num_q_tiles = (s->Nq - 1) / 64 + 1;
    pl->num_k_tiles = (s->Nk - 1) / kBlockK + 1;
    const int64_t key_heads = int64_t(s->B) * s->H_kv, ctas = key_heads * pl->num_k_tiles;
    const int64_t iterations = int64_t(pl->num_q_tiles) * (s->H / s->H_kv);
    // the iterations of a CTA are counted in 32 bits; the prepare kernel has a block per query tile and head
    if (ctas > INT32_MAX || int64_t(s->B) * s->H * pl->num_q_tiles > INT32_MAX || iterations > INT32_MAX)
        return STREAMKL_ERR_UNSUPPORTED;
    // The rule of the score gradients (see bwd_splits).  Here, us in a graph, 1 split, the chosen number, the best of 1 to 8 where that
    // is another:
    //   4096 rows, 8 heads on 2: causal 444, 143 (5), 134 (4); full 444, 299, 237 (2); window of 256 66, 70, 47 (2); documents 182, 83
    //   1024 rows, 32 on 8: causal 129, 64 (4); full 129, 90, 78 (2); window 45, 49, 37 (2); documents 64, 51, 47 (2)
    //   2 x 2048 rows, 16 on 4: causal 250, 169 (3), 152 (2); full 248, 274; window 68, 94; documents 119, 102
    //   3 x 1001 rows, 12 on 4, d = 64: causal 88, 55 (3); full 97, 77; window 33, 39; documents 58, 47, 45 (2)
    //   4 x 1024 rows, 8 on 8: 1 chosen, and the best under every mask
    // The parts are twice those of the score gradients (dK and dV), and windows want fewer of them.
    pl->splits = opt && opt->num_splits > 0 ? std::min(opt->num_splits, kMaxSplits) : bwd_splits(ctas, iterations, sms);
    if (ctas * pl->splits > INT32_MAX) return STREAMKL_ERR_UNSUPPORTED;
    pl->ctas = static_cast<int>(ctas * pl->splits);
    pl->group = order_group(key_heads, pl->num_k_tiles, sms);
    const size_t heads = size_t(s->B) * s->H;
    pl->row_bytes = (attn_bwd_row_bytes(heads, pl->num_q_tiles) + 255) / 256 * 256;
    pl->key_bytes = (attn_bwd_key_bytes(s->B, pl->num_q_tiles) + 255) / 256 * 256;
    pl->part_bytes = pl->splits > 1 ? 2 * size_t(pl->splits) * key_heads * s->Nk * s->d * sizeof(float) : 0;
    pl->ws_bytes = kStatusBytes + pl->row_bytes + pl->key_bytes + pl->part_bytes + heads * s->Nq * s->d * sizeof(float);
    return STREAMKL_OK;
}

ScoreParams ranges_of(const int32_t* begin, const int32_t* end, const int32_t* offset, int causal) {
    ScoreParams sp{};
    sp.begin = begin;
    sp.end = end;
    sp.offset = offset;
    sp.causal = causal ? 1 : 0;
    return sp;
}

}  // namespace

extern "C" {

streamkl_status streamkl_attn_fwd_plan(const streamkl_attn* desc, const streamkl_options* opt, streamkl_plan* plan) {
    if (!plan) return STREAMKL_ERR_INVALID_ARG;
    AttnFwdPlan pl{};
    streamkl_status st = plan_attn_fwd(desc, opt, &pl);
    if (st != STREAMKL_OK) return st;
    plan->path = 0;
    plan->num_splits = pl.p.num_splits;
    plan->num_ctas = pl.ctas;
    plan->launches = pl.p.parts > 1 ? 2 : 1;
    plan->workspace_bytes = pl.ws_bytes;
    return STREAMKL_OK;
}

streamkl_status streamkl_attn_fwd(const streamkl_attn* desc, const void* Q, const void* K, const void* V,
                                  const int32_t* begin, const int32_t* end, const int32_t* offset, float scale, int causal,
                                  void* O, void* rest, float* LSE, void* workspace, size_t workspace_bytes,
                                  const streamkl_options* opt, streamkl_stream_t stream) {
    streamkl_status st = check_desc(desc, false);
    if (st != STREAMKL_OK) return st;
    const void* need[4] = {Q, K, V, O};
    for (const void* q : need)
        if (!q || !aligned16(q)) return STREAMKL_ERR_INVALID_ARG;
    if (!aligned16(rest) || !LSE || !aligned4(LSE) || !aligned4(begin) || !aligned4(end) || !aligned4(offset))
        return STREAMKL_ERR_INVALID_ARG;
    AttnFwdPlan pl{};
    if ((st = plan_attn_fwd(desc, opt, &pl)) != STREAMKL_OK) return st;
    // without parts only the error word stands in the workspace
    if (workspace ? !aligned16(workspace) || workspace_bytes < pl.ws_bytes : pl.p.parts > 1) return STREAMKL_ERR_WORKSPACE;

    AttnFwdParams& p = pl.p;
    CUtensorMap maps[3];
    const streamkl_attn& s = *desc;
    if (!make_map_strided(&maps[0], Q, s.d, s.Nq, s.H, s.B, used(s.q, s.B, s.H, s.Nq, s.d), p.rows, p.heads) ||
        !make_map_strided(&maps[1], K, s.d, s.Nk, s.H_kv, s.B, used(s.k, s.B, s.H_kv, s.Nk, s.d), kBlockK) ||
        !make_map_strided(&maps[2], V, s.d, s.Nk, s.H_kv, s.B, used(s.v, s.B, s.H_kv, s.Nk, s.d), kBlockK))
        return STREAMKL_ERR_CUDA;
    p.c = resolve_scale(scale, s.d) * kLog2e;
    p.O = O;
    p.o_b = s.o.b;
    p.o_h = s.o.h;
    p.o_n = s.o.n;
    p.rest = rest;
    p.LSE = LSE;
    if (p.parts > 1) {
        p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
        p.part_ml = reinterpret_cast<float2*>(p.part + size_t(p.parts) * s.B * s.H * s.Nq * s.d);
    }
    p.status = static_cast<unsigned int*>(workspace);
    p.wait_ns = static_cast<unsigned long long>(wait_limit(opt));
    p.inject_stall = (opt && (opt->debug_flags & STREAMKL_DEBUG_INJECT_STALL)) ? 1 : 0;
    return launch_attn_fwd(s.d, maps, p, ranges_of(begin, end, offset, causal), pl.ctas,
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? STREAMKL_OK
               : STREAMKL_ERR_CUDA;
}

streamkl_status streamkl_attn_bwd_plan(const streamkl_attn* desc, const streamkl_options* opt, streamkl_plan* plan) {
    if (!plan) return STREAMKL_ERR_INVALID_ARG;
    AttnBwdPlan pl{};
    streamkl_status st = plan_attn_bwd(desc, opt, &pl);
    if (st != STREAMKL_OK) return st;
    plan->path = 2;
    plan->num_splits = pl.splits;
    plan->num_ctas = pl.ctas;
    plan->launches = 3;  // prepare, gradients, finish
    plan->workspace_bytes = pl.ws_bytes;
    return STREAMKL_OK;
}

streamkl_status streamkl_attn_bwd(const streamkl_attn* desc, const void* dO, const void* Q, const void* K, const void* V,
                                  const void* O, const void* rest, const float* LSE, const int32_t* begin,
                                  const int32_t* end, const int32_t* offset, float scale, int causal, void* dQ, void* dK,
                                  void* dV, void* workspace, size_t workspace_bytes, const streamkl_options* opt,
                                  streamkl_stream_t stream) {
    streamkl_status st = check_desc(desc, true);
    if (st != STREAMKL_OK) return st;
    const void* need[8] = {dO, Q, K, V, O, dQ, dK, dV};
    for (const void* q : need)
        if (!q || !aligned16(q)) return STREAMKL_ERR_INVALID_ARG;
    if (!aligned16(rest) || !LSE || !aligned4(LSE) || !aligned4(begin) || !aligned4(end) || !aligned4(offset))
        return STREAMKL_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace)) return STREAMKL_ERR_WORKSPACE;
    AttnBwdPlan pl{};
    if ((st = plan_attn_bwd(desc, opt, &pl)) != STREAMKL_OK) return st;
    if (workspace_bytes < pl.ws_bytes) return STREAMKL_ERR_WORKSPACE;

    const streamkl_attn& s = *desc;
    CUtensorMap maps[4];
    if (!make_map_strided(&maps[0], Q, s.d, s.Nq, s.H, s.B, used(s.q, s.B, s.H, s.Nq, s.d), 64) ||
        !make_map_strided(&maps[1], K, s.d, s.Nk, s.H_kv, s.B, used(s.k, s.B, s.H_kv, s.Nk, s.d), kBlockK) ||
        !make_map_strided(&maps[2], V, s.d, s.Nk, s.H_kv, s.B, used(s.v, s.B, s.H_kv, s.Nk, s.d), kBlockK) ||
        !make_map_strided(&maps[3], dO, s.d, s.Nq, s.H, s.B, used(s.d_o, s.B, s.H, s.Nq, s.d), 64))
        return STREAMKL_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace) + kStatusBytes;
    AttnBwdParams p{};
    p.B = s.B;
    p.H = s.H;
    p.H_kv = s.H_kv;
    p.Nq = s.Nq;
    p.Nk = s.Nk;
    p.group = s.H / s.H_kv;
    p.num_q_tiles = pl.num_q_tiles;
    p.num_k_tiles = pl.num_k_tiles;
    p.num_splits = pl.splits;
    p.order_group = pl.group;
    p.scale = resolve_scale(scale, s.d);
    p.c = p.scale * kLog2e;
    p.K = K;
    p.k_b = s.k.b, p.k_h = s.k.h, p.k_n = s.k.n;
    p.dO = dO;
    p.g_b = s.d_o.b, p.g_h = s.d_o.h, p.g_n = s.d_o.n;
    p.O = O;
    p.o_b = s.o.b, p.o_h = s.o.h, p.o_n = s.o.n;
    p.rest = rest;
    p.LSE = LSE;
    p.dQ = dQ;
    p.dK = dK;
    p.dV = dV;
    p.rows = reinterpret_cast<float*>(ws);
    p.keys = ws + pl.row_bytes;
    p.parts = reinterpret_cast<float*>(ws + pl.row_bytes + pl.key_bytes);
    p.dQacc = reinterpret_cast<float*>(ws + pl.row_bytes + pl.key_bytes + pl.part_bytes);
    p.status = static_cast<unsigned int*>(workspace);
    p.wait_ns = static_cast<unsigned long long>(wait_limit(opt));
    p.inject_stall = (opt && (opt->debug_flags & STREAMKL_DEBUG_INJECT_STALL)) ? 1 : 0;
    return launch_attn_bwd(s.d, maps, p, ranges_of(begin, end, offset, causal), pl.ctas, pl.sms,
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? STREAMKL_OK
               : STREAMKL_ERR_CUDA;
}

}  // extern "C"
