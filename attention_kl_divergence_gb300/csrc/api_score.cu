// api_score.cu -- C ABI of the score-modified divergence: argument validation,
// launch planning and launches on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "score.cuh"

using namespace streamkl;

namespace {

// tanh(u)/u in powers of u^2 on |u| <= kTanhNear and |u| <= kTanhMid, through
// the Chebyshev nodes of the interval.
constexpr double kNearCoef[4] = {0.9999999402412298, -0.3333197106742687, 0.1328443122754951, -0.04826890785307327};
constexpr double kMidCoef[8] = {0.9999999523634755,   -0.3333290796692471,    0.1332698583380004,
                                -0.053599467131741484, 0.020784093490706108,  -0.007036776496182169,
                                0.0017139283831984046, -0.0002083194733779128};

bool capped(float cap) { return cap > 0.f; }

// One side's score function.  False: a cap that the float32 polynomials cannot
// carry (scale / cap, raised to the sixth power, would leave float32's range).
bool make_side(float cap, const float* slopes, float scale, ScoreSide* s) {
    *s = ScoreSide{};
    s->slopes = slopes;
    s->c = scale * kLog2e;
    if (!capped(cap)) return true;
    const double r = double(scale) / cap, lim = double(cap) * 1.4426950408889634;
    if (!(r >= 1e-5 && r <= 1e5) || !(lim < 1e30)) return false;
    for (int k = 0; k < 4; ++k) s->near[k] = static_cast<float>(lim * r * kNearCoef[k] * std::pow(r, 2 * k));
    for (int k = 0; k < 8; ++k) s->mid[k] = static_cast<float>(lim * kMidCoef[k]);
    s->z_near = static_cast<float>(kTanhNear / r);
    s->z_mid = static_cast<float>(kTanhMid / r);
    s->ratio = static_cast<float>(r);
    s->lim = static_cast<float>(lim);
    s->inv_lim = static_cast<float>(1.0 / lim);
    return true;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

streamkl_status check_score(const streamkl_score* s) {
    if (!s) return STREAMKL_OK;
    const float caps[2] = {s->cap1, s->cap2};
    for (float c : caps)
        if (std::isnan(c) || std::isinf(c) || c < 0.f) return STREAMKL_ERR_INVALID_ARG;
    const void* ptrs[5] = {s->slopes1, s->slopes2, s->begin, s->end, s->offset};
    for (const void* p : ptrs)
        if (!aligned4(p)) return STREAMKL_ERR_INVALID_ARG;
    return STREAMKL_OK;
}

// Kernel variant and parameters.  The variant is that of the worse side: a side
// that needs running maxima, or no cap, takes the other along (8192 causal rows, 32
// heads: both sides capped at 50 729 us, one of them 773, both at 60 885; plain 511).
streamkl_status make_score(const streamkl_score* s, float scale, int causal, ScoreParams* out, int* mode) {
    *out = ScoreParams{};
    const streamkl_score none{};
    if (!s) s = &none;
    if (!make_side(s->cap1, s->slopes1, scale, &out->side[0]) || !make_side(s->cap2, s->slopes2, scale, &out->side[1]))
        return STREAMKL_ERR_UNSUPPORTED;
    out->begin = s->begin;
    out->end = s->end;
    out->offset = s->offset;
    out->causal = causal ? 1 : 0;
    const bool bias = s->slopes1 || s->slopes2;
    const bool bounded = capped(s->cap1) && capped(s->cap2) && out->side[0].lim <= kBoundedMax &&
                         out->side[1].lim <= kBoundedMax;
    *mode = bias                                        ? kScoreBias
            : !capped(s->cap1) && !capped(s->cap2) ? kScorePlain
            : bounded                              ? kScoreBounded
                                                   : kScoreGeneral;
    return STREAMKL_OK;
}

bool options_ok(const streamkl_options* opt) {
    return !opt || (opt->num_splits >= 0 && (opt->grad_bf16 == 0 || opt->grad_bf16 == 1) && opt->bwd_mode == 0 &&
                    !(opt->debug_flags & ~STREAMKL_DEBUG_INJECT_STALL));
}

// Key splits of the tile forward: those of the unmodified forward where they
// save more than the combine launch costs, about three key tiles (256 x 256 keys,
// 2 heads: 1 split 7.5 us, 2 splits 6.5 + 3.0 us).
int tile_splits(int64_t units, int k_tiles, int sms) {
    const int s = choose_splits(units, k_tiles, sms);
    return (k_tiles + s - 1) / s + 3 < k_tiles ? s : 1;
}

struct ScoreFwdPlan {
    bool decode;
    int heads_per_cta, num_splits, ctas, num_q_tiles, num_k_tiles, group, sms;
    size_t ws_bytes;
};

streamkl_status plan_score_fwd(const streamkl_shape* s, const streamkl_options* opt, ScoreFwdPlan* pl) {
    streamkl_status st = check_shape(s, 0);  // a causal row may see no key here: Nq > Nk is allowed
    if (st != STREAMKL_OK) return st;
    if (!options_ok(opt)) return STREAMKL_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != STREAMKL_OK) return st;
    const int64_t BH = int64_t(s->B) * s->H;
    pl->decode = s->Nq <= kDecodeMaxQ;
    pl->num_q_tiles = pl->decode ? 1 : (s->Nq + kBlockQ - 1) / kBlockQ;
    pl->num_k_tiles = (s->Nk + kBlockK - 1) / kBlockK;
    pl->heads_per_cta = 1;
    if (pl->decode) {  // the largest divisor of the group whose queries fit the 16 columns
        const int group = s->H / kv_heads(s);
        for (int c = group; c > 1; --c)
            if (group % c == 0 && c * s->Nq <= kDecodeMaxQ) {
                pl->heads_per_cta = c;
                break;
            }
    }
    const int64_t units = BH / pl->heads_per_cta * pl->num_q_tiles;
    int splits = opt && opt->num_splits > 0 ? std::min(opt->num_splits, pl->num_k_tiles)
                 : pl->decode               ? decode_splits(units, pl->num_k_tiles, sms)
                                            : tile_splits(units, pl->num_k_tiles, sms);
    if (splits > kMaxSplits) splits = kMaxSplits;
    if (units * splits > INT32_MAX || BH * s->Nq > (int64_t(1) << 38)) return STREAMKL_ERR_UNSUPPORTED;
    pl->num_splits = splits;
    pl->ctas = static_cast<int>(units * splits);
    pl->group = order_group(BH, pl->num_q_tiles, sms);
    pl->sms = sms;
    pl->ws_bytes = kStatusBytes;
    if (splits > 1) pl->ws_bytes += size_t(5) * splits * size_t(BH) * s->Nq * sizeof(float);
    return STREAMKL_OK;
}

struct ScoreBwdPlan {
    int ctas, num_q_tiles, num_k_tiles, group, splits, sms;
    bool bf16;
    size_t row_bytes, key_bytes, part_bytes, ws_bytes;
};

streamkl_status plan_score_bwd(const streamkl_shape* s, int setting, const streamkl_options* opt, ScoreBwdPlan* pl) {
    streamkl_status st = check_shape(s, 0);
    if (st != STREAMKL_OK) return st;
    if ((setting != 1 && setting != 2) || !options_ok(opt)) return STREAMKL_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != STREAMKL_OK) return st;
    pl->num_q_tiles = (s->Nq + 63) / 64;
    pl->num_k_tiles = (s->Nk + kBlockK - 1) / kBlockK;
    const int64_t ctas = int64_t(s->B) * kv_heads(s) * pl->num_k_tiles;
    // the iterations of a CTA are counted in 32 bits; the prepare kernel has a block per query tile and head
    if (ctas > INT32_MAX || int64_t(s->B) * s->H * pl->num_q_tiles > INT32_MAX || int64_t(pl->num_q_tiles) * (s->H / kv_heads(s)) > INT32_MAX)
        return STREAMKL_ERR_UNSUPPORTED;
    pl->sms = sms;
    pl->splits = opt && opt->num_splits > 0
                     ? std::min(opt->num_splits, kMaxSplits)
                     : bwd_splits(ctas, int64_t(pl->num_q_tiles) * (s->H / kv_heads(s)), sms);
    if (ctas * pl->splits > INT32_MAX) return STREAMKL_ERR_UNSUPPORTED;
    pl->ctas = static_cast<int>(ctas * pl->splits);
    pl->group = order_group(int64_t(s->B) * kv_heads(s), pl->num_k_tiles, sms);
    pl->bf16 = opt && opt->grad_bf16 == 1;
    pl->row_bytes = (score_bwd_row_bytes(int64_t(s->B) * s->H, pl->num_q_tiles) + 255) / 256 * 256;
    pl->key_bytes = (score_bwd_key_bytes(s->B, pl->num_q_tiles) + 255) / 256 * 256;
    pl->part_bytes = pl->splits > 1 ? size_t(pl->splits) * s->B * kv_heads(s) * s->Nk * s->d * sizeof(float) : 0;
    pl->ws_bytes = kStatusBytes + pl->row_bytes + pl->key_bytes + pl->part_bytes;
    if (pl->bf16) pl->ws_bytes += size_t(s->B) * s->H * s->Nq * s->d * sizeof(float);
    return STREAMKL_OK;
}

}  // namespace

extern "C" {

streamkl_status streamkl_score_fwd_plan(const streamkl_shape* shape, const streamkl_options* opt, streamkl_plan* plan) {
    if (!plan) return STREAMKL_ERR_INVALID_ARG;
    ScoreFwdPlan pl{};
    streamkl_status st = plan_score_fwd(shape, opt, &pl);
    if (st != STREAMKL_OK) return st;
    plan->path = pl.decode ? 1 : 0;
    plan->num_splits = pl.num_splits;
    plan->num_ctas = pl.ctas;
    plan->launches = pl.num_splits > 1 ? 2 : 1;
    plan->workspace_bytes = pl.ws_bytes;
    return STREAMKL_OK;
}

streamkl_status streamkl_score_fwd(const streamkl_shape* shape, const streamkl_score* score, const void* Q1,
                                   const void* K1, const void* Q2, const void* K2, float scale, int causal, float* KL,
                                   float* LSE1, float* LSE2, void* workspace, size_t workspace_bytes,
                                   const streamkl_options* opt, streamkl_stream_t stream) {
    streamkl_status st = check_shape(shape, 0);
    if (st != STREAMKL_OK) return st;
    if ((st = check_score(score)) != STREAMKL_OK) return st;
    const void* qk[4] = {Q1, K1, Q2, K2};
    for (const void* q : qk)
        if (!q || !aligned16(q)) return STREAMKL_ERR_INVALID_ARG;
    const void* rows[3] = {KL, LSE1, LSE2};
    for (const void* q : rows)
        if (!q || !aligned4(q)) return STREAMKL_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace)) return STREAMKL_ERR_WORKSPACE;
    const float sc = resolve_scale(scale, shape->d);
    ScoreParams sp;
    int mode = 0;
    if ((st = make_score(score, sc, causal, &sp, &mode)) != STREAMKL_OK) return st;
    ScoreFwdPlan pl{};
    if ((st = plan_score_fwd(shape, opt, &pl)) != STREAMKL_OK) return st;
    if (workspace_bytes < pl.ws_bytes) return STREAMKL_ERR_WORKSPACE;

    const int qrows = pl.decode ? shape->Nq : kBlockQ;  // decode: a box is the Nq rows of heads_per_cta heads
    CUtensorMap maps[4];
    if (!make_map(&maps[0], Q1, shape, true, qrows, pl.heads_per_cta) || !make_map(&maps[1], K1, shape, false, kBlockK) ||
        !make_map(&maps[2], Q2, shape, true, qrows, pl.heads_per_cta) || !make_map(&maps[3], K2, shape, false, kBlockK))
        return STREAMKL_ERR_CUDA;
    FwdParams p{};
    p.B = shape->B;
    p.H = shape->H;
    p.Nq = shape->Nq;
    p.Nk = shape->Nk;
    p.num_q_tiles = pl.num_q_tiles;
    p.num_k_tiles = pl.num_k_tiles;
    p.num_splits = pl.num_splits;
    p.kv_group = shape->H / kv_heads(shape);
    p.heads_per_cta = pl.heads_per_cta;
    p.order_group = pl.group;
    p.take_over = pl.ctas > pl.sms ? pl.sms : 0;
    p.scale = mode == kScorePlain ? sc : kLn2;  // unit of the running state: raw products, or log2(e) S
    p.scale_log2e = sc * kLog2e;
    p.KL = KL;
    p.LSE1 = LSE1;
    p.LSE2 = LSE2;
    p.part = pl.num_splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes) : nullptr;
    p.status = static_cast<unsigned int*>(workspace);
    p.wait_ns = static_cast<unsigned long long>(wait_limit(opt));
    p.inject_stall = (opt && (opt->debug_flags & STREAMKL_DEBUG_INJECT_STALL)) ? 1 : 0;
    return launch_score_fwd(shape->d, mode, pl.decode, maps, p, sp, pl.ctas, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? STREAMKL_OK
               : STREAMKL_ERR_CUDA;
}

streamkl_status streamkl_score_bwd_plan(const streamkl_shape* shape, int setting, const streamkl_options* opt,
                                        streamkl_plan* plan) {
    if (!plan) return STREAMKL_ERR_INVALID_ARG;
    ScoreBwdPlan pl{};
    streamkl_status st = plan_score_bwd(shape, setting, opt, &pl);
    if (st != STREAMKL_OK) return st;
    plan->path = 2;
    plan->num_splits = pl.splits;
    plan->num_ctas = pl.ctas;
    plan->launches = pl.bf16 || pl.splits > 1 ? 3 : 2;  // prepare (zeros dQ), gradient kernel (+ finish)
    plan->workspace_bytes = pl.ws_bytes;
    return STREAMKL_OK;
}

streamkl_status streamkl_score_bwd(const streamkl_shape* shape, const streamkl_score* score, int setting,
                                   const float* g, const void* Q1, const void* K1, const void* Q2, const void* K2,
                                   const float* KL, const float* LSE1, const float* LSE2, float scale, int causal,
                                   void* dQ, void* dK, void* workspace, size_t workspace_bytes,
                                   const streamkl_options* opt, streamkl_stream_t stream) {
    streamkl_status st = check_shape(shape, 0);
    if (st != STREAMKL_OK) return st;
    if (setting != 1 && setting != 2) return STREAMKL_ERR_INVALID_ARG;
    if ((st = check_score(score)) != STREAMKL_OK) return st;
    const void* qk[4] = {Q1, K1, Q2, K2};
    for (const void* q : qk)
        if (!q || !aligned16(q)) return STREAMKL_ERR_INVALID_ARG;
    const void* rows[4] = {g, KL, LSE1, LSE2};
    for (const void* q : rows)
        if (!q || !aligned4(q)) return STREAMKL_ERR_INVALID_ARG;
    if (!dQ || !dK || !aligned16(dQ) || !aligned16(dK)) return STREAMKL_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace)) return STREAMKL_ERR_WORKSPACE;
    const float sc = resolve_scale(scale, shape->d);
    ScoreParams sp;
    int mode = 0;
    if ((st = make_score(score, sc, causal, &sp, &mode)) != STREAMKL_OK) return st;
    ScoreBwdPlan pl{};
    if ((st = plan_score_bwd(shape, setting, opt, &pl)) != STREAMKL_OK) return st;
    if (workspace_bytes < pl.ws_bytes) return STREAMKL_ERR_WORKSPACE;

    uint8_t* ws = static_cast<uint8_t*>(workspace);
    sp.rows = reinterpret_cast<float*>(ws + kStatusBytes);
    sp.keys = ws + kStatusBytes + pl.row_bytes;
    sp.dk_parts = reinterpret_cast<float*>(ws + kStatusBytes + pl.row_bytes + pl.key_bytes);
    // Q boxes of 64 rows, K boxes of 128 rows
    CUtensorMap maps[4];
    if (!make_map(&maps[0], Q1, shape, true, 64) || !make_map(&maps[1], K1, shape, false, kBlockK) ||
        !make_map(&maps[2], Q2, shape, true, 64) || !make_map(&maps[3], K2, shape, false, kBlockK))
        return STREAMKL_ERR_CUDA;
    BwdParams p{};
    p.B = shape->B;
    p.H = shape->H;
    p.Nq = shape->Nq;
    p.Nk = shape->Nk;
    p.num_q_tiles = pl.num_q_tiles;
    p.num_k_tiles = pl.num_k_tiles;
    p.H_kv = kv_heads(shape);
    p.kv_group = shape->H / p.H_kv;
    p.num_splits = pl.splits;
    p.order_group = pl.group;
    p.scale = sc;
    p.scale_log2e = sc * kLog2e;
    p.g = g;
    p.KL = KL;
    p.LSE1 = LSE1;
    p.LSE2 = LSE2;
    p.dQ = dQ;
    p.dK = dK;
    p.grad_bf16 = pl.bf16 ? 1 : 0;
    p.dQacc = pl.bf16 ? reinterpret_cast<float*>(ws + kStatusBytes + pl.row_bytes + pl.key_bytes + pl.part_bytes)
                        : static_cast<float*>(dQ);
    p.status = static_cast<unsigned int*>(workspace);
    p.wait_ns = static_cast<unsigned long long>(wait_limit(opt));
    p.inject_stall = (opt && (opt->debug_flags & STREAMKL_DEBUG_INJECT_STALL)) ? 1 : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launch_score_bwd(shape->d, setting, mode, maps, p, sp, pl.ctas, pl.sms, s) == cudaSuccess ? STREAMKL_OK
                                                                                                     : STREAMKL_ERR_CUDA;
}

streamkl_status streamkl_key_ranges(int32_t B, int32_t Nq, int32_t Nk, int causal, int32_t window,
                                    const int32_t* q_lengths, const int32_t* k_lengths, const int32_t* prefix,
                                    const int32_t* docs, int32_t num_bounds, int32_t docs_per_batch, int32_t* begin,
                                    int32_t* end, int32_t* offset, streamkl_stream_t stream) {
    if (B < 1 || Nq < 1 || Nk < 1 || window < 0 || !begin || !end || !offset) return STREAMKL_ERR_INVALID_ARG;
    if (docs ? num_bounds < 2 : num_bounds != 0) return STREAMKL_ERR_INVALID_ARG;
    if (prefix && (window > 0 || docs)) return STREAMKL_ERR_UNSUPPORTED;  // the visible keys would not be one range
    const void* ptrs[7] = {q_lengths, k_lengths, prefix, docs, begin, end, offset};
    for (const void* p : ptrs)
        if (!aligned4(p)) return STREAMKL_ERR_INVALID_ARG;
    if (B > 65535 || Nq > INT32_MAX - 255) return STREAMKL_ERR_UNSUPPORTED;  // the grid, counted in blocks of 256 rows
    KeyRangeParams p{};
    p.B = B;
    p.Nq = Nq;
    p.Nk = Nk;
    p.causal = causal ? 1 : 0;
    p.window = window;
    p.q_lengths = q_lengths;
    p.k_lengths = k_lengths;
    p.prefix = prefix;
    p.docs = docs;
    p.num_docs = num_bounds;
    p.doc_stride = docs_per_batch ? num_bounds : 0;
    p.begin = begin;
    p.end = end;
    p.offset = offset;
    return launch_key_ranges(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? STREAMKL_OK
                                                                                       : STREAMKL_ERR_CUDA;
}

}  // extern "C"
