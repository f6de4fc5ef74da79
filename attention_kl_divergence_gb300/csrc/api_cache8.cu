// api_cache8.cu -- C ABI of the 8-bit cache and the attention over it: argument
// validation, planning and launches on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "cache8.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "score.cuh"

using namespace streamkl;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Element strides of a [B, heads, N, d] bf16 tensor: multiples of 8 (16 bytes);
// an axis with one entry has a stride that is never used.  Rows that are written
// must not overlap; rows that are read may be repeated along an axis (stride 0).
bool strides_ok(const streamkl_strides& s, int B, int heads, int N, int d, bool written) {
    const int64_t st[3] = {s.b, s.h, s.n};
    const int n[3] = {B, heads, N};
    for (int k = 0; k < 3; ++k)
        if (n[k] > 1 && (st[k] < (written ? d : 0) || st[k] % 8 != 0 || st[k] > (int64_t(1) << 38))) return false;
    return true;
}

streamkl_status check_cache(const streamkl_cache8* s) {
    if (!s) return STREAMKL_ERR_INVALID_ARG;
    if (s->pages < 1 || s->H_kv < 1 || s->B < 1 || s->M < 1) return STREAMKL_ERR_INVALID_ARG;
    if (s->d != 64 && s->d != 128) return STREAMKL_ERR_UNSUPPORTED;
    if (s->T != 16 && s->T != 32 && s->T != 64 && s->T != 128) return STREAMKL_ERR_UNSUPPORTED;
    // token positions and the pool's rows are counted in 32 bits, heads in a grid's y
    if (int64_t(s->M) * s->T > (int64_t(1) << 30) || s->H_kv > 65535 || int64_t(s->pages) * s->H_kv > INT32_MAX / s->T)
        return STREAMKL_ERR_UNSUPPORTED;
    return STREAMKL_OK;
}

bool make_view(const streamkl_cache8* s, void* k, void* v, float* k_scale, float* v_scale, const int32_t* table,
               const int32_t* lengths, CacheView* c) {
    if (!k || !v || !aligned16(k) || !aligned16(v)) return false;
    const void* rest[4] = {k_scale, v_scale, table, lengths};
    for (const void* p : rest)
        if (!p || !aligned4(p)) return false;
    *c = CacheView{};
    c->values[0] = static_cast<uint8_t*>(k);
    c->values[1] = static_cast<uint8_t*>(v);
    c->scales[0] = k_scale;
    c->scales[1] = v_scale;
    c->pages = s->pages;
    c->H_kv = s->H_kv;
    c->T = s->T;
    c->d = s->d;
    while ((1 << c->log_T) < s->T) ++c->log_T;
    c->table = table;
    c->lengths = lengths;
    c->B = s->B;
    c->M = s->M;
    return true;
}

struct CacheAttnPlan {
    int tile_rows, row_groups, teams, spread, cluster, ctas;
    size_t ws_bytes;
};

streamkl_status plan_cache_attn(const streamkl_cache8* s, const streamkl_options* opt, CacheAttnPlan* pl) {
    streamkl_status st = check_cache(s);
    if (st != STREAMKL_OK) return st;
    if (s->H < 1 || s->H % s->H_kv != 0 || s->N < 1) return STREAMKL_ERR_INVALID_ARG;
    if (s->N > kDecodeMaxQ || int64_t(s->B) * s->H > (int64_t(1) << 24)) return STREAMKL_ERR_UNSUPPORTED;
    if (!strides_ok(s->x, s->B, s->H, s->N, s->d, false) || !strides_ok(s->y, s->B, s->H, s->N, s->d, true))
        return STREAMKL_ERR_INVALID_ARG;
    if (opt && (opt->num_splits < 0 || opt->bwd_mode != 0 || opt->grad_bf16 != 0 ||
                (opt->debug_flags & ~STREAMKL_DEBUG_INJECT_STALL)))
        return STREAMKL_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != STREAMKL_OK) return st;
    const int64_t rows = int64_t(s->H / s->H_kv) * s->N;
    pl->tile_rows = rows <= 8 ? 8 : 16;
    const int64_t row_tiles = (rows + pl->tile_rows - 1) / pl->tile_rows;
    pl->teams = 1;
    while (pl->teams < row_tiles && pl->teams < kCacheTeams) pl->teams *= 2;
    const int64_t row_groups = (row_tiles + pl->teams - 1) / pl->teams, segments = int64_t(s->B) * s->H_kv * row_groups;
    if (segments > INT32_MAX) return STREAMKL_ERR_UNSUPPORTED;
    pl->row_groups = static_cast<int>(row_groups);
    // A segment's CTAs form a cluster, as many as find room at a time (with this much shared memory no more than about a
    // dozen clusters of 8).  Where that leaves a CTA more than a few steps of 256 keys, for the longest sequence that the
    // table allows, equal shares of all sequences serve better than equal CTAs for unequal ones.  One token, 32 heads on
    // 8, unequal lengths up to 4096 / 8192 / 16384 of 4 sequences: 12.9 / 16.9 / 26.3 us with clusters of 4, 21.4 / 24.1 /
    // 30.3 with equal shares; of 8 sequences: 16.8 / 25.3 / 45.3 with clusters of 2, 24.1 / 29.0 / 45.1.  Eight tokens of
    // 8: 38.0 / 64.7 / 117.6 against 42.5 / 58.8 / 94.7.  Nor are equal shares better for so many sequences that their
    // segments fill the SMs by themselves, from 8 segments an SM on.  One token, 32 heads on 8, sequences of 16384, of up to that, and
    // one of 16384 among ones of 300 (equal shares / whole segments): 152 sequences 602 / 585, 441 / 350, 111 / 77; 76 sequences
    // 306 / 296, 253 / 201, 78 / 76; 20 sequences 96 / 147, 92 / 66, 53 / 76.
    const int64_t capacity = int64_t(s->M) * s->T, steps = (capacity + 255) / 256;
    int cluster = 1;
    while (cluster < 8 && 2 * cluster <= steps && segments * 2 * cluster <= (cluster == 4 ? sms / 2 : sms)) cluster *= 2;
    const bool few = (steps + cluster - 1) / cluster <= (pl->tile_rows == 8 ? 16 : 8);
    const int64_t wanted = opt && opt->num_splits > 0 ? opt->num_splits : !few && segments < 8 * int64_t(sms) ? sms : 0;
    pl->spread = wanted > 0;
    pl->cluster = pl->spread ? 1 : cluster;
    pl->ctas = static_cast<int>(wanted > 0 ? std::min<int64_t>({wanted, segments * steps, int64_t(1) << 20}) : segments * pl->cluster);
    pl->ws_bytes = kStatusBytes;
    if (pl->spread) pl->ws_bytes += size_t(pl->ctas) * 2 * pl->tile_rows * pl->teams * (size_t(s->d) + 4) * sizeof(float);
    return STREAMKL_OK;
}

}  // namespace

extern "C" {

streamkl_status streamkl_cache8_append(const streamkl_cache8* desc, void* k, void* v, float* k_scale, float* v_scale,
                                       const int32_t* table, const int32_t* lengths, const void* new_k, const void* new_v,
                                       const int32_t* counts, streamkl_stream_t stream) {
    streamkl_status st = check_cache(desc);
    if (st != STREAMKL_OK) return st;
    const streamkl_cache8& s = *desc;
    if (s.N < 0 || !strides_ok(s.x, s.B, s.H_kv, s.N, s.d, false) || !strides_ok(s.y, s.B, s.H_kv, s.N, s.d, false))
        return STREAMKL_ERR_INVALID_ARG;
    if (int64_t(s.B) * ((int64_t(s.N) + s.T - 2) / s.T + 1) > INT32_MAX) return STREAMKL_ERR_UNSUPPORTED;
    if (s.N == 0) return STREAMKL_OK;
    CacheAppendParams p{};
    if (!make_view(desc, k, v, k_scale, v_scale, table, lengths, &p.c) || !new_k || !new_v || !aligned16(new_k) ||
        !aligned16(new_v) || !aligned4(counts))
        return STREAMKL_ERR_INVALID_ARG;
    p.x[0] = new_k;
    p.x[1] = new_v;
    p.x_b[0] = s.x.b, p.x_h[0] = s.x.h, p.x_n[0] = s.x.n;
    p.x_b[1] = s.y.b, p.x_h[1] = s.y.h, p.x_n[1] = s.y.n;
    p.N = s.N;
    p.counts = counts;
    return launch_cache8_append(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? STREAMKL_OK : STREAMKL_ERR_CUDA;
}

streamkl_status streamkl_cache8_read(const streamkl_cache8* desc, const void* k, const void* v, const float* k_scale,
                                     const float* v_scale, const int32_t* table, const int32_t* lengths, void* out_k,
                                     void* out_v, streamkl_stream_t stream) {
    streamkl_status st = check_cache(desc);
    if (st != STREAMKL_OK) return st;
    const streamkl_cache8& s = *desc;
    if (s.N < 0 || !strides_ok(s.x, s.B, s.H_kv, s.N, s.d, true) || !strides_ok(s.y, s.B, s.H_kv, s.N, s.d, true))
        return STREAMKL_ERR_INVALID_ARG;
    if (s.N == 0) return STREAMKL_OK;
    CacheReadParams p{};
    if (!make_view(desc, const_cast<void*>(k), const_cast<void*>(v), const_cast<float*>(k_scale), const_cast<float*>(v_scale),
                   table, lengths, &p.c) ||
        !out_k || !out_v || !aligned16(out_k) || !aligned16(out_v))
        return STREAMKL_ERR_INVALID_ARG;
    p.y[0] = out_k;
    p.y[1] = out_v;
    p.y_b[0] = s.x.b, p.y_h[0] = s.x.h, p.y_n[0] = s.x.n;
    p.y_b[1] = s.y.b, p.y_h[1] = s.y.h, p.y_n[1] = s.y.n;
    p.N = s.N;
    return launch_cache8_read(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? STREAMKL_OK : STREAMKL_ERR_CUDA;
}

streamkl_status streamkl_attn_cache8_plan(const streamkl_cache8* desc, const streamkl_options* opt, streamkl_plan* plan) {
    if (!plan) return STREAMKL_ERR_INVALID_ARG;
    CacheAttnPlan pl{};
    streamkl_status st = plan_cache_attn(desc, opt, &pl);
    if (st != STREAMKL_OK) return st;
    plan->path = 1;
    plan->num_splits = pl.spread ? pl.ctas : pl.cluster;
    plan->num_ctas = pl.ctas;
    plan->launches = pl.spread ? 2 : 1;
    plan->workspace_bytes = pl.ws_bytes;
    return STREAMKL_OK;
}

streamkl_status streamkl_attn_cache8(const streamkl_cache8* desc, const void* Q, const void* k, const void* v,
                                     const float* k_scale, const float* v_scale, const int32_t* table,
                                     const int32_t* lengths, float scale, void* O, float* LSE, void* workspace,
                                     size_t workspace_bytes, const streamkl_options* opt, streamkl_stream_t stream) {
    streamkl_status st = check_cache(desc);
    if (st != STREAMKL_OK) return st;
    const streamkl_cache8& s = *desc;
    CacheAttnParams p{};
    if (!make_view(desc, const_cast<void*>(k), const_cast<void*>(v), const_cast<float*>(k_scale), const_cast<float*>(v_scale),
                   table, lengths, &p.c) ||
        !Q || !O || !LSE || !aligned16(Q) || !aligned16(O) || !aligned4(LSE))
        return STREAMKL_ERR_INVALID_ARG;
    CacheAttnPlan pl{};
    if ((st = plan_cache_attn(desc, opt, &pl)) != STREAMKL_OK) return st;
    // where no parts are combined only the error word stands in the workspace
    if (workspace ? !aligned16(workspace) || workspace_bytes < pl.ws_bytes : pl.spread != 0) return STREAMKL_ERR_WORKSPACE;
    p.H = s.H;
    p.Nq = s.N;
    p.group = s.H / s.H_kv;
    p.tile_rows = pl.tile_rows;
    p.row_groups = pl.row_groups;
    p.teams = pl.teams;
    p.spread = pl.spread;
    p.cluster = pl.cluster;
    p.Q = Q;
    p.q_b = s.x.b, p.q_h = s.x.h, p.q_n = s.x.n;
    p.O = O;
    p.o_b = s.y.b, p.o_h = s.y.h, p.o_n = s.y.n;
    p.LSE = LSE;
    p.scale_log2e = resolve_scale(scale, s.d) * kLog2e;
    if (pl.spread) {
        p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
        p.part_state = reinterpret_cast<float4*>(p.part + size_t(pl.ctas) * 2 * pl.tile_rows * pl.teams * s.d);
    }
    p.status = static_cast<unsigned int*>(workspace);
    p.wait_ns = static_cast<unsigned long long>(wait_limit(opt));
    p.inject_stall = (opt && (opt->debug_flags & STREAMKL_DEBUG_INJECT_STALL)) ? 1 : 0;
    CUtensorMap maps[2];
    const int64_t rows = int64_t(s.pages) * s.H_kv * s.T;
    if (!make_map_bytes(&maps[0], k, s.d, rows) || !make_map_bytes(&maps[1], v, s.d, rows)) return STREAMKL_ERR_CUDA;
    return launch_cache8_attn(maps, p, pl.ctas, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? STREAMKL_OK : STREAMKL_ERR_CUDA;
}

}  // extern "C"
