// api_norm_rope.cu -- C ABI of the query/key norm with rotation: argument
// validation and launches on the caller's stream.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "host.h"
#include "kernels.h"

using namespace streamkl;

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Element strides of a tensor of `heads` heads: multiples of 8 (16-byte rows
// of bf16), zero allowed on axes that are read only (broadcast inputs).  A
// written tensor's rows must not share elements along an axis.
bool strides_ok(const streamkl_strides& s, int B, int heads, int N, int d, bool written) {
    const int64_t st[3] = {s.b, s.h, s.n};
    const int n[3] = {B, heads, N};
    for (int k = 0; k < 3; ++k) {
        if (st[k] < 0 || st[k] % 8 != 0 || st[k] > (int64_t(1) << 38)) return false;
        if (written && n[k] > 1 && st[k] < d) return false;
    }
    return true;
}

// Checks that need no device; `backward` checks the gradients' strides too.
streamkl_status check_desc(const streamkl_norm_rope* s, bool backward) {
    if (!s) return STREAMKL_ERR_INVALID_ARG;
    if (s->B < 1 || s->Hq < 1 || s->Hk < 1 || s->N < 0) return STREAMKL_ERR_INVALID_ARG;
    if (s->d != 64 && s->d != 128) return STREAMKL_ERR_UNSUPPORTED;
    if (s->rot < 0 || s->rot > s->d || s->rot % 8 != 0) return STREAMKL_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f) || s->eps > 1e30f) return STREAMKL_ERR_INVALID_ARG;
    const int flags[4] = {s->interleaved, s->weight_bf16, s->grad_bf16, s->pos_int64};
    for (int v : flags)
        if (v != 0 && v != 1) return STREAMKL_ERR_INVALID_ARG;
    if (s->rot > 0 && s->table_rows < 1) return STREAMKL_ERR_INVALID_ARG;
    if (s->table_rows < 0 || s->table_rows > (int64_t(1) << 40)) return STREAMKL_ERR_INVALID_ARG;
    if (int64_t(s->B) * s->N > (int64_t(1) << 27) || s->Hq > 65536 || s->Hk > 65536) return STREAMKL_ERR_UNSUPPORTED;
    const int64_t groups = (int64_t(s->B) * s->N + 7) / 8;
    if (groups * ((s->Hq + 7) / 8 + (s->Hk + 7) / 8) > INT32_MAX) return STREAMKL_ERR_UNSUPPORTED;
    if (!strides_ok(s->q, s->B, s->Hq, s->N, s->d, false) || !strides_ok(s->k, s->B, s->Hk, s->N, s->d, false) ||
        !strides_ok(s->yq, s->B, s->Hq, s->N, s->d, !backward) || !strides_ok(s->yk, s->B, s->Hk, s->N, s->d, !backward))
        return STREAMKL_ERR_INVALID_ARG;
    if (backward && (!strides_ok(s->dq, s->B, s->Hq, s->N, s->d, true) || !strides_ok(s->dk, s->B, s->Hk, s->N, s->d, true)))
        return STREAMKL_ERR_INVALID_ARG;
    return STREAMKL_OK;
}

NormRopeParams make_params(const streamkl_norm_rope* s, const void* q, const void* k, const void* wq, const void* wk,
                           const float* table, const void* positions) {
    NormRopeParams p{};
    const void* x[2] = {q, k};
    const void* w[2] = {wq, wk};
    const streamkl_strides* xs[2] = {&s->q, &s->k};
    const streamkl_strides* ys[2] = {&s->yq, &s->yk};
    const streamkl_strides* ds[2] = {&s->dq, &s->dk};
    for (int i = 0; i < 2; ++i) {
        NormRopeSide& t = p.side[i];
        t.H = i ? s->Hk : s->Hq;
        t.x = x[i];
        t.w = w[i];
        t.x_b = xs[i]->b, t.x_h = xs[i]->h, t.x_n = xs[i]->n;
        t.y_b = ys[i]->b, t.y_h = ys[i]->h, t.y_n = ys[i]->n;
        t.dx_b = ds[i]->b, t.dx_h = ds[i]->h, t.dx_n = ds[i]->n;
    }
    p.B = s->B;
    p.N = s->N;
    p.Hq = s->Hq;
    p.Hk = s->Hk;
    p.rot = s->rot;
    p.interleaved = s->interleaved != 0;
    p.weight_bf16 = s->weight_bf16 != 0;
    p.grad_bf16 = s->grad_bf16 != 0;
    p.pos_int64 = s->pos_int64 != 0;
    p.eps = s->eps;
    p.table = table;
    p.table_rows = s->table_rows;
    p.positions = positions;
    p.start = s->start;
    return p;
}

// Pointers shared by both directions; weights and positions may be absent.
bool pointers_ok(const streamkl_norm_rope* s, const void* q, const void* k, const void* wq, const void* wk,
                 const float* table, const void* positions) {
    return q && k && aligned16(q) && aligned16(k) && aligned16(wq) && aligned16(wk) && aligned16(table) &&
           (s->rot == 0 || table) && aligned(positions, s->pos_int64 ? 8 : 4);
}

streamkl_status plan_bwd_norm(const streamkl_norm_rope* s, int* ctas_q, int* ctas, size_t* bytes) {
    int sms = 0;
    streamkl_status st = device_sms(&sms);
    if (st != STREAMKL_OK) return st;
    NormRopeParams p{};
    p.B = s->B;
    p.N = s->N;
    p.Hq = s->Hq;
    p.Hk = s->Hk;
    norm_rope_bwd_ctas(p, sms, ctas_q, ctas);
    *bytes = kStatusBytes + size_t(*ctas) * s->d * sizeof(float);
    return STREAMKL_OK;
}

}  // namespace

extern "C" {

streamkl_status streamkl_norm_rope_fwd(const streamkl_norm_rope* desc, const void* q, const void* k, const void* wq,
                                       const void* wk, const float* table, const void* positions, void* yq, void* yk,
                                       streamkl_stream_t stream) {
    streamkl_status st = check_desc(desc, false);
    if (st != STREAMKL_OK) return st;
    if (desc->N == 0) return STREAMKL_OK;
    if (!pointers_ok(desc, q, k, wq, wk, table, positions)) return STREAMKL_ERR_INVALID_ARG;
    if (!yq || !yk || !aligned16(yq) || !aligned16(yk)) return STREAMKL_ERR_INVALID_ARG;
    NormRopeParams p = make_params(desc, q, k, wq, wk, table, positions);
    p.side[0].y = yq;
    p.side[1].y = yk;
    return launch_norm_rope_fwd(desc->d, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? STREAMKL_OK
               : STREAMKL_ERR_CUDA;
}

size_t streamkl_norm_rope_workspace_bytes(const streamkl_norm_rope* desc) {
    int cq = 0, c = 0;
    size_t bytes = 0;
    if (check_desc(desc, true) != STREAMKL_OK || plan_bwd_norm(desc, &cq, &c, &bytes) != STREAMKL_OK) return 0;
    return bytes;
}

streamkl_status streamkl_norm_rope_bwd(const streamkl_norm_rope* desc, const void* dyq, const void* dyk, const void* q,
                                       const void* k, const void* wq, const void* wk, const float* table,
                                       const void* positions, void* dq, void* dk, void* dwq, void* dwk,
                                       void* workspace, size_t workspace_bytes, streamkl_stream_t stream) {
    streamkl_status st = check_desc(desc, true);
    if (st != STREAMKL_OK) return st;
    if ((dwq && !wq) || (dwk && !wk) || !aligned16(dwq) || !aligned16(dwk)) return STREAMKL_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t wbytes = size_t(desc->d) * (desc->weight_bf16 ? 2 : 4);
    if (desc->N == 0) {  // no rows: the weights' gradients are sums of nothing
        if (dwq && cudaMemsetAsync(dwq, 0, wbytes, s) != cudaSuccess) return STREAMKL_ERR_CUDA;
        if (dwk && cudaMemsetAsync(dwk, 0, wbytes, s) != cudaSuccess) return STREAMKL_ERR_CUDA;
        return STREAMKL_OK;
    }
    if (!pointers_ok(desc, q, k, wq, wk, table, positions)) return STREAMKL_ERR_INVALID_ARG;
    const void* ptrs[4] = {dyq, dyk, dq, dk};
    for (const void* v : ptrs)
        if (!v || !aligned16(v)) return STREAMKL_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace)) return STREAMKL_ERR_WORKSPACE;
    int ctas_q = 0, ctas = 0;
    size_t bytes = 0;
    if ((st = plan_bwd_norm(desc, &ctas_q, &ctas, &bytes)) != STREAMKL_OK) return st;
    if (workspace_bytes < bytes) return STREAMKL_ERR_WORKSPACE;
    NormRopeParams p = make_params(desc, q, k, wq, wk, table, positions);
    p.side[0].y = const_cast<void*>(dyq);
    p.side[1].y = const_cast<void*>(dyk);
    p.side[0].dx = dq;
    p.side[1].dx = dk;
    p.side[0].dw = dwq;
    p.side[1].dw = dwk;
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
    p.ctas_q = ctas_q;
    return launch_norm_rope_bwd(desc->d, p, ctas, s) == cudaSuccess ? STREAMKL_OK : STREAMKL_ERR_CUDA;
}

streamkl_status streamkl_rope_table(const double* inv_freq, int64_t rows, int32_t half, float* table,
                                    streamkl_stream_t stream) {
    if (!inv_freq || !table || !aligned(inv_freq, 8) || !aligned16(table)) return STREAMKL_ERR_INVALID_ARG;
    if (rows < 1 || rows > (int64_t(1) << 31) || half < 1 || half > 64) return STREAMKL_ERR_INVALID_ARG;
    int sms = 0;
    streamkl_status st = device_sms(&sms);
    if (st != STREAMKL_OK) return st;
    return launch_rope_table(inv_freq, rows, half, table, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? STREAMKL_OK
               : STREAMKL_ERR_CUDA;
}

}  // extern "C"
