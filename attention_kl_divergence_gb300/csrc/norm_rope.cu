// norm_rope.cu -- the norm of every query and key head and the rotation by its
// position in one pass over the heads, and the gradient of both.
//
//   forward    n = x r,  r = (mean(x^2) + eps)^-1/2,  y = R (w n)
//   backward   u = R^T dy,  dx = r (w u - n mean(w u n)),  dw = sum over rows of u n
//
// R turns the first `rot` values of a head as rot/2 pairs, (e, e + rot/2) or
// (2e, 2e + 1), by the angles whose cosines and sines the table holds for the
// row's position.  Statistics, rotation and the sums of dw are in float32;
// every output is rounded once.
//
// Every element is read and written once and takes a handful of operations, so
// the passes are bound by HBM.  A row is held by d / 8 lanes with 8 values
// each, chosen so that both members of a pair sit in one lane: the rotation
// needs no exchange and the norm a few shuffles.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace streamkl {

namespace {

constexpr int kNrThreads = 256;
constexpr int kNrHeads = 8;                  // heads of one token that a warp takes at a time
constexpr int kNrTokens = kNrThreads / 32;   // neighbouring tokens of a CTA, one per warp

// Offsets of a lane's two groups of 4 values within a head.
struct Span {
    int a, b;
    bool turned;  // the lane's values are rotated
    int pair;     // its first pair
};

__device__ __forceinline__ Span lane_span(int t, int rot, bool interleaved) {
    Span s;
    s.turned = 8 * t < rot;
    s.pair = 4 * t;
    if (s.turned && !interleaved) {
        s.a = 4 * t;
        s.b = rot / 2 + 4 * t;
    } else {
        s.a = 8 * t;
        s.b = 8 * t + 4;
    }
    return s;
}

__device__ __forceinline__ void load4(const void* p, bool bf16, int64_t at, float (&v)[4]) {
    if (bf16) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
        v[0] = __uint_as_float(u.x << 16);
        v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16);
        v[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        v[0] = f.x;
        v[1] = f.y;
        v[2] = f.z;
        v[3] = f.w;
    }
}

// 4 values as they lie in memory, so that a warp's loads can all be issued
// before the first of them is used.
template <bool BF16>
struct Raw4 {
    uint2 u;
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
    }
    __device__ __forceinline__ void zero() { u = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = __uint_as_float(u.x << 16);
        v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16);
        v[3] = __uint_as_float(u.y & 0xffff0000u);
    }
};
template <>
struct Raw4<false> {
    float4 f;
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        f = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    }
    __device__ __forceinline__ void zero() { f = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w; }
};

__device__ __forceinline__ void store4(void* p, int64_t at, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// Cosines and sines of a lane's 4 pairs; a position outside the table gives NaN.
struct Turn {
    float c[4], s[4];
};

__device__ __forceinline__ Turn load_turn(const NormRopeParams& p, const Span& sp, int b, int n) {
    Turn t;
    if (!sp.turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) t.c[e] = 1.f, t.s[e] = 0.f;
        return t;
    }
    const int64_t at = static_cast<int64_t>(b) * p.N + n;
    const int64_t pos = !p.positions ? p.start + n
                        : p.pos_int64 ? static_cast<const int64_t*>(p.positions)[at]
                                      : static_cast<const int32_t*>(p.positions)[at];
    if (pos < 0 || pos >= p.table_rows) {
#pragma unroll
        for (int e = 0; e < 4; ++e) t.c[e] = t.s[e] = __int_as_float(0x7fc00000);
        return t;
    }
    const float4* f = reinterpret_cast<const float4*>(p.table + (pos * (p.rot / 2) + sp.pair) * 2);
    const float4 lo = __ldg(f), hi = __ldg(f + 1);
    t.c[0] = lo.x, t.s[0] = lo.y, t.c[1] = lo.z, t.s[1] = lo.w;
    t.c[2] = hi.x, t.s[2] = hi.y, t.c[3] = hi.z, t.s[3] = hi.w;
    return t;
}

// Turn a lane's pairs by the angles (inverse: by their negatives).
template <bool INVERSE>
__device__ __forceinline__ void rotate(float (&a)[4], float (&b)[4], const Turn& t, bool interleaved) {
    if (interleaved) {  // pairs (a0, a1), (a2, a3), (b0, b1), (b2, b3)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float& x = e < 2 ? a[2 * (e & 1)] : b[2 * (e & 1)];
            float& y = e < 2 ? a[2 * (e & 1) + 1] : b[2 * (e & 1) + 1];
            const float s = INVERSE ? -t.s[e] : t.s[e];
            const float u = x * t.c[e] - y * s, v = y * t.c[e] + x * s;
            x = u;
            y = v;
        }
    } else {  // pairs (a_e, b_e)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float s = INVERSE ? -t.s[e] : t.s[e];
            const float u = a[e] * t.c[e] - b[e] * s, v = b[e] * t.c[e] + a[e] * s;
            a[e] = u;
            b[e] = v;
        }
    }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void load_weights(const void* w, bool bf16, const Span& sp, float (&wa)[4], float (&wb)[4]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 4; ++e) wa[e] = wb[e] = 1.f;
        return;
    }
    load4(w, bf16, sp.a, wa);
    load4(w, bf16, sp.b, wb);
}

}  // namespace

// One CTA: kNrTokens neighbouring tokens x kNrHeads heads of q or of k.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kNrThreads) norm_rope_fwd_kernel(const NormRopeParams p) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = lane % LANES, sub = lane / LANES;
    const int chunks_q = (p.Hq + kNrHeads - 1) / kNrHeads, chunks = chunks_q + (p.Hk + kNrHeads - 1) / kNrHeads;
    const int64_t token = static_cast<int64_t>(blockIdx.x / chunks) * kNrTokens + warp;
    if (token >= static_cast<int64_t>(p.B) * p.N) return;
    const int chunk = blockIdx.x % chunks;
    const NormRopeSide& s = p.side[chunk >= chunks_q];
    const int h0 = (chunk - (chunk >= chunks_q ? chunks_q : 0)) * kNrHeads;
    const int b = static_cast<int>(token / p.N), n = static_cast<int>(token - static_cast<int64_t>(b) * p.N);
    const Span sp = lane_span(t, p.rot, INTERLEAVED);
    const int64_t xin = b * s.x_b + n * s.x_n, yout = b * s.y_b + n * s.y_n;
    constexpr int STEPS = kNrHeads / ROWS;
    Raw4<true> ra[STEPS], rb[STEPS];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const int h = h0 + k * ROWS + sub;
        ra[k].zero();
        rb[k].zero();
        if (h < s.H) {
            ra[k].load(s.x, xin + h * s.x_h + sp.a);
            rb[k].load(s.x, xin + h * s.x_h + sp.b);
        }
    }
    const Turn turn = load_turn(p, sp, b, n);
    float wa[4], wb[4];
    load_weights(s.w, p.weight_bf16, sp, wa, wb);
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const int h = h0 + k * ROWS + sub;
        const bool live = h < s.H;
        float xa[4], xb[4];
        ra[k].get(xa);
        rb[k].get(xb);
        float q = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) q = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], q));
        const float r = rsqrtf(row_sum<LANES>(q) * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) xa[e] = xa[e] * r * wa[e], xb[e] = xb[e] * r * wb[e];
        if (sp.turned) rotate<false>(xa, xb, turn, INTERLEAVED);
        if (live) {
            store4(s.y, yout + h * s.y_h + sp.a, xa);
            store4(s.y, yout + h * s.y_h + sp.b, xb);
        }
    }
}

// Gradient.  CTAs [0, ctas_q) walk the query heads, the others the key heads;
// each sums its rows' part of dw in registers, then over its warps, and writes
// it to part[cta][D].  The order of every sum is fixed.
template <int D, bool INTERLEAVED, bool GRAD_BF16>
__global__ void __launch_bounds__(kNrThreads) norm_rope_bwd_kernel(const NormRopeParams p) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES;
    __shared__ float red[kNrThreads / 32][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = lane % LANES, sub = lane / LANES;
    const bool keys = static_cast<int>(blockIdx.x) >= p.ctas_q;
    const NormRopeSide& s = p.side[keys];
    const int first = keys ? blockIdx.x - p.ctas_q : blockIdx.x;
    const int step = keys ? static_cast<int>(gridDim.x) - p.ctas_q : p.ctas_q;
    const int chunks = (s.H + kNrHeads - 1) / kNrHeads;
    const int64_t tokens = static_cast<int64_t>(p.B) * p.N;
    const int64_t items = (tokens + kNrTokens - 1) / kNrTokens * chunks;
    const Span sp = lane_span(t, p.rot, INTERLEAVED);
    constexpr int STEPS = kNrHeads / ROWS;
    float wa[4], wb[4], da[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};
    load_weights(s.w, p.weight_bf16, sp, wa, wb);
    for (int64_t it = first; it < items; it += step) {
        const int64_t token = it / chunks * kNrTokens + warp;
        if (token >= tokens) continue;
        const int h0 = static_cast<int>(it % chunks) * kNrHeads;
        const int b = static_cast<int>(token / p.N), n = static_cast<int>(token - static_cast<int64_t>(b) * p.N);
        const int64_t xin = b * s.x_b + n * s.x_n, gin = b * s.y_b + n * s.y_n, dout = b * s.dx_b + n * s.dx_n;
        Raw4<true> rxa[STEPS], rxb[STEPS];
        Raw4<GRAD_BF16> rua[STEPS], rub[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const int h = h0 + k * ROWS + sub;
            rxa[k].zero();
            rxb[k].zero();
            rua[k].zero();
            rub[k].zero();
            if (h < s.H) {
                rxa[k].load(s.x, xin + h * s.x_h + sp.a);
                rxb[k].load(s.x, xin + h * s.x_h + sp.b);
                rua[k].load(s.y, gin + h * s.y_h + sp.a);
                rub[k].load(s.y, gin + h * s.y_h + sp.b);
            }
        }
        const Turn turn = load_turn(p, sp, b, n);
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const int h = h0 + k * ROWS + sub;
            const bool live = h < s.H;
            float xa[4], xb[4], ua[4], ub[4];
            rxa[k].get(xa);
            rxb[k].get(xb);
            rua[k].get(ua);
            rub[k].get(ub);
            if (sp.turned) rotate<true>(ua, ub, turn, INTERLEAVED);
            float q = 0.f, m = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                q = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], q));
                m = fmaf(ua[e] * wa[e], xa[e], fmaf(ub[e] * wb[e], xb[e], m));
            }
            const float r = rsqrtf(row_sum<LANES>(q) * (1.f / D) + p.eps);
            const float c = row_sum<LANES>(m) * r * (1.f / D);  // mean(w u n)
            if (live) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float na = xa[e] * r, nb = xb[e] * r;
                    da[e] = fmaf(ua[e], na, da[e]);
                    db[e] = fmaf(ub[e], nb, db[e]);
                    ua[e] = r * (ua[e] * wa[e] - na * c);
                    ub[e] = r * (ub[e] * wb[e] - nb * c);
                }
                store4(s.dx, dout + h * s.dx_h + sp.a, ua);
                store4(s.dx, dout + h * s.dx_h + sp.b, ub);
            }
        }
    }
    if (!s.dw) return;
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            da[e] += __shfl_xor_sync(0xffffffffu, da[e], o);
            db[e] += __shfl_xor_sync(0xffffffffu, db[e], o);
        }
    }
    if (lane < LANES) {
#pragma unroll
        for (int e = 0; e < 4; ++e) red[warp][sp.a + e] = da[e], red[warp][sp.b + e] = db[e];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += blockDim.x) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kNrThreads / 32; ++w) v += red[w][e];
        p.part[static_cast<size_t>(blockIdx.x) * D + e] = v;
    }
}

// dw = the CTAs' parts in a fixed order: block (side, 32 columns), 8 warps
// taking every 8th part.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const NormRopeParams p, int d, int ctas) {
    __shared__ float red[8][32];
    const NormRopeSide& s = p.side[blockIdx.y];
    if (!s.dw) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.x * 32 + lane;
    const int lo = blockIdx.y ? p.ctas_q : 0, hi = blockIdx.y ? ctas : p.ctas_q;
    float v = 0.f;
    for (int c = lo + warp; c < hi; c += 8) v += p.part[static_cast<size_t>(c) * d + e];
    red[warp][lane] = v;
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < 8; ++w) v += red[w][lane];
    if (p.weight_bf16)
        static_cast<uint16_t*>(s.dw)[e] = static_cast<uint16_t>(pack_bf16(v, 0.f) & 0xffffu);
    else
        static_cast<float*>(s.dw)[e] = v;
}

// table[n][e] = (cos, sin) of n * inv_freq[e]: the angle, and its reduction, in 64 bits.
__global__ void __launch_bounds__(256) rope_table_kernel(const double* inv_freq, int64_t rows, int half, float2* table) {
    const int64_t total = rows * half;
    for (int64_t k = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; k < total; k += int64_t(gridDim.x) * blockDim.x) {
        double s, c;
        sincos(static_cast<double>(k / half) * inv_freq[k % half], &s, &c);
        table[k] = make_float2(static_cast<float>(c), static_cast<float>(s));
    }
}

// CTAs of the gradient pass: enough to fill the GPU, no more than there are
// items, shared between q and k by their items (at least one each).
void norm_rope_bwd_ctas(const NormRopeParams& p, int sms, int* ctas_q, int* ctas) {
    const int64_t groups = (int64_t(p.B) * p.N + kNrTokens - 1) / kNrTokens;
    const int64_t iq = groups * ((p.Hq + kNrHeads - 1) / kNrHeads), ik = groups * ((p.Hk + kNrHeads - 1) / kNrHeads);
    const int64_t slots = int64_t(sms) * 4;
    if (iq + ik <= slots) {
        *ctas_q = static_cast<int>(iq);
        *ctas = static_cast<int>(iq + ik);
        return;
    }
    int64_t q = (slots * iq + (iq + ik) / 2) / (iq + ik);
    q = std::min<int64_t>(std::max<int64_t>(q, 1), slots - 1);
    *ctas_q = static_cast<int>(std::min(q, iq));
    *ctas = *ctas_q + static_cast<int>(std::min(slots - q, ik));
}

cudaError_t launch_norm_rope_fwd(int d, const NormRopeParams& p, cudaStream_t stream) {
    const int64_t groups = (int64_t(p.B) * p.N + kNrTokens - 1) / kNrTokens;
    const int64_t ctas = groups * ((p.Hq + kNrHeads - 1) / kNrHeads + (p.Hk + kNrHeads - 1) / kNrHeads);
    const unsigned grid = static_cast<unsigned>(ctas);
    if (d == 128)
        p.interleaved ? norm_rope_fwd_kernel<128, true><<<grid, kNrThreads, 0, stream>>>(p)
                      : norm_rope_fwd_kernel<128, false><<<grid, kNrThreads, 0, stream>>>(p);
    else
        p.interleaved ? norm_rope_fwd_kernel<64, true><<<grid, kNrThreads, 0, stream>>>(p)
                      : norm_rope_fwd_kernel<64, false><<<grid, kNrThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

namespace {
template <int D>
void launch_bwd_d(const NormRopeParams& p, int ctas, cudaStream_t stream) {
    if (p.interleaved)
        p.grad_bf16 ? norm_rope_bwd_kernel<D, true, true><<<ctas, kNrThreads, 0, stream>>>(p)
                    : norm_rope_bwd_kernel<D, true, false><<<ctas, kNrThreads, 0, stream>>>(p);
    else
        p.grad_bf16 ? norm_rope_bwd_kernel<D, false, true><<<ctas, kNrThreads, 0, stream>>>(p)
                    : norm_rope_bwd_kernel<D, false, false><<<ctas, kNrThreads, 0, stream>>>(p);
}
}  // namespace

cudaError_t launch_norm_rope_bwd(int d, const NormRopeParams& p, int ctas, cudaStream_t stream) {
    if (d == 128)
        launch_bwd_d<128>(p, ctas, stream);
    else
        launch_bwd_d<64>(p, ctas, stream);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!p.side[0].dw && !p.side[1].dw)) return e;
    norm_rope_dw_kernel<<<dim3(d / 32, 2), 256, 0, stream>>>(p, d, ctas);
    return cudaGetLastError();
}

cudaError_t launch_rope_table(const double* inv_freq, int64_t rows, int half, float* table, int sms,
                              cudaStream_t stream) {
    const int64_t blocks = std::min<int64_t>((rows * half + 255) / 256, int64_t(sms) * 16);
    rope_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(inv_freq, rows, half,
                                                                        reinterpret_cast<float2*>(table));
    return cudaGetLastError();
}

}  // namespace streamkl
