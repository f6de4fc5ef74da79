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
// needs no exchange and the norm a few shuffles.  32 + 8 heads of d = 128: 65536
// tokens forward 220 us (6.2 TB/s), gradient 341 us (6.0 TB/s); 8192 tokens
// forward 31 us (5.5 TB/s: start and end of a short grid).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace streamkl {

namespace {

constexpr int kNrThreads = 256;
constexpr int kNrHeads = 8;                  // heads of one token that a warp takes at a time
// CTAs of the gradient pass per SM, all resident.  Loads in flight of each: 32 KB
// for d = 128 and bf16 gradients, 48 KB for float32 ones, half of it for d = 64.
// 64K tokens of 32 + 8 heads: 2 CTAs 371 us, 3 341 us, 4 (half the heads at a
// time, to fit the registers) 415 us.
constexpr int kNrBwdCtas = 3;
constexpr int kNrTokens = kNrThreads / 32;   // neighbouring tokens of a CTA, one per warp

// A lane's 8 values of a head lie in two groups of 4, at a and b, and are held
// as 4 pairs (f[e], g[e]): f the first members, g the second.  With halves, f is
// group a and g group b; interleaved, the members alternate through both groups.
struct Span {
    int a, b;
    bool turned;  // the lane's values are rotated
    int pair;     // its first pair in the table
};

template <bool INTERLEAVED>
__device__ __forceinline__ Span lane_span(int t, int rot) {
    Span s;
    s.turned = 8 * t < rot;
    s.pair = 4 * t;
    if (s.turned && !INTERLEAVED) {
        s.a = 4 * t;
        s.b = rot / 2 + 4 * t;
    } else {
        s.a = 8 * t;
        s.b = 8 * t + 4;
    }
    return s;
}

struct Pairs {
    float2 f[2], g[2];  // f[0], f[1] | f[2], f[3] and so on: packed float32 arithmetic
};

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// A lane's 8 values as they lie in memory, so that a warp's loads are all issued
// before the first of them is used.
template <bool BF16>
struct Raw {
    uint2 a, b;
    __device__ __forceinline__ void load(const void* pa, const void* pb) {
        a = *static_cast<const uint2*>(pa);
        b = *static_cast<const uint2*>(pb);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint2(0u, 0u); }
    template <bool INTERLEAVED>
    __device__ __forceinline__ Pairs get() const {
        Pairs p;
        if (INTERLEAVED) {
            p.f[0] = make_float2(bf_lo(a.x), bf_lo(a.y));
            p.f[1] = make_float2(bf_lo(b.x), bf_lo(b.y));
            p.g[0] = make_float2(bf_hi(a.x), bf_hi(a.y));
            p.g[1] = make_float2(bf_hi(b.x), bf_hi(b.y));
        } else {
            p.f[0] = make_float2(bf_lo(a.x), bf_hi(a.x));
            p.f[1] = make_float2(bf_lo(a.y), bf_hi(a.y));
            p.g[0] = make_float2(bf_lo(b.x), bf_hi(b.x));
            p.g[1] = make_float2(bf_lo(b.y), bf_hi(b.y));
        }
        return p;
    }
};
template <>
struct Raw<false> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* pa, const void* pb) {
        a = *static_cast<const float4*>(pa);
        b = *static_cast<const float4*>(pb);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    template <bool INTERLEAVED>
    __device__ __forceinline__ Pairs get() const {
        Pairs p;
        if (INTERLEAVED) {
            p.f[0] = make_float2(a.x, a.z);
            p.f[1] = make_float2(b.x, b.z);
            p.g[0] = make_float2(a.y, a.w);
            p.g[1] = make_float2(b.y, b.w);
        } else {
            p.f[0] = make_float2(a.x, a.y);
            p.f[1] = make_float2(a.z, a.w);
            p.g[0] = make_float2(b.x, b.y);
            p.g[1] = make_float2(b.z, b.w);
        }
        return p;
    }
};

template <bool INTERLEAVED>
__device__ __forceinline__ void store_pairs(void* pa, void* pb, const Pairs& p) {
    uint2 a, b;
    if (INTERLEAVED) {
        a = make_uint2(pack_bf16(p.f[0].x, p.g[0].x), pack_bf16(p.f[0].y, p.g[0].y));
        b = make_uint2(pack_bf16(p.f[1].x, p.g[1].x), pack_bf16(p.f[1].y, p.g[1].y));
    } else {
        a = make_uint2(pack_bf16(p.f[0].x, p.f[0].y), pack_bf16(p.f[1].x, p.f[1].y));
        b = make_uint2(pack_bf16(p.g[0].x, p.g[0].y), pack_bf16(p.g[1].x, p.g[1].y));
    }
    *static_cast<uint2*>(pa) = a;
    *static_cast<uint2*>(pb) = b;
}

// Cosines and sines of a lane's 4 pairs; a position outside the table gives NaN.
struct Turn {
    float2 c[2], s[2];
};

__device__ __forceinline__ Turn load_turn(const NormRopeParams& p, const Span& sp, uint32_t token, uint32_t n) {
    Turn t;
    t.c[0] = t.c[1] = make_float2(1.f, 1.f);
    t.s[0] = t.s[1] = make_float2(0.f, 0.f);
    if (!sp.turned) return t;
    const int64_t pos = !p.positions ? p.start + n
                        : p.pos_int64 ? static_cast<const int64_t*>(p.positions)[token]
                                      : static_cast<const int32_t*>(p.positions)[token];
    if (pos < 0 || pos >= p.table_rows) {
        const float nan = __int_as_float(0x7fc00000);
        t.c[0] = t.c[1] = t.s[0] = t.s[1] = make_float2(nan, nan);
        return t;
    }
    const float4* f = reinterpret_cast<const float4*>(p.table + (pos * (p.rot / 2) + sp.pair) * 2);
    const float4 lo = __ldg(f), hi = __ldg(f + 1);
    t.c[0] = make_float2(lo.x, lo.z), t.s[0] = make_float2(lo.y, lo.w);
    t.c[1] = make_float2(hi.x, hi.z), t.s[1] = make_float2(hi.y, hi.w);
    return t;
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <bool INTERLEAVED>
__device__ __forceinline__ Pairs load_weights(const void* w, bool bf16, const Span& sp) {
    if (!w) {
        Pairs p;
        p.f[0] = p.f[1] = p.g[0] = p.g[1] = make_float2(1.f, 1.f);
        return p;
    }
    if (bf16) {
        Raw<true> r;
        r.load(static_cast<const uint16_t*>(w) + sp.a, static_cast<const uint16_t*>(w) + sp.b);
        return r.get<INTERLEAVED>();
    }
    Raw<false> r;
    r.load(static_cast<const float*>(w) + sp.a, static_cast<const float*>(w) + sp.b);
    return r.get<INTERLEAVED>();
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Sum over a lane's 8 products.
__device__ __forceinline__ float dot(const Pairs& a, const Pairs& b) {
    float2 u = mul2(a.f[0], b.f[0]), v = mul2(a.f[1], b.f[1]);
    u = fma2(a.g[0], b.g[0], u);
    v = fma2(a.g[1], b.g[1], v);
    return (u.x + u.y) + (v.x + v.y);
}

__device__ __forceinline__ const char* at_bytes(const void* p, int64_t bytes) { return static_cast<const char*>(p) + bytes; }

}  // namespace

// One CTA: kNrTokens neighbouring tokens x kNrHeads heads of q or of k.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kNrThreads) norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES, STEPS = kNrHeads / ROWS;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = lane % LANES, sub = lane / LANES;
    const uint32_t chunks_q = (p.Hq + kNrHeads - 1) / kNrHeads, chunks = chunks_q + (p.Hk + kNrHeads - 1) / kNrHeads;
    const uint32_t group = blockIdx.x / chunks, chunk = blockIdx.x - group * chunks;
    const uint32_t token = group * kNrTokens + warp;  // B N < 2^28
    if (token >= static_cast<uint32_t>(p.B) * p.N) return;
    const NormRopeSide& s = p.side[chunk >= chunks_q];
    const int h0 = static_cast<int>(chunk - (chunk >= chunks_q ? chunks_q : 0)) * kNrHeads + sub;
    const uint32_t b = token / static_cast<uint32_t>(p.N), n = token - b * p.N;
    const Span sp = lane_span<INTERLEAVED>(t, p.rot);
    const char* xp = at_bytes(s.x, 2 * (b * s.x_b + n * s.x_n + h0 * s.x_h + sp.a));
    char* yp = const_cast<char*>(at_bytes(s.y, 2 * (b * s.y_b + n * s.y_n + h0 * s.y_h + sp.a)));
    const int ab = 2 * (sp.b - sp.a);  // bytes from group a to group b
    const int64_t xs = 2 * ROWS * s.x_h, ys = 2 * ROWS * s.y_h;
    Raw<true> raw[STEPS];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        raw[k].zero();
        if (h0 + k * ROWS < s.H) raw[k].load(xp, xp + ab);
        xp += xs;
    }
    const Turn turn = load_turn(p, sp, token, n);
    const Pairs w = load_weights<INTERLEAVED>(s.w, p.weight_bf16, sp);
    // y_f = r (f (w_f c) - g (w_g s)),  y_g = r (g (w_g c) + f (w_f s))
    float2 fc[2], gs[2], gc[2], fs[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        fc[e] = mul2(w.f[e], turn.c[e]);
        fs[e] = mul2(w.f[e], turn.s[e]);
        gc[e] = mul2(w.g[e], turn.c[e]);
        gs[e] = neg2(mul2(w.g[e], turn.s[e]));
    }
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const Pairs x = raw[k].template get<INTERLEAVED>();
        const float2 r = both(rsqrtf(row_sum<LANES>(dot(x, x)) * (1.f / D) + p.eps));
        Pairs y;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            y.f[e] = mul2(r, fma2(x.f[e], fc[e], mul2(x.g[e], gs[e])));
            y.g[e] = mul2(r, fma2(x.g[e], gc[e], mul2(x.f[e], fs[e])));
        }
        if (h0 + k * ROWS < s.H) store_pairs<INTERLEAVED>(yp, yp + ab, y);
        yp += ys;
    }
}

// Gradient.  CTAs [0, ctas_q) walk the query heads, the others the key heads;
// each sums its rows' part of dw in registers, then over its warps, and writes
// it to part[cta][D].  The order of every sum is fixed.
template <int D, bool INTERLEAVED, bool GRAD_BF16>
__global__ void __launch_bounds__(kNrThreads, kNrBwdCtas) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES, STEPS = kNrHeads / ROWS, GB = GRAD_BF16 ? 2 : 4;
    __shared__ float red[kNrThreads / 32][D];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = lane % LANES, sub = lane / LANES;
    const bool keys = static_cast<int>(blockIdx.x) >= p.ctas_q;
    const NormRopeSide& s = p.side[keys];
    const uint32_t first = keys ? blockIdx.x - p.ctas_q : blockIdx.x;
    const uint32_t step = keys ? gridDim.x - p.ctas_q : p.ctas_q;
    const uint32_t chunks = (s.H + kNrHeads - 1) / kNrHeads;
    const uint32_t tokens = static_cast<uint32_t>(p.B) * p.N;
    const uint32_t items = (tokens + kNrTokens - 1) / kNrTokens * chunks;  // < 2^31, as the forward's CTAs
    const Span sp = lane_span<INTERLEAVED>(t, p.rot);
    const int ab = sp.b - sp.a;
    const Pairs w = load_weights<INTERLEAVED>(s.w, p.weight_bf16, sp);
    Pairs dw;
    dw.f[0] = dw.f[1] = dw.g[0] = dw.g[1] = make_float2(0.f, 0.f);
    for (uint32_t it = first; it < items; it += step) {
        const uint32_t group = it / chunks, token = group * kNrTokens + warp;
        if (token >= tokens) continue;
        const int h0 = static_cast<int>(it - group * chunks) * kNrHeads + sub;
        const uint32_t b = token / static_cast<uint32_t>(p.N), n = token - b * p.N;
        const char* xp = at_bytes(s.x, 2 * (b * s.x_b + n * s.x_n + h0 * s.x_h + sp.a));
        const char* gp = at_bytes(s.y, GB * (b * s.y_b + n * s.y_n + h0 * s.y_h + sp.a));
        char* op = const_cast<char*>(at_bytes(s.dx, 2 * (b * s.dx_b + n * s.dx_n + h0 * s.dx_h + sp.a)));
        const int64_t xs = 2 * ROWS * s.x_h, gs = GB * ROWS * s.y_h, os = 2 * ROWS * s.dx_h;
        Raw<true> rx[STEPS];
        Raw<GRAD_BF16> rg[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            rx[k].zero();
            rg[k].zero();
            if (h0 + k * ROWS < s.H) {
                rx[k].load(xp, xp + 2 * ab);
                rg[k].load(gp, gp + GB * ab);
            }
            xp += xs;
            gp += gs;
        }
        const Turn turn = load_turn(p, sp, token, n);
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const Pairs x = rx[k].template get<INTERLEAVED>(), g = rg[k].template get<INTERLEAVED>();
            Pairs u, wu;
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // u = R^T dy
                u.f[e] = fma2(g.f[e], turn.c[e], mul2(g.g[e], turn.s[e]));
                u.g[e] = fma2(g.g[e], turn.c[e], neg2(mul2(g.f[e], turn.s[e])));
                wu.f[e] = mul2(w.f[e], u.f[e]);
                wu.g[e] = mul2(w.g[e], u.g[e]);
            }
            const float r = rsqrtf(row_sum<LANES>(dot(x, x)) * (1.f / D) + p.eps);
            // dx = r wu - n mean(wu n),  n = x r
            const float m = row_sum<LANES>(dot(wu, x)) * r * (1.f / D);
            const float2 rr = both(r), mm = both(-m * r);
            if (h0 + k * ROWS < s.H) {
                Pairs dx;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 nf = mul2(x.f[e], rr), ng = mul2(x.g[e], rr);
                    dw.f[e] = fma2(u.f[e], nf, dw.f[e]);
                    dw.g[e] = fma2(u.g[e], ng, dw.g[e]);
                    dx.f[e] = fma2(wu.f[e], rr, mul2(nf, mm));
                    dx.g[e] = fma2(wu.g[e], rr, mul2(ng, mm));
                }
                store_pairs<INTERLEAVED>(op, op + 2 * ab, dx);
            }
            op += os;
        }
    }
    if (!s.dw) return;
    // back to the order of memory, then over the lanes that hold the same columns
    float va[4], vb[4];
    if (INTERLEAVED) {
        va[0] = dw.f[0].x, va[1] = dw.g[0].x, va[2] = dw.f[0].y, va[3] = dw.g[0].y;
        vb[0] = dw.f[1].x, vb[1] = dw.g[1].x, vb[2] = dw.f[1].y, vb[3] = dw.g[1].y;
    } else {
        va[0] = dw.f[0].x, va[1] = dw.f[0].y, va[2] = dw.f[1].x, va[3] = dw.f[1].y;
        vb[0] = dw.g[0].x, vb[1] = dw.g[0].y, vb[2] = dw.g[1].x, vb[3] = dw.g[1].y;
    }
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            va[e] += __shfl_xor_sync(0xffffffffu, va[e], o);
            vb[e] += __shfl_xor_sync(0xffffffffu, vb[e], o);
        }
    }
    if (lane < LANES) {
#pragma unroll
        for (int e = 0; e < 4; ++e) red[warp][sp.a + e] = va[e], red[warp][sp.b + e] = vb[e];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += blockDim.x) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kNrThreads / 32; ++k) v += red[k][e];
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
    const int64_t slots = int64_t(sms) * kNrBwdCtas;
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
