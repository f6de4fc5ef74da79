// cache8.cu -- a paged cache of keys and values in 8 bits: new tokens written,
// tokens read back.
//
// Every page and head has one scale for its keys and one for its values, a power
// of two: the smallest 2^e, e >= -100, with all of the page's values within 448 2^e
// (448 is e4m3's largest).  A scale of 2^e costs a floating-point format no bits,
// only range at its small end, and one that grows as tokens arrive moves the stored
// values by a whole number of binades: they keep their bits, but for the least ones
// (below 2^-6 of the scale's unit), which are rounded again.  Scales never shrink
// while a page is being filled.  A NaN or an infinity is stored as NaN and does not
// count towards the scale.
//
// Both passes read each value once and write it once.  4 prompts of up to 4096 tokens, 8
// heads, d = 128, pages of 64: written in 16.5 us, read back in 16.2, 5.0 TB/s; the append
// is bound by its arithmetic (reading for values that are not finite as it goes: 22.2), the
// read by the start and end of a short grid (an index worked out from a flat one: 19.7).
#include <algorithm>

#include "cache8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace streamkl {

namespace {

constexpr int kCaThreads = 256;

__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 cvt_from_e4m3x2(uint32_t u) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(u)));
    float2 r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(r.x), "=f"(r.y) : "r"(h));
    return r;
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// The smallest e >= -100 with a <= 448 2^e; 448 = 1.75 2^8.
__device__ __forceinline__ int scale_exponent(float a) {
    const int u = __float_as_int(a), k = (u >> 23) - 127;
    return max((u & 0x7fffff) <= 0x600000 ? k - 8 : k - 7, kCacheLeastExponent);
}

// 8 bf16 times r as e4m3; what is not finite becomes NaN (CHECK: there may be such values).
template <bool CHECK>
__device__ __forceinline__ uint2 quantize8(uint4 x, float r) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xffff0000u);
        lo = !CHECK || fabsf(lo) < INFINITY ? lo * r : __int_as_float(0x7fc00000);
        hi = !CHECK || fabsf(hi) < INFINITY ? hi * r : __int_as_float(0x7fc00000);
        q[k] = cvt_e4m3x2(lo, hi);
    }
    return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// The block's largest half of `top`.
__device__ __forceinline__ uint32_t block_max(uint32_t top, uint32_t* red) {
    uint32_t most = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kCaThreads / 32; ++k) most = max(most, red[k]);
    return most;
}

__device__ __forceinline__ uint32_t requantize4(uint32_t u, float r) {
    const float2 a = cvt_from_e4m3x2(u & 0xffffu), b = cvt_from_e4m3x2(u >> 16);
    return cvt_e4m3x2(a.x * r, a.y * r) | cvt_e4m3x2(b.x * r, b.y * r) << 16;
}

}  // namespace

// One CTA per (sequence, one of the pages that its new tokens touch; head; keys or
// values).  The tokens stay in registers between the pass that finds the largest
// magnitude and the one that writes.
template <int D>
__global__ void __launch_bounds__(kCaThreads) cache8_append_kernel(const __grid_constant__ CacheAppendParams p, int slots) {
    constexpr int W = D / 8;                       // 8-value vectors of a token
    constexpr int STEPS = 128 * W / kCaThreads;    // of a page of 128 tokens, per thread
    __shared__ uint32_t red[kCaThreads / 32];
    const CacheView& c = p.c;
    const int b = blockIdx.x / slots, slot = blockIdx.x - b * slots, hk = blockIdx.y, kv = blockIdx.z;
    const int64_t len = max(c.lengths[b], 0);
    const int count = p.counts ? min(max(p.counts[b], 0), p.N) : p.N;
    const int64_t m = len / c.T + slot;            // page of the sequence
    if (count == 0 || m >= c.M) return;
    const int64_t t0 = m * c.T;                    // the page's first token; new ones are rows [lo, hi)
    const int lo = static_cast<int>(max(len - t0, int64_t(0))), hi = static_cast<int>(min(len + count - t0, int64_t(c.T)));
    if (lo >= hi) return;
    const int page = c.table[static_cast<int64_t>(b) * c.M + m];
    if (page < 0 || page >= c.pages) return;
    const int64_t ph = static_cast<int64_t>(page) * c.H_kv + hk;
    uint8_t* dst = c.values[kv] + ph * c.T * D;
    float* scale = c.scales[kv] + ph;
    const uint16_t* src = static_cast<const uint16_t*>(p.x[kv]) + b * p.x_b[kv] + hk * p.x_h[kv] + (t0 - len) * p.x_n[kv];
    const float old = lo > 0 ? *scale : 0.f;

    uint4 x[STEPS];
    uint32_t top = 0;  // pairs of magnitudes, as their bits
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const int v = threadIdx.x + k * kCaThreads, row = v / W;
        x[k] = make_uint4(0u, 0u, 0u, 0u);
        if (row >= lo && row < hi) x[k] = __ldg(reinterpret_cast<const uint4*>(src + row * p.x_n[kv] + (v % W) * 8));
    }
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
    }
    uint32_t most = block_max(top, red);
    const bool odd = most >= 0x7f80u;  // there are values that are not finite: they do not count
    if (odd) {
        top = 0;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a = w[e] & 0x7fff7fffu;
                top = __vmaxu2(top, a & ~__vcmpgeu2(a, 0x7f807f80u));
            }
        }
        __syncthreads();
        most = block_max(top, red);
    }
    const float want = power_of_two(scale_exponent(__uint_as_float(most << 16)));
    const float now = lo > 0 ? fmaxf(old, want) : want, r = 1.f / now;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const int v = threadIdx.x + k * kCaThreads, row = v / W;
        if (row >= lo && row < hi) *reinterpret_cast<uint2*>(dst + 8 * v) = odd ? quantize8<true>(x[k], r) : quantize8<false>(x[k], r);
    }
    if (lo > 0 && now != old) {  // the tokens that the page held move to the new scale
        for (int v = threadIdx.x; v < lo * W; v += kCaThreads) {
            uint2* q = reinterpret_cast<uint2*>(dst + 8 * v);
            const uint2 u = *q;
            *q = make_uint2(requantize4(u.x, old * r), requantize4(u.y, old * r));
        }
    }
    if (threadIdx.x == 0 && now != old) *scale = now;
}

// 16 values of a row per thread, of kReadRows rows whose look-ups and loads are under way together.  Rows behind a
// sequence's length are zeros, rows of a page that is not there are NaN.
constexpr int kReadRows = 4;

template <int D>
__global__ void __launch_bounds__(256) cache8_read_kernel(const __grid_constant__ CacheReadParams p) {
    constexpr int W = D / 16, kRows = 256 / W;
    const CacheView& c = p.c;
    const int kv = blockIdx.z, w = threadIdx.x % W;
    const uint32_t n0 = blockIdx.x * (kReadRows * kRows) + threadIdx.x / W;
    for (int64_t bh = blockIdx.y; bh < static_cast<int64_t>(c.B) * c.H_kv; bh += gridDim.y) {
        const int b = static_cast<int>(bh / c.H_kv), hk = static_cast<int>(bh - static_cast<int64_t>(b) * c.H_kv), len = c.lengths[b];
        const int32_t* table = c.table + static_cast<int64_t>(b) * c.M;
        int page[kReadRows];  // -1: not there
        float s[kReadRows];
        uint4 u[kReadRows];
#pragma unroll
        for (int k = 0; k < kReadRows; ++k) {
            const uint32_t n = n0 + k * kRows, m = n >> c.log_T;
            page[k] = static_cast<int64_t>(n) < len && n < static_cast<uint32_t>(p.N) && m < static_cast<uint32_t>(c.M) ? table[m] : -1;
            if (page[k] >= c.pages) page[k] = -1;
        }
#pragma unroll
        for (int k = 0; k < kReadRows; ++k) {
            if (page[k] < 0) continue;
            const int64_t ph = static_cast<int64_t>(page[k]) * c.H_kv + hk;
            s[k] = c.scales[kv][ph];
            u[k] = *reinterpret_cast<const uint4*>(c.values[kv] + (ph * c.T + ((n0 + k * kRows) & (c.T - 1))) * D + 16 * w);
        }
#pragma unroll
        for (int k = 0; k < kReadRows; ++k) {
            const uint32_t n = n0 + k * kRows;
            if (n >= static_cast<uint32_t>(p.N)) break;
            uint32_t out[8];
            if (page[k] >= 0) {
                const uint32_t q[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 a = cvt_from_e4m3x2(q[e] & 0xffffu), d = cvt_from_e4m3x2(q[e] >> 16);
                    out[2 * e] = pack_bf16(a.x * s[k], a.y * s[k]);
                    out[2 * e + 1] = pack_bf16(d.x * s[k], d.y * s[k]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] = static_cast<int64_t>(n) < len ? 0x7fc07fc0u : 0u;
            }
            uint16_t* y = static_cast<uint16_t*>(p.y[kv]) + b * p.y_b[kv] + hk * p.y_h[kv] + n * p.y_n[kv] + 16 * w;
            if ((reinterpret_cast<uintptr_t>(y) & 31u) == 0) {
                st_global_v8(y, out[0], out[1], out[2], out[3], out[4], out[5], out[6], out[7]);
            } else {
                reinterpret_cast<uint4*>(y)[0] = make_uint4(out[0], out[1], out[2], out[3]);
                reinterpret_cast<uint4*>(y)[1] = make_uint4(out[4], out[5], out[6], out[7]);
            }
        }
    }
}

cudaError_t launch_cache8_append(const CacheAppendParams& p, cudaStream_t stream) {
    // a run of N tokens touches this many pages at most
    const int slots = static_cast<int>((static_cast<int64_t>(p.N) + p.c.T - 2) / p.c.T) + 1;
    const dim3 grid(static_cast<unsigned>(p.c.B) * slots, p.c.H_kv, 2);
    if (p.c.d == 128)
        cache8_append_kernel<128><<<grid, kCaThreads, 0, stream>>>(p, slots);
    else
        cache8_append_kernel<64><<<grid, kCaThreads, 0, stream>>>(p, slots);
    return cudaGetLastError();
}

cudaError_t launch_cache8_read(const CacheReadParams& p, cudaStream_t stream) {
    const unsigned rows = kReadRows * 256 / (p.c.d / 16);
    const dim3 grid((static_cast<unsigned>(p.N) + rows - 1) / rows, std::min<int64_t>(int64_t(p.c.B) * p.c.H_kv, 65535), 2);
    if (p.c.d == 128)
        cache8_read_kernel<128><<<grid, 256, 0, stream>>>(p);
    else
        cache8_read_kernel<64><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace streamkl
