// cache8_attn.cu -- attention of a few new tokens over the 8-bit cache.
//
//   x_ij = log2(e) scale s_K q_i k_j,  O_i = sum_j 2^(x_ij - m_i) s_V v_j / l_i
//
// with k_j, v_j the stored e4m3 values and s_K, s_V the scales of their page.  Every
// key and value byte is read once for the 16 rows (query heads of a key head x new
// tokens) of a tile, and that is the bound: HBM.  The products are small beside it,
// so they run on warp-level f16 MMAs, whose operands are the stored bytes turned to
// f16 (exact) in registers: no pass through shared memory, no wait on another warp.
// A row of q is f16 after a scaling by a power of two.  Probabilities are f16 with
// 2^7 more than their value, so that they keep all 11 bits down to 2^-21.
//
// Warps take the 16-key chunks of a CTA's share in turn, each with a ring of copies
// of its own whose bytes are read by the lane that copied them.
#include <cuda_fp16.h>

#include "bwd_common.cuh"
#include "cache8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "score.cuh"

namespace streamkl {

namespace {

constexpr int kCwWarps = 8;
constexpr int kCwStages = 4;      // chunks in flight per warp
constexpr float kCwTau = 8.f;     // references may stay this far (log2) below the largest value
constexpr float kCwShift = 7.f;   // probabilities are at most 2^(8 + 7) < 65504

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
    const uint32_t n = there ? BYTES : 0;  // the rest is zeros
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t u) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(u)));
    return h;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A page's value scale as 2^e x f with 1 <= f < 2, so that no factor made of it leaves float32's range.  0 (and
// what is below the normal numbers) has e = -inf and f = 0, what is no number f = NaN.
__device__ __forceinline__ float2 split_scale(float s) {
    const int u = __float_as_int(s);
    if (s >= 1.17549435e-38f && s < INFINITY) return make_float2(static_cast<float>((u >> 23) - 127), __int_as_float((u & 0x7fffff) | 0x3f800000));
    return make_float2(-INFINITY, s > 0.f && s < INFINITY ? 0.f : 0.f * s);
}

// States of one row merge by their references: m of the probabilities, w of the output.
struct CacheState {
    float m, l, w;
};

__device__ __forceinline__ float ratio(float from, float to) { return from == -INFINITY ? 0.f : ex2(from - to); }

// The row's output from sums relative to m and w.
__device__ __forceinline__ float output_factor(const CacheState& s) { return s.w == -INFINITY ? 0.f / s.l : ex2(s.w - kCwShift - s.m) / s.l; }

}  // namespace

template <int D>
__global__ void __launch_bounds__(32 * kCwWarps, 1) cache8_attn_kernel(const __grid_constant__ CacheAttnParams p) {
    constexpr int KS = D / 16;                // k-steps of a score
    constexpr int NT = D / 8;                 // 8-column tiles of the output
    constexpr int kStage = 2 * 16 * D;        // bytes of a chunk: 16 keys and values
    constexpr int VB = D / 8;                 // bytes that a lane reads of a value row
    extern __shared__ __align__(128) uint8_t smem[];
    const CacheView& c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rt = blockIdx.x % p.row_tiles, bh = blockIdx.x / p.row_tiles, split = blockIdx.y;
    const int b = bh / c.H_kv, hk = bh - b * c.H_kv;
    const int R = p.group * p.Nq;
    const int64_t capacity = static_cast<int64_t>(c.M) * c.T;
    const int given = max(c.lengths[b], 0);
    const int len = static_cast<int>(min(static_cast<int64_t>(given), capacity));
    // rows g and g + 8 of the tile: keys below lim are seen
    int lim[2];
    const uint16_t* qrow[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = rt * 16 + g + 8 * k, h = r / p.Nq, i = r - h * p.Nq;
        lim[k] = r < R ? len - p.Nq + 1 + i : 0;
        qrow[k] = r < R ? static_cast<const uint16_t*>(p.Q) + b * p.q_b + (hk * p.group + h) * p.q_h + i * p.q_n : nullptr;
    }
    // Query fragments.  Any order of d serves a score, if q and k have the same: lane t holds the 16-byte pieces
    // t (and t + 4, d = 128) of a row, four values of one piece to a k-step.
    uint32_t q[KS][4];
    float qf[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t raw[KS][2];
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const uint2 u = qrow[k] ? *reinterpret_cast<const uint2*>(qrow[k] + 64 * (s >> 2) + 16 * t + 4 * (s & 3)) : make_uint2(0u, 0u);
            raw[s][0] = u.x, raw[s][1] = u.y;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t a = raw[s][e] & 0x7fff7fffu;
                top = __vmaxu2(top, a & ~__vcmpgeu2(a, 0x7f807f80u));
            }
        }
        int most = max(top & 0xffffu, top >> 16);
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const int e = max((most >> 7) - 127, -100);  // the row's largest magnitude is below 2^(e + 1)
        const float up = __int_as_float((10 - e + 127) << 23);  // brings it to [2^10, 2^11): f16 takes every bit of the row's larger values
        qf[k] = p.scale_log2e * __int_as_float((e - 10 + 127) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                q[s][k + 2 * x] = pack_f16(__uint_as_float(raw[s][x] << 16) * up, __uint_as_float(raw[s][x] & 0xffff0000u) * up);
    }

    // this split's share of the chunks, of which the warp takes every kCwWarps-th
    const int chunks = (len + 15) / 16, per = (chunks + p.num_splits - 1) / p.num_splits;
    const int first = split * per + warp, last = min(chunks, split * per + per);
    const int mine = first < last ? (last - first + kCwWarps - 1) / kCwWarps : 0;
    const float nan = __int_as_float(0x7fc00000);
    // lane l knows the page and the scales of the warp's chunks 32 i + l: of this group and the next
    int page[2] = {-1, -1};
    float ks[2] = {nan, nan}, vs[2] = {0.f, 0.f};
    auto look_up = [&](int group, int& pg, float& sk, float& sv) {
        const int k = 32 * group + lane;
        pg = -1, sk = nan, sv = 0.f;
        if (k < mine) {
            const int m = (first + k * kCwWarps) * 16 >> c.log_T;
            pg = c.table[static_cast<int64_t>(b) * c.M + m];
            if (pg >= 0 && pg < c.pages) {
                const int64_t ph = static_cast<int64_t>(pg) * c.H_kv + hk;
                sk = c.scales[0][ph];
                sv = c.scales[1][ph];
            } else {
                pg = -1;  // a page that is not there: its scores are NaN
            }
        }
    };
    const uint32_t ring = smem_u32(smem) + warp * (kCwStages * kStage);
    auto fetch = [&](int k) {  // chunk k of the warp, whose page stands in group k / 32
        const int pg = __shfl_sync(0xffffffffu, (k >> 5) & 1 ? page[1] : page[0], k & 31);
        if (k < mine) {
            const int j0 = (first + k * kCwWarps) * 16, row0 = j0 & (c.T - 1);
            const int64_t at = ((static_cast<int64_t>(max(pg, 0)) * c.H_kv + hk) * c.T + row0) * D;
            const uint8_t* kp = c.values[0] + at;
            const uint8_t* vp = c.values[1] + at;
            uint32_t dst = ring + (k % kCwStages) * kStage + lane * 16;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < D / 64; ++h, dst += 512)
                    copy_async<16>(dst, kp + (8 * j + g) * D + 64 * h + 16 * t, pg >= 0 && j0 + 8 * j + g < len);
            dst = ring + (k % kCwStages) * kStage + 16 * D + lane * VB;
#pragma unroll
            for (int x = 0; x < 4; ++x, dst += 32 * VB) {
                const int j = 2 * t + (x & 1) + 8 * (x >> 1);
                copy_async<VB>(dst, vp + j * D + VB * g, pg >= 0 && j0 + j < len);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(0, page[0], ks[0], vs[0]);
    look_up(1, page[1], ks[1], vs[1]);
#pragma unroll
    for (int k = 0; k < kCwStages - 1; ++k) fetch(k);

    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, w[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const int all = len - p.Nq + 1;  // keys that every row sees
    for (int k = 0; k < mine; ++k) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kCwStages - 2) : "memory");
        const uint32_t at = ring + (k % kCwStages) * kStage;
        const float sk = __shfl_sync(0xffffffffu, (k >> 5) & 1 ? ks[1] : ks[0], k & 31);
        const float sv = __shfl_sync(0xffffffffu, (k >> 5) & 1 ? vs[1] : vs[0], k & 31);
        const int j0 = (first + k * kCwWarps) * 16;
        float s[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                uint32_t u[4];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(at + (j * (D / 64) + h) * 512 + lane * 16) : "memory");
#pragma unroll
                for (int e = 0; e < 4; ++e) mma_f16(s[j], q[4 * h + e], f16x2_of_e4m3x2(u[e] & 0xffffu), f16x2_of_e4m3x2(u[e] >> 16));
            }
        }
        const float f[2] = {qf[0] * sk, qf[1] * sk};
        const bool masked = j0 + 16 > all;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[j][e] *= f[e >> 1];
                if (masked && j0 + 8 * j + 2 * t + (e & 1) >= lim[e >> 1]) s[j][e] = -INFINITY;
            }
        const float2 scale = split_scale(sv);
        const float lv = scale.x + 1.f;  // log2 of a bound of the scale
        float top[2];
        bool raise = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            top[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            raise |= top[r] > m[r] + kCwTau || top[r] + lv > w[r] + kCwTau;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                if (top[r] > m[r] + kCwTau) {
                    const float next = ceilf(top[r]);
                    l[r] *= ratio(m[r], next);
                    m[r] = next;
                }
                if (top[r] + lv > w[r] + kCwTau) {
                    const float next = ceilf(top[r]) + lv, x = ratio(w[r], next);
#pragma unroll
                    for (int n = 0; n < NT; ++n) o[n][2 * r] *= x, o[n][2 * r + 1] *= x;
                    w[r] = next;
                }
            }
        }
        uint32_t a[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float ref = m[r] == -INFINITY ? 0.f : m[r];
            // a probability's factor in the output's units
            const float x = w[r] == -INFINITY ? 0.f * scale.y : scale.y * ex2(ref - w[r] + kCwShift + fmaxf(scale.x, -256.f));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p0 = ex2(s[j][2 * r] - ref), p1 = ex2(s[j][2 * r + 1] - ref);
                l[r] += p0 + p1;
                a[2 * j + r] = pack_f16(p0 * x, p1 * x);
            }
        }
        // values: lane (g, t) has bytes VB g .. of keys 2t, 2t + 1, 2t + 8, 2t + 9; output tile n is byte n of each
        uint32_t v[4][VB / 4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t src = at + 16 * D + x * 32 * VB + lane * VB;
            if (VB == 16)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[x][0]), "=r"(v[x][1]), "=r"(v[x][VB / 4 - 2]), "=r"(v[x][VB / 4 - 1]) : "r"(src) : "memory");
            else
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[x][0]), "=r"(v[x][1]) : "r"(src) : "memory");
        }
        // into the slot of the chunk before this one
        const int next = k + kCwStages - 1;
        if ((next & 31) == 8 && next > 32) {  // the group behind next's: its pages replace those of the group before
            if ((next >> 5) & 1)
                look_up((next >> 5) + 1, page[0], ks[0], vs[0]);
            else
                look_up((next >> 5) + 1, page[1], ks[1], vs[1]);
        }
        fetch(next);
#pragma unroll
        for (int e = 0; e < VB / 4; ++e)
#pragma unroll
            for (int pair = 0; pair < 2; ++pair) {
                const uint32_t sel = pair ? 0x7362u : 0x5140u;  // bytes (2 pair, 2 pair + 1) of both keys
                const uint32_t x = __byte_perm(v[0][e], v[1][e], sel), y = __byte_perm(v[2][e], v[3][e], sel);
                mma_f16(o[4 * e + 2 * pair], a, f16x2_of_e4m3x2(x & 0xffffu), f16x2_of_e4m3x2(y & 0xffffu));
                mma_f16(o[4 * e + 2 * pair + 1], a, f16x2_of_e4m3x2(x >> 16), f16x2_of_e4m3x2(y >> 16));
            }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // the warps' states and sums meet in shared memory (the rings are done with)
    float* sums = reinterpret_cast<float*>(smem);                      // [warps][16][D]
    float* states = sums + kCwWarps * 16 * D;                          // [warps][3][16]
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        const int row = g + 8 * r;
        if (t == 0) {
            states[(warp * 3) * 16 + row] = m[r];
            states[(warp * 3 + 1) * 16 + row] = l[r];
            states[(warp * 3 + 2) * 16 + row] = w[r];
        }
        float* dst = sums + (warp * 16 + row) * D + 2 * NT * t;  // columns 2t and 2t + 1 of tile n: d = 2 NT t + n, + NT
#pragma unroll
        for (int n = 0; n < NT; n += 4) {
            *reinterpret_cast<float4*>(dst + n) = make_float4(o[n][2 * r], o[n + 1][2 * r], o[n + 2][2 * r], o[n + 3][2 * r]);
            *reinterpret_cast<float4*>(dst + NT + n) =
                make_float4(o[n][2 * r + 1], o[n + 1][2 * r + 1], o[n + 2][2 * r + 1], o[n + 3][2 * r + 1]);
        }
    }
    __syncthreads();
    constexpr int kPer = 16 * D / (32 * kCwWarps);  // values of a row per thread: 16 threads to a row
    const int row = threadIdx.x / 16, d0 = (threadIdx.x % 16) * kPer, r = rt * 16 + row;
    if (r >= R) return;
    CacheState st{-INFINITY, 0.f, -INFINITY};
#pragma unroll
    for (int x = 0; x < kCwWarps; ++x) {
        st.m = fmaxf(st.m, states[(x * 3) * 16 + row]);
        st.w = fmaxf(st.w, states[(x * 3 + 2) * 16 + row]);
    }
    float v[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] = 0.f;
#pragma unroll
    for (int x = 0; x < kCwWarps; ++x) {
        const float mx = states[(x * 3) * 16 + row], lx = states[(x * 3 + 1) * 16 + row], wx = states[(x * 3 + 2) * 16 + row];
        st.l += mx == -INFINITY ? lx : lx * ex2(mx - st.m);  // without a reference: 0, or NaN scores alone
        const float f = wx == -INFINITY ? 1.f : ex2(wx - st.w);
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = fmaf(sums[(x * 16 + row) * D + d0 + e], f, v[e]);
    }
    if (given > capacity) st.l = nan;  // tokens that the table has no page for
    const int h = hk * p.group + r / p.Nq, i = r % p.Nq;
    const size_t flat = (static_cast<size_t>(b) * p.H + h) * p.Nq + i;
    if (p.num_splits > 1) {
        const size_t at = static_cast<size_t>(split) * c.B * p.H * p.Nq + flat;
        float4* dst = reinterpret_cast<float4*>(p.part + at * D + d0);
#pragma unroll
        for (int e = 0; e < kPer; e += 4) dst[e / 4] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        if (d0 == 0) p.part_state[at] = make_float4(st.m, st.l, st.w, 0.f);
        return;
    }
    const bool empty = len - p.Nq + 1 + i <= 0 && given <= capacity;
    const float f = empty ? 0.f : output_factor(st);
    uint16_t* out = static_cast<uint16_t*>(p.O) + b * p.o_b + h * p.o_h + i * p.o_n + d0;
#pragma unroll
    for (int e = 0; e < kPer; e += 4)
        *reinterpret_cast<uint2*>(out + e) = empty ? make_uint2(0u, 0u) : make_uint2(pack_bf16(v[e] * f, v[e + 1] * f), pack_bf16(v[e + 2] * f, v[e + 3] * f));
    if (d0 == 0) p.LSE[flat] = empty ? -INFINITY : fmaf(st.m, kLn2, logf(st.l));
}

// One warp per row: the splits' sums, brought to the largest references.
template <int D>
__global__ void __launch_bounds__(256) cache8_combine_kernel(const __grid_constant__ CacheAttnParams p) {
    constexpr int V = D / 32;
    const size_t R = static_cast<size_t>(p.c.B) * p.H * p.Nq, row = blockIdx.x * size_t(8) + (threadIdx.x >> 5);
    if (row >= R) return;
    const int lane = threadIdx.x & 31;
    const int i = static_cast<int>(row % p.Nq), h = static_cast<int>(row / p.Nq % p.H), b = static_cast<int>(row / p.Nq / p.H);
    CacheState st{-INFINITY, 0.f, -INFINITY};
    for (int s = lane; s < p.num_splits; s += 32) {
        const float4 x = p.part_state[s * R + row];
        st.m = fmaxf(st.m, x.x);
        st.w = fmaxf(st.w, x.z);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        st.m = fmaxf(st.m, __shfl_xor_sync(0xffffffffu, st.m, o));
        st.w = fmaxf(st.w, __shfl_xor_sync(0xffffffffu, st.w, o));
    }
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.f;
    for (int s = 0; s < p.num_splits; ++s) {
        const float4 x = p.part_state[s * R + row];
        st.l += x.x == -INFINITY ? x.y : x.y * ex2(x.x - st.m);
        const float f = x.z == -INFINITY ? 1.f : ex2(x.z - st.w);
        const float* part = p.part + (s * R + row) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = fmaf(part[e], f, v[e]);
    }
    const bool empty = p.c.lengths[b] - p.Nq + 1 + i <= 0;
    const float f = empty ? 0.f : output_factor(st);
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.O) + b * p.o_b + h * p.o_h + i * p.o_n + lane * V);
#pragma unroll
    for (int e = 0; e < V; e += 2) out[e / 2] = empty ? 0u : pack_bf16(v[e] * f, v[e + 1] * f);
    if (lane == 0) p.LSE[row] = empty ? -INFINITY : fmaf(st.m, kLn2, logf(st.l));
}

namespace {
template <int D>
cudaError_t launch_cache8_attn_d(const CacheAttnParams& p, cudaStream_t stream) {
    constexpr int ring = kCwWarps * kCwStages * 2 * 16 * D, merge = (kCwWarps * 16 * D + kCwWarps * 48) * 4;
    constexpr int bytes = ring > merge ? ring : merge;
    auto k = cache8_attn_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k<<<dim3(static_cast<unsigned>(p.c.B) * p.c.H_kv * p.row_tiles, p.num_splits), 32 * kCwWarps, bytes, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess || p.num_splits == 1) return e;
    const int64_t rows = int64_t(p.c.B) * p.H * p.Nq;
    cache8_combine_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_cache8_attn(const CacheAttnParams& p, cudaStream_t stream) {
    return p.c.d == 128 ? launch_cache8_attn_d<128>(p, stream) : launch_cache8_attn_d<64>(p, stream);
}

}  // namespace streamkl
