// cache8_attn.cu -- attention of a few new tokens over the 8-bit cache.
//
//   x_ij = log2(e) scale s_K q_i k_j,  O_i = sum_j 2^(x_ij - m_i) s_V v_j / l_i
//
// with k_j, v_j the stored e4m3 values and s_K, s_V the scales of their page.  Every
// key and value byte is read once for the rows (query heads of a key head x new
// tokens) of a tile, and that is the bound: HBM.  The products are small beside it,
// so they run on warp-level f16 MMAs, whose operands are the stored bytes turned to
// f16 (exact) in registers: no wait on another warp.  Keys stand on the MMAs' M side
// in the scores and features in the output, and 8 rows fill their N side: a tile of
// 8 rows takes half the MMAs, exponentials and registers of one of 16.  A row of q is
// f16 after a scaling by a power of two.  Probabilities are f16 with 2^7 more than
// their value, so that they keep all 11 bits down to 2^-21.
//
// Sums of the output stand against a reference of their own, as scales of pages may lie any
// distance apart: a probability has an exponent for l and one for the output.  (Its value for
// l times a factor is as fast with one row tile, and with 32 rows 111 us where this takes
// 113, 8 caches of up to 16384; but the factor leaves float32's range.)
//
// A segment is one sequence's keys of one key head.  Its chunks are dealt out to the
// warps of a CTA, each of which has a ring of its own that TMA fills, 16 tokens of a
// page at a time.  With more than one row tile, teams of warps share the copies.
// Short segments have a cluster of CTAs each, which add up their sums through shared
// memory.  The lengths are known on the device alone: where the table allows long
// ones, every CTA takes the same number of chunks of all segments, one after the
// other, and a second kernel adds up the parts of segments that were cut.
//
// One token, 32 heads on 8, d = 128, 4 sequences of up to 131072 tokens: 164 us, 5.7 TB/s
// (a copy: 6.8): about 20 us are start, ends and the second kernel, the rest runs near
// the copy rate.  Five tokens of 3 sequences of up to 1000: 12.7 us (one CTA a segment:
// 21.5), a chain of latencies.  With two teams (17 to 32 rows) the MMAs and conversions,
// which each team does for itself, are the bound: 6600 cycles for 256 keys, 2.9 TB/s.
#include "bwd_common.cuh"
#include "cache8.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "ptx.cuh"
#include "score.cuh"

namespace streamkl {

namespace {

// Row tiles of 8 NQ rows; chunks of KH halves of 16 keys, each half of one page.  Both
// shapes take 256 keys in a step of the CTA.  16 warps hide the latencies of their
// dependent steps where 8 rows leave the registers for them.
template <int NQ>
struct CacheShape {
    static constexpr int kHalves = NQ == 1 ? 1 : 2;
    static constexpr int kWarps = 16 / kHalves;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRows = 8 * NQ;
    static constexpr int kKeys = 16 * kHalves;
};
constexpr int kCwStages = 3;      // a warp's chunks in its ring: one in use, the others on their way
constexpr float kCwTau = 8.f;     // references may stay this far (log2) below the largest value
constexpr float kCwShift = 7.f;   // probabilities are at most 2^(8 + 7) < 65504
constexpr float kCwNone = -3.4e38f;  // the output's reference where there is none yet: below any score

// 16 rows of d bytes, swizzled so that 8 rows' pieces lie in different banks.
__device__ __forceinline__ void copy_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(bar)
        : "memory");
}

// Byte offset of 16-byte piece `piece` of row `row` under the swizzle of d-byte rows (128: 8 pieces, 64: 4).
template <int D>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    return row * D + ((D == 128 ? piece ^ (row & 7) : piece ^ ((row >> 1) & 3)) << 4);
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

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// A page's value scale as 2^e x f with 1 <= f < 2, so that no factor made of it leaves float32's range.  0 (and
// what is below the normal numbers) has e = -inf and f = 0, what is no number f = NaN.
__device__ __forceinline__ float2 split_scale(float s) {
    const int u = __float_as_int(s);
    if (s >= 1.17549435e-38f && s < INFINITY) return make_float2(static_cast<float>((u >> 23) - 127), __int_as_float((u & 0x7fffff) | 0x3f800000));
    return make_float2(-INFINITY, s > 0.f && s < INFINITY ? 0.f : 0.f * s);
}

// What a half needs of its page.
struct PageEntry {
    int page;  // -1: not there
    float ks, vs;
    int pad;
};

// States of one row merge by their references: m of the probabilities, and how far above it (log2) that of the output's
// sums lies.  (A distance: both are whole numbers, and float32 adds 7 or a scale's exponent to a distance exactly, to a
// score beyond 2^24 not.)
struct CacheState {
    float m, l, up;
};

__device__ __forceinline__ float ratio(float from, float to) { return from == -INFINITY ? 0.f : ex2(from - to); }

__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }

// The distance from another m, not below the state's own.  A state without m has sums of 0, or NaN: its weight is 1.
__device__ __forceinline__ float up_from(float m, float up, float top) { return m == -INFINITY ? -INFINITY : up + (m - top); }

// Chunks of `keys` keys of sequence b.
__device__ __forceinline__ int chunks_of(const CacheView& c, int b, int keys) {
    return (min(max(c.lengths[b], 0), c.M * c.T) + keys - 1) / keys;  // a table has up to 2^30 tokens
}

// A warp sums the chunks of all sequences, and of those before b.
__device__ __forceinline__ int64_t sum_chunks(const CacheView& c, int b, int keys, int64_t* before) {
    int64_t all = 0, less = 0;
    for (int k = threadIdx.x & 31; k < c.B; k += 32) {
        const int n = chunks_of(c, k, keys);
        all += n;
        less += k < b ? n : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        less += __shfl_xor_sync(0xffffffffu, less, o);
    }
    *before = less;
    return all;
}

// A CTA's share of `total` chunks: a multiple of what its warps take at a time.
__device__ __forceinline__ int64_t share_of(int64_t total, int ctas, int warps) {
    const int64_t n = (total + ctas - 1) / ctas;
    return max((n + warps - 1) / warps * warps, int64_t(warps));
}

// The 8 x 8 transpose of f16 pairs: lane 4g + t gives (row g, columns 2t, 2t + 1) and gets (row 2t, 2t + 1; column g).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t of_rank(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The row's output from its sums: two factors, one after the other.  `up` is at most 137 (scales up to 2^127) and may be any
// number below, so that its power of two alone may leave float32's range where the output does not.
__device__ __forceinline__ float2 output_factors(const CacheState& s) {
    const float e = s.up - kCwShift, near = fminf(fmaxf(e, -100.f), 100.f);
    return s.up == -INFINITY ? make_float2(0.f / s.l, 1.f) : make_float2(ex2(near) / s.l, ex2(e - near));
}

constexpr int64_t kToOutputs = -1, kToCluster = -2;

// One segment's chunks [c0, c1) for a group of row tiles; the sums go to the outputs, together with those of the
// cluster's other CTAs, or (part >= 0) to that part.
// `uses`: how many steps filled the rings before, to tell the phases of their barriers.  False: a wait gave up, and
// the rows are NaN; nothing is copied in a segment that begins with `alive` false.
template <int D, int NQ, bool SHARED>
__device__ __forceinline__ bool attend(const CacheAttnParams& p, const CUtensorMap* tK, const CUtensorMap* tV, uint8_t* smem, int& uses,
                                       const WaitCtx& wc, bool alive, int b, int hk, int rg, int c0, int c1, int64_t part) {
    using S = CacheShape<NQ>;
    constexpr int W = S::kWarps, KH = S::kHalves, ROWS = S::kRows;
    constexpr int KS = D / 16;                // k-steps of a score
    constexpr int MT = D / 16;                // 16-feature tiles of the output
    constexpr int kHalf = 2 * 16 * D;         // bytes of a half: 16 keys, then 16 values
    constexpr int kStage = KH * kHalf;
    constexpr int VB = D / 8;                 // bytes that a lane reads of a value row
    constexpr int kBlock = S::kThreads;       // halves whose pages are looked up at a time, one per thread
    const CacheView& c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int TW = SHARED ? W / 2 : W;    // warps of a team at most
    const int teams = SHARED ? p.teams : 1, team = SHARED ? warp % teams : 0;
    const int rt = rg * teams + team;
    const int R = p.group * p.Nq;
    const int64_t capacity = static_cast<int64_t>(c.M) * c.T;
    const int given = max(c.lengths[b], 0);
    const int len = static_cast<int>(min(static_cast<int64_t>(given), capacity));

    // the pages of the segment's halves, a block ahead of the copies
    const int count = alive ? c1 - c0 : 0, steps = (count + W - 1) / W;
    const float nan = __int_as_float(0x7fc00000);
    PageEntry* entries = reinterpret_cast<PageEntry*>(smem + W * kCwStages * kStage);  // [2][kBlock]
    auto look_up = [&](int block) {
        PageEntry e{-1, nan, 0.f, 0};
        const int64_t j0 = (static_cast<int64_t>(KH * c0) + block * kBlock + threadIdx.x) * 16;
        if (j0 < len) {
            const int page = c.table[static_cast<int64_t>(b) * c.M + (j0 >> c.log_T)];
            if (page >= 0 && page < c.pages) {  // else: a page that is not there, its scores are NaN
                const int64_t ph = static_cast<int64_t>(page) * c.H_kv + hk;
                e.page = page;
                e.ks = c.scales[0][ph];
                e.vs = c.scales[1][ph];
            }
        }
        return e;
    };
    auto entry_of = [&](int half) { return entries[half % (2 * kBlock)]; };
    const uint32_t ring = smem_u32(smem);
    const uint32_t bars = ring + W * kCwStages * kStage + 2 * kBlock * static_cast<uint32_t>(sizeof(PageEntry));  // [stages][W]
    int fetched = 0;
    // step s: the warp's chunk W s + warp.  Every slot is used in every step, by a copy or by an arrival alone.
    auto fetch = [&](int s) {
        const int chunk = W * s + warp, slot = (uses + s) % kCwStages;
        if (s >= steps) return;
        ++fetched;
        if (lane != 0 || (p.inject_stall && blockIdx.x == 0 && warp == 0 && s == 0)) return;  // the latter a test aid
        uint32_t dst = ring + (slot * W + warp) * kStage;
        const uint32_t bar = bars + 8 * (slot * W + warp);
        int page[KH];
        uint32_t bytes = 0;
#pragma unroll
        for (int half = 0; half < KH; ++half) {
            page[half] = chunk < count ? entry_of(KH * chunk + half).page : -1;
            bytes += page[half] >= 0 ? kHalf : 0;
        }
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int half = 0; half < KH; ++half, dst += kHalf) {
            if (page[half] < 0) continue;
            const int j0 = (c0 + chunk) * S::kKeys + 16 * half, row = (page[half] * c.H_kv + hk) * c.T + (j0 & (c.T - 1));
            copy_rows(dst, tK, bar, row);
            copy_rows(dst + 16 * D, tV, bar, row);
        }
    };
    // the query rows (see below) are on their way while the pages are looked up
    uint32_t q[NQ][KS][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int r = rt * ROWS + 8 * n + g, h = r / p.Nq, i = r - h * p.Nq;
        const uint16_t* row = r < R ? static_cast<const uint16_t*>(p.Q) + b * p.q_b + (hk * p.group + h) * p.q_h + i * p.q_n : nullptr;
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
            const uint4 u = row ? *reinterpret_cast<const uint4*>(row + 64 * (s >> 2) + 16 * t + 4 * (s & 3)) : make_uint4(0u, 0u, 0u, 0u);
            q[n][s][0] = u.x, q[n][s][1] = u.y, q[n][s + 1][0] = u.z, q[n][s + 1][1] = u.w;
        }
    }
    bool ok = alive;
    entries[threadIdx.x] = look_up(0);
    PageEntry ahead = look_up(1);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kCwStages; ++s) fetch(s);

    // Query fragments: lane (g, t) has row g of each 8-row tile.  Any order of d serves a score, if q and k have the
    // same: the lane holds the 16-byte pieces t (and t + 4, d = 128) of a row, four values of one piece to a k-step.
    float qf[NQ][2];   // of rows 2t and 2t + 1 of a tile, the lane's columns of a score: its factor
    int lim[NQ][2];    // and the keys below lim are seen
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t a = q[n][s][e] & 0x7fff7fffu;
                top = __vmaxu2(top, a & ~__vcmpgeu2(a, 0x7f807f80u));
            }
        }
        int most = max(top & 0xffffu, top >> 16);
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const int e = max((most >> 7) - 127, -100);  // the row's largest magnitude is below 2^(e + 1)
        const float up = __int_as_float((10 - e + 127) << 23);  // brings it to [2^10, 2^11): f16 takes every bit of the row's larger values
        const float down = p.scale_log2e * __int_as_float((e - 10 + 127) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int x = 0; x < 2; ++x)
                q[n][s][x] = pack_f16(__uint_as_float(q[n][s][x] << 16) * up, __uint_as_float(q[n][s][x] & 0xffff0000u) * up);
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
            const int x = 2 * t + e2, rx = rt * ROWS + 8 * n + x;
            qf[n][e2] = __shfl_sync(0xffffffffu, down, 4 * x);
            lim[n][e2] = rx < R ? len - p.Nq + 1 + rx % p.Nq : 0;
        }
    }

    float o[NQ][MT][4];
    float m[NQ][2], up[NQ][2], l[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int x = 0; x < MT; ++x) o[n][x][0] = o[n][x][1] = o[n][x][2] = o[n][x][3] = 0.f;
        m[n][0] = m[n][1] = -INFINITY, up[n][0] = up[n][1] = kCwNone;
        l[n][0] = l[n][1] = 0.f;
    }
    const int all = len - p.Nq + 1;  // keys that every row sees
    // the segment's chunk, in the ring at `at`
    auto take = [&](int chunk, uint32_t at) {
        float ks[KH], lv[KH];
        float2 scale[KH];
        float s[KH][NQ][4];  // (key g, rows 2t, 2t + 1), (key g + 8, the same)
#pragma unroll
        for (int half = 0; half < KH; ++half) {
            const PageEntry en = entry_of(KH * chunk + half);
            ks[half] = en.ks;
            scale[half] = split_scale(en.vs);
            lv[half] = fmaxf(scale[half].x, -1e29f) + 1.f;  // log2 of a bound of the scale
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[half][n][0] = s[half][n][1] = s[half][n][2] = s[half][n][3] = 0.f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                uint32_t u[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u[j][0]), "=r"(u[j][1]), "=r"(u[j][2]), "=r"(u[j][3]) : "r"(at + half * kHalf + piece_at<D>(8 * j + g, 4 * h + t)) : "memory");
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t a[4] = {f16x2_of_e4m3x2(u[0][e] & 0xffffu), f16x2_of_e4m3x2(u[1][e] & 0xffffu),
                                           f16x2_of_e4m3x2(u[0][e] >> 16), f16x2_of_e4m3x2(u[1][e] >> 16)};
#pragma unroll
                    for (int n = 0; n < NQ; ++n) mma_f16(s[half][n], a, q[n][4 * h + e]);
                }
            }
        }
        const int j0 = (c0 + chunk) * S::kKeys;
#pragma unroll
        for (int half = 0; half < KH; ++half)
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[half][n][e] = s[half][n][e] * qf[n][e & 1] * ks[half];  // qf ks may be infinite where the score is 0
        if (j0 + S::kKeys > all) {
#pragma unroll
            for (int half = 0; half < KH; ++half)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j0 + 16 * half + 8 * (e >> 1) + g >= lim[n][e & 1]) s[half][n][e] = -INFINITY;
        }
        // scores against m from here on (without one yet, as they are: up is kCwNone then, and any score raises)
        bool raise = false;
#pragma unroll
        for (int half = 0; half < KH; ++half)
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ref = reference(m[n][e]);
                    s[half][n][e] -= ref;
                    s[half][n][2 + e] -= ref;
                    const float top = fmaxf(s[half][n][e], s[half][n][2 + e]);
                    raise |= top > kCwTau || top + lv[half] > up[n][e] + kCwTau;
                }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float tm = fmaxf(s[0][n][e], s[0][n][2 + e]);
                    if (KH == 2) tm = fmaxf(tm, fmaxf(s[KH - 1][n][e], s[KH - 1][n][2 + e]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, x));
                    if (tm > (m[n][e] == -INFINITY ? -INFINITY : kCwTau)) {
                        const float ref = reference(m[n][e]), next = ref + ceilf(tm), by = next - ref;
                        l[n][e] *= ratio(m[n][e], next);
                        if (m[n][e] != -INFINITY) up[n][e] -= by;
#pragma unroll
                        for (int half = 0; half < KH; ++half) s[half][n][e] -= by, s[half][n][2 + e] -= by;
                        m[n][e] = next;
                    }
                    float tw = fmaxf(s[0][n][e], s[0][n][2 + e]) + lv[0];
                    if (KH == 2) tw = fmaxf(tw, fmaxf(s[KH - 1][n][e], s[KH - 1][n][2 + e]) + lv[KH - 1]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) tw = fmaxf(tw, __shfl_xor_sync(0xffffffffu, tw, x));
                    if (tw > up[n][e] + kCwTau) {
                        const float next = ceilf(tw), f = ex2(up[n][e] - next);
#pragma unroll
                        for (int x = 0; x < MT; ++x) o[n][x][e] *= f, o[n][x][2 + e] *= f;
                        up[n][e] = next;
                    }
                }
        }
#pragma unroll
        for (int half = 0; half < KH; ++half) {
            const int h0 = j0 + 16 * half;
            const bool tail = h0 + 16 > all;  // some row does not see all of these keys
            uint32_t pr[NQ][2];  // (keys 2t, 2t + 1 and 2t + 8, 2t + 9; row g)
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[n][e] += ex2(s[half][n][e]) + ex2(s[half][n][2 + e]);
                    // In the output's units a probability has an exponent of its own.  (As a factor of the one against m it may
                    // be infinite: the largest score may stand in pages of so small a scale that others, far behind, weigh more.)
                    const float by = kCwShift + scale[half].x - up[n][e];
                    v[e] = scale[half].y * ex2(s[half][n][e] + by);
                    v[2 + e] = scale[half].y * ex2(s[half][n][2 + e] + by);
                }
                if (tail) {  // a scale that is no number must not reach rows that do not see its page
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (h0 + 8 * (e >> 1) + g >= lim[n][e & 1]) v[e] = 0.f;
                }
                pr[n][0] = transpose8(pack_f16(v[0], v[1]));
                pr[n][1] = transpose8(pack_f16(v[2], v[3]));
            }
            // values: lane (g, t) has bytes VB g .. of keys 2t, 2t + 1, 2t + 8, 2t + 9; output tile x has bytes 2x, 2x + 1
            uint32_t v[4][VB / 4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int key = 2 * t + (x & 1) + 8 * (x >> 1);
                const uint32_t src = at + half * kHalf + 16 * D + (VB == 16 ? piece_at<D>(key, g) : piece_at<D>(key, g >> 1) + 8 * (g & 1));
                if (VB == 16)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[x][0]), "=r"(v[x][1]), "=r"(v[x][VB / 4 - 2]), "=r"(v[x][VB / 4 - 1]) : "r"(src) : "memory");
                else
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[x][0]), "=r"(v[x][1]) : "r"(src) : "memory");
            }
            if (tail) {
                // A probability of 0 does not hide a NaN (e4m3 has no infinity): keys that not every row sees and that have
                // one become zeros, as what stands behind the tokens does, and the rows that see them NaN.
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int mine = h0 + 2 * t + (x & 1) + 8 * (x >> 1);
                    uint32_t found = 0u;
#pragma unroll
                    for (int e = 0; e < VB / 4; ++e) found |= __vcmpeq4(v[x][e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    const uint32_t lanes = __ballot_sync(0xffffffffu, found != 0u && mine >= all && mine < len);
                    if (mine >= len || (lanes >> t & 0x11111111u)) {
#pragma unroll
                        for (int e = 0; e < VB / 4; ++e) v[x][e] = 0u;
                    }
                    if (lanes == 0u) continue;
#pragma unroll 1
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if ((lanes >> k & 0x11111111u) && h0 + 2 * k + (x & 1) + 8 * (x >> 1) < lim[n][e]) {
#pragma unroll
                                    for (int y = 0; y < MT; ++y) o[n][y][e] = o[n][y][2 + e] = nan;
                                }
                }
            }
#pragma unroll
            for (int e = 0; e < VB / 4; ++e)
#pragma unroll
                for (int pair = 0; pair < 2; ++pair) {
                    const uint32_t sel = pair ? 0x7362u : 0x5140u;  // bytes (2 pair, 2 pair + 1) of both keys
                    const uint32_t x = __byte_perm(v[0][e], v[1][e], sel), y = __byte_perm(v[2][e], v[3][e], sel);
                    const uint32_t a[4] = {f16x2_of_e4m3x2(x & 0xffffu), f16x2_of_e4m3x2(x >> 16), f16x2_of_e4m3x2(y & 0xffffu),
                                           f16x2_of_e4m3x2(y >> 16)};
#pragma unroll
                    for (int n = 0; n < NQ; ++n) mma_f16(o[n][2 * e + pair], a, pr[n]);
                }
        }
    };
    constexpr int kBlockSteps = kBlock / (KH * W);
    for (int s = 0; s < steps; ++s) {
        if (s % kBlockSteps == 0) {  // the next block's pages replace those of the block before this one
            const int block = s / kBlockSteps;
            __syncthreads();
            entries[(block + 1) % 2 * kBlock + threadIdx.x] = ahead;
            __syncthreads();
            ahead = look_up(block + 2);
        }
        // the step before is done with: its slot takes the copy of the last step of the ring
        if (SHARED)
            __syncthreads();
        else
            __syncwarp();
        if (ok && s > 0) fetch(s + kCwStages - 1);
        const int slot = (uses + s) % kCwStages, phase = (uses + s) / kCwStages & 1;
        const uint32_t slots = ring + slot * W * kStage, full = bars + 8 * slot * W;
        if (SHARED) {
#pragma unroll 1
            for (int j = warp / teams; j < W; j += W / teams) {
                const int chunk = W * s + j;
                ok = ok && wait_all(full + 8 * j, phase, wc, kErrWaitK);
                if (ok && chunk < count) take(chunk, slots + j * kStage);
            }
        } else {
            ok = ok && wait_all(full + 8 * warp, phase, wc, kErrWaitK);
            if (ok && W * s + warp < count) take(W * s + warp, slots + warp * kStage);
        }
    }
    uses += steps;
    ok = __syncthreads_and(ok);
    if (!ok) {
        for (int s = max(0, fetched - kCwStages); s < fetched; ++s)  // the warp's copies land before the CTA ends
            drain_wait_b(bars + 8 * ((uses - steps + s) % kCwStages * W + warp), (uses - steps + s) / kCwStages & 1, kDrainNs);
#pragma unroll
        for (int n = 0; n < NQ; ++n) l[n][0] = l[n][1] = nan;
        __syncthreads();
    }

    // the states and sums of a team's warps meet in shared memory (the ring is done with)
    float* sums = reinterpret_cast<float*>(smem);                      // [warps][ROWS][D]
    float* states = sums + W * ROWS * D;                               // [warps][3][ROWS]
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
            const int row = 8 * n + 2 * t + e;
            if (g == 0) {
                states[(warp * 3) * ROWS + row] = m[n][e];
                states[(warp * 3 + 1) * ROWS + row] = l[n][e];
                states[(warp * 3 + 2) * ROWS + row] = up[n][e];
            }
            float* dst = sums + (warp * ROWS + row) * D + VB * g;  // tile x: d = VB g + 2x, + 1
#pragma unroll
            for (int x = 0; x < MT; x += 2)
                *reinterpret_cast<float4*>(dst + 2 * x) = make_float4(o[n][x][e], o[n][x][2 + e], o[n][x + 1][e], o[n][x + 1][2 + e]);
        }
    __syncthreads();
    // the rows' references, and what each warp's sums are worth against them
    float* merged = states + 3 * W * ROWS;                             // [3][teams x ROWS]
    float* outbox = merged + 3 * W * ROWS;                             // [teams x ROWS][D], [teams x ROWS][4]
    auto store = [&](int r, int d0, const CacheState& st, const float4& v) {
        const int h = hk * p.group + r / p.Nq, i = r % p.Nq;
        const bool empty = len - p.Nq + 1 + i <= 0;
        const float2 f = output_factors(st);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + b * p.o_b + h * p.o_h + i * p.o_n + d0) =
            empty ? make_uint2(0u, 0u) : make_uint2(pack_bf16(v.x * f.x * f.y, v.y * f.x * f.y), pack_bf16(v.z * f.x * f.y, v.w * f.x * f.y));
        if (d0 == 0) p.LSE[(static_cast<size_t>(b) * p.H + h) * p.Nq + i] = empty ? -INFINITY : fmaf(st.m, kLn2, logf(st.l));
    };
    for (int x = threadIdx.x; x < teams * ROWS; x += S::kThreads) {
        const int row = x % ROWS, tm = x / ROWS;
        CacheState st{-INFINITY, 0.f, -INFINITY}, in[TW];
#pragma unroll
        for (int k = 0; k < TW; ++k) {
            const float* at = states + (tm + k * teams) * 3 * ROWS + row;
            in[k] = tm + k * teams < W ? CacheState{at[0], at[ROWS], at[2 * ROWS]} : CacheState{-INFINITY, 0.f, -INFINITY};
            st.m = fmaxf(st.m, in[k].m);
        }
#pragma unroll
        for (int k = 0; k < TW; ++k) {
            in[k].up = up_from(in[k].m, in[k].up, st.m);
            st.up = fmaxf(st.up, in[k].up);
            st.l += in[k].m == -INFINITY ? in[k].l : in[k].l * ex2(in[k].m - st.m);
        }
#pragma unroll
        for (int k = 0; k < TW; ++k)
            if (tm + k * teams < W) states[((tm + k * teams) * 3 + 2) * ROWS + row] = in[k].m == -INFINITY ? 1.f : ex2(in[k].up - st.up);
        merged[x] = st.m, merged[teams * ROWS + x] = st.l, merged[2 * teams * ROWS + x] = st.up;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < teams * ROWS * (D / 4); x += S::kThreads) {
        const int line = x / (D / 4), d0 = (x % (D / 4)) * 4, row = line % ROWS, tm = line / ROWS, r = (rg * teams + tm) * ROWS + row;
        if (r >= R) continue;
        CacheState st{merged[line], merged[teams * ROWS + line], merged[2 * teams * ROWS + line]};
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int y = tm; y < W; y += teams) {
            const float f = states[(y * 3 + 2) * ROWS + row];
            const float4 u = *reinterpret_cast<const float4*>(sums + (y * ROWS + row) * D + d0);
            v.x = fmaf(u.x, f, v.x), v.y = fmaf(u.y, f, v.y), v.z = fmaf(u.z, f, v.z), v.w = fmaf(u.w, f, v.w);
        }
        if (given > capacity) st.l = nan;  // tokens that the table has no page for
        if (part == kToCluster) {
            *reinterpret_cast<float4*>(outbox + line * D + d0) = v;
            if (d0 == 0) *reinterpret_cast<float4*>(outbox + teams * ROWS * D + 4 * line) = make_float4(st.m, st.l, st.up, 0.f);
            continue;
        }
        if (part >= 0) {
            const int64_t at = part * (ROWS * teams) + line;
            *reinterpret_cast<float4*>(p.part + at * D + d0) = v;
            if (d0 == 0) p.part_state[at] = make_float4(st.m, st.l, st.up, 0.f);
            continue;
        }
        store(r, d0, st, v);
    }
    if (part == kToCluster) {  // the sums of the cluster's CTAs, each of which writes some of the rows
        cluster_sync();
        const uint32_t box = smem_u32(outbox);
        const int rank = blockIdx.x & (p.cluster - 1);  // a power of two
        for (int x = rank * S::kThreads + threadIdx.x; x < teams * ROWS * (D / 4); x += p.cluster * S::kThreads) {
            const int line = x / (D / 4), d0 = (x % (D / 4)) * 4, r = rg * teams * ROWS + line;
            if (r >= R) continue;
            CacheState st{-INFINITY, 0.f, -INFINITY};
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            CacheState in[8];
            float4 u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                in[k] = CacheState{-INFINITY, 0.f, -INFINITY};
                u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < p.cluster) {
                    const float4 s = ld_cluster(of_rank(box + 4 * (teams * ROWS * D + 4 * line), k));
                    in[k] = CacheState{s.x, s.y, s.z};
                    u[k] = ld_cluster(of_rank(box + 4 * (line * D + d0), k));
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) st.m = fmaxf(st.m, in[k].m);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                in[k].up = up_from(in[k].m, in[k].up, st.m);
                st.up = fmaxf(st.up, in[k].up);
                st.l += in[k].m == -INFINITY ? in[k].l : in[k].l * ex2(in[k].m - st.m);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float f = in[k].m == -INFINITY ? 1.f : ex2(in[k].up - st.up);
                v.x = fmaf(u[k].x, f, v.x), v.y = fmaf(u[k].y, f, v.y), v.z = fmaf(u[k].z, f, v.z), v.w = fmaf(u[k].w, f, v.w);
            }
            store(r, d0, st, v);
        }
        cluster_sync();  // the others read this CTA's shared memory
    }
    fence_proxy_async_smem();  // the ring may be filled again
    __syncthreads();
    return ok;
}

}  // namespace

template <int D, int NQ, bool SHARED>
__global__ void __launch_bounds__(CacheShape<NQ>::kThreads, 1)
    cache8_attn_kernel(const __grid_constant__ CUtensorMap tK, const __grid_constant__ CUtensorMap tV,
                       const __grid_constant__ CacheAttnParams p) {
    using S = CacheShape<NQ>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ int abort_word;
    const CacheView& c = p.c;
    const uint32_t bars = smem_u32(smem) + S::kWarps * kCwStages * 2 * S::kKeys * D + 2 * S::kThreads * static_cast<uint32_t>(sizeof(PageEntry));
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tK);
        prefetch_tensormap(&tV);
        for (int k = 0; k < kCwStages * S::kWarps; ++k) mbar_init(bars + 8 * k, 1);
        abort_word = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    const WaitCtx wc{&abort_word, p.status, p.wait_ns};
    int uses = 0;
    bool alive = true;
    const int per_b = c.H_kv * p.row_groups;  // segments of a sequence
    if (!p.spread) {
        const int cluster = p.cluster, segment = static_cast<unsigned>(blockIdx.x) >> (__ffs(cluster) - 1), rank = blockIdx.x & (cluster - 1);
        const int b = segment / per_b, s = segment - b * per_b, hk = p.row_groups == 1 ? s : s / p.row_groups;
        const int n = chunks_of(c, b, S::kKeys);  // below 2^26
        const int share = (((n + S::kWarps - 1) / S::kWarps + cluster - 1) >> (__ffs(cluster) - 1)) * S::kWarps;  // whole steps
        attend<D, NQ, SHARED>(p, &tK, &tV, smem, uses, wc, alive, b, hk, s - hk * p.row_groups, min(rank * share, n),
                              min((rank + 1) * share, n), cluster > 1 ? kToCluster : kToOutputs);
        return;
    }
    // this CTA's chunks [lo, hi) of all, counted through the segments of one sequence after the other
    int64_t before = 0;
    const int64_t total = sum_chunks(c, 0, S::kKeys, &before) * per_b, share = share_of(total, gridDim.x, S::kWarps);
    const int64_t lo = blockIdx.x * share, hi = min(total, lo + share);
    int64_t at = 0;  // first chunk of sequence b
    for (int b = 0; b < c.B && at < hi; ++b) {
        const int n = chunks_of(c, b, S::kKeys);
        const int64_t end = at + static_cast<int64_t>(n) * per_b;
        if (end > lo && n > 0) {
            for (int s = lo > at ? static_cast<int>((lo - at) / n) : 0; s < per_b; ++s) {
                const int64_t a = at + static_cast<int64_t>(s) * n;  // first chunk of the segment
                if (a >= hi) break;
                const bool whole = a >= lo && a + n <= hi;
                alive = attend<D, NQ, SHARED>(p, &tK, &tV, smem, uses, wc, alive, b, s / p.row_groups, s % p.row_groups,
                                      static_cast<int>(max(lo - a, int64_t(0))), static_cast<int>(min(hi - a, static_cast<int64_t>(n))),
                                      whole ? kToOutputs : 2 * static_cast<int64_t>(blockIdx.x) + (a < lo ? 0 : 1));
            }
        }
        at = end;
    }
}

// One warp per row: the parts of a segment that was cut, brought to the largest
// references; rows of sequences without tokens.
template <int D, int NQ>
__global__ void __launch_bounds__(256) cache8_combine_kernel(const __grid_constant__ CacheAttnParams p, int ctas) {
    constexpr int V = D / 32, ROWS = CacheShape<NQ>::kRows, keys = CacheShape<NQ>::kKeys;
    const CacheView& c = p.c;
    const size_t rows = static_cast<size_t>(c.B) * p.H * p.Nq, row = blockIdx.x * size_t(8) + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int lane = threadIdx.x & 31;
    const int i = static_cast<int>(row % p.Nq), h = static_cast<int>(row / p.Nq % p.H), b = static_cast<int>(row / p.Nq / p.H);
    const int hk = h / p.group, r = (h - hk * p.group) * p.Nq + i, line = r % (ROWS * p.teams), rg = r / (ROWS * p.teams);
    const int per_b = c.H_kv * p.row_groups, n = chunks_of(c, b, keys);
    int64_t before = 0;
    const int64_t total = sum_chunks(c, b, keys, &before) * per_b;
    const int64_t share = share_of(total, ctas, CacheShape<NQ>::kWarps);
    const int64_t a = before * per_b + static_cast<int64_t>(hk * p.row_groups + rg) * n;
    const int first = static_cast<int>(a / share), last = n > 0 ? static_cast<int>((a + n - 1) / share) : first;
    if (n > 0 && first == last) return;  // the segment's CTA has written the row
    CacheState st{-INFINITY, 0.f, -INFINITY};
    auto index = [&](int k) { return (2 * static_cast<int64_t>(k) + (a < k * share ? 0 : 1)) * (ROWS * p.teams) + line; };
    for (int k = first + lane; n > 0 && k <= last; k += 32) st.m = fmaxf(st.m, p.part_state[index(k)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) st.m = fmaxf(st.m, __shfl_xor_sync(0xffffffffu, st.m, o));
    for (int k = first + lane; n > 0 && k <= last; k += 32) {
        const float4 x = p.part_state[index(k)];
        st.up = fmaxf(st.up, up_from(x.x, x.z, st.m));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) st.up = fmaxf(st.up, __shfl_xor_sync(0xffffffffu, st.up, o));
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.f;
    for (int k = first; n > 0 && k <= last; ++k) {
        const float4 x = p.part_state[index(k)];
        st.l += x.x == -INFINITY ? x.y : x.y * ex2(x.x - st.m);
        const float f = x.x == -INFINITY ? 1.f : ex2(up_from(x.x, x.z, st.m) - st.up);
        const float* part = p.part + index(k) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = fmaf(part[e], f, v[e]);
    }
    const bool empty = max(c.lengths[b], 0) - p.Nq + 1 + i <= 0;
    const float2 f = output_factors(st);
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.O) + b * p.o_b + h * p.o_h + i * p.o_n + lane * V);
#pragma unroll
    for (int e = 0; e < V; e += 2) out[e / 2] = empty ? 0u : pack_bf16(v[e] * f.x * f.y, v[e + 1] * f.x * f.y);
    if (lane == 0) p.LSE[row] = empty ? -INFINITY : fmaf(st.m, kLn2, logf(st.l));
}

namespace {
template <int D, int NQ, bool SHARED>
cudaError_t launch_cache8_attn_d(const CUtensorMap* maps, const CacheAttnParams& p, int ctas, cudaStream_t stream) {
    using S = CacheShape<NQ>;
    constexpr int ring = S::kWarps * kCwStages * 2 * S::kKeys * D, merge = S::kWarps * S::kRows * (D + 6) * 4;
    static_assert(merge + S::kRows * kCacheTeams * (D + 4) * 4 <= ring, "the states meet in the ring's space");
    constexpr int bytes = ring + 2 * S::kThreads * static_cast<int>(sizeof(PageEntry)) + 8 * kCwStages * S::kWarps + 1024;
    static_assert(bytes <= 232448, "shared memory");
    auto k = cache8_attn_kernel<D, NQ, SHARED>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(k, bytes, &done);
    if (e != cudaSuccess) return e;
    if (p.cluster > 1) {
        cudaLaunchAttribute shape{};
        shape.id = cudaLaunchAttributeClusterDimension;
        shape.val.clusterDim.x = p.cluster;
        shape.val.clusterDim.y = shape.val.clusterDim.z = 1;
        cudaLaunchConfig_t how{};
        how.gridDim = dim3(ctas);
        how.blockDim = dim3(S::kThreads);
        how.dynamicSmemBytes = bytes;
        how.stream = stream;
        how.attrs = &shape;
        how.numAttrs = 1;
        return cudaLaunchKernelEx(&how, k, maps[0], maps[1], p);
    }
    k<<<ctas, S::kThreads, bytes, stream>>>(maps[0], maps[1], p);
    if ((e = cudaGetLastError()) != cudaSuccess || !p.spread) return e;
    const int64_t rows = int64_t(p.c.B) * p.H * p.Nq;
    cache8_combine_kernel<D, NQ><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(p, ctas);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_cache8_attn_r(const CUtensorMap* maps, const CacheAttnParams& p, int ctas, cudaStream_t stream) {
    return p.tile_rows == 8 ? launch_cache8_attn_d<D, 1, false>(maps, p, ctas, stream)
           : p.teams == 1   ? launch_cache8_attn_d<D, 2, false>(maps, p, ctas, stream)
                            : launch_cache8_attn_d<D, 2, true>(maps, p, ctas, stream);
}
}  // namespace

cudaError_t launch_cache8_attn(const CUtensorMap* maps, const CacheAttnParams& p, int ctas, cudaStream_t stream) {
    return p.c.d == 128 ? launch_cache8_attn_r<128>(maps, p, ctas, stream) : launch_cache8_attn_r<64>(maps, p, ctas, stream);
}

}  // namespace streamkl
