// score.cuh -- how a raw dot product z = <q, k> becomes a score, and which keys
// a query row sees; shared by the forward and backward kernels of the
// score-modified divergence.
//
//   S = cap tanh(scale z / cap) - slope |i + offset - j|      (cap 0: scale z)
//
// The kernels keep x = log2(e) S, so that a probability is one ex2.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace streamkl {

// What the kernels are compiled for.
//   kScorePlain    no cap, no bias: x = c z, applied inside the exponent's FMA
//   kScoreBounded  both sides capped, |x| <= kBoundedMax: sums of 2^x of any
//                  length fit float32, so no running maximum is needed
//   kScoreGeneral  any caps, no bias, running maxima
//   kScoreBias     any caps and a bias, running maxima
constexpr int kScorePlain = 0, kScoreBounded = 1, kScoreGeneral = 2, kScoreBias = 3;
// 2^x with |x| <= 80: a sum of 2^31 of them is at most 2^111, times a score
// difference (2^8) at most 2^119; the smallest one, 2^-80, is a normal number.
constexpr float kBoundedMax = 80.f;

// tanh(u) / u as a polynomial in u^2 (interpolated at the Chebyshev nodes of
// the interval, so close to the best of its degree):
//   4 terms, |u| <= 0.375: relative error 6e-8
//   8 terms, |u| <= 1.2:   relative error 5e-8
// beyond, 1 - 2 / (1 + e^2u) has no cancellation left to lose bits to.
constexpr float kTanhNear = 0.375f, kTanhMid = 1.2f;

// With r = scale / cap and u = r z.  An uncapped side has lim = 0.
struct ScoreSide {
    float near[4];       // coefficients of z, z^3, z^5, z^7 (lim, r and its powers folded in)
    float mid[8];        // coefficients of u, u^3, ... (lim folded in)
    float z_near, z_mid; // bounds of the polynomials on |z|
    float ratio;         // r
    float lim;           // log2(e) cap
    float inv_lim;       // 1 / lim (0 when uncapped)
    float c;             // log2(e) scale
    const float* slopes; // [H] or null
};

struct ScoreParams {
    ScoreSide side[2];
    const int32_t* begin;   // [B, Nq] or null: 0
    const int32_t* end;     // [B, Nq] or null: Nk
    const int32_t* offset;  // [B] or null: Nk - Nq
    int causal;
    float* rows;            // backward: per-row constants and key ranges of the
    void* keys;             // query tiles (score_bwd.cu)
    float* dk_parts;        // backward: float32 parts of dK, [splits][B*H_kv*Nk, d], when there are several
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Position of query row i of batch b among the keys.
__device__ __forceinline__ int64_t row_position(const ScoreParams& s, int Nq, int Nk, int b, int i) {
    return static_cast<int64_t>(i) + (s.offset ? s.offset[b] : Nk - Nq);
}

// Keys [x, y) that row i sees, inside [0, Nk); (0, 0) for none or a row past the end.
__device__ __forceinline__ int2 row_range(const ScoreParams& s, int Nq, int Nk, int b, int i) {
    if (i >= Nq) return make_int2(0, 0);
    const size_t r = static_cast<size_t>(b) * Nq + i;
    const int lo = s.begin ? max(s.begin[r], 0) : 0;
    int hi = s.end ? min(s.end[r], Nk) : Nk;
    if (s.causal) {
        const int64_t next = row_position(s, Nq, Nk, b, i) + 1;
        hi = static_cast<int>(next < hi ? (next > 0 ? next : 0) : hi);
    }
    return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}

// Unit u of heads x tiles in groups of `group` heads: (head, tile), tiles slow and heads fast in a group.
__device__ __forceinline__ int2 grouped_order(int u, int tiles, int heads, int group) {
    const int g = u / (group * tiles), first = g * group, n = min(group, heads - first);
    const int r = u - first * tiles, t = r / n;
    return make_int2(first + r - t * n, t);
}

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// Any finite z.  An infinite one becomes NaN, as it would without the cap: the
// cap does not hide a broken token.  NaN stays NaN.
__device__ __forceinline__ float score_far(float z, const ScoreSide& s) {
    const float u = z * s.ratio, a = fabsf(u), y = u * u;
    float r = s.mid[7];
#pragma unroll
    for (int k = 6; k >= 0; --k) r = fmaf(r, y, s.mid[k]);
    const float t = fmaf(a, 0.f, s.lim - __fdividef(2.f * s.lim, 1.f + ex2(a * (2.f * kLog2e))));
    return a <= kTanhMid ? u * r : copysignf(t, z);
}

template <int W>
__device__ __forceinline__ float abs_max(const float (&z)[W]) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int e = 0; e < W; e += 4) {
        a = max3f(a, fabsf(z[e]), fabsf(z[e + 1]));
        b = max3f(b, fabsf(z[e + 2]), fabsf(z[e + 3]));
    }
    return fmaxf(a, b);  // NaN is passed over: every form below keeps it NaN
}

template <int W>
__device__ __forceinline__ void cap_near(float (&z)[W], const ScoreSide& s) {
#pragma unroll
    for (int e = 0; e < W; e += 2) {
        const float2 v = make_float2(z[e], z[e + 1]), y = __fmul2_rn(v, v);
        float2 r = __ffma2_rn(splat(s.near[3]), y, splat(s.near[2]));
        r = __ffma2_rn(r, y, splat(s.near[1]));
        r = __ffma2_rn(r, y, splat(s.near[0]));
        const float2 x = __fmul2_rn(v, r);
        z[e] = x.x;
        z[e + 1] = x.y;
    }
}

template <int W>
__device__ __forceinline__ void cap_mid(float (&z)[W], const ScoreSide& s) {
#pragma unroll
    for (int e = 0; e < W; e += 2) {
        const float2 u = __fmul2_rn(make_float2(z[e], z[e + 1]), splat(s.ratio)), y = __fmul2_rn(u, u);
        float2 r = splat(s.mid[7]);
#pragma unroll
        for (int k = 6; k >= 0; --k) r = __ffma2_rn(r, y, splat(s.mid[k]));
        const float2 x = __fmul2_rn(u, r);
        z[e] = x.x;
        z[e + 1] = x.y;
    }
}

// z -> x in place for both sides, without the bias.  A warp takes the shortest
// form that fits every score of its lanes (those with `use`: the others' results
// are not used), of both sides: one vote, one branch.  8192 causal rows, caps of 50:
// 730 us where the 4 terms do, 1040 where a teacher of nine times the scores takes
// the student along to the longer forms.  A vote per side has not been measured.
template <int MODE, int W>
__device__ __forceinline__ void cap_scores(float (&z1)[W], float (&z2)[W], const ScoreSide& s1, const ScoreSide& s2,
                                           bool use = true) {
    if (MODE == kScorePlain) return;
    const float top1 = use ? abs_max(z1) : 0.f, top2 = use ? abs_max(z2) : 0.f;
    if (MODE >= kScoreGeneral) {  // a side may have no cap
        if (s1.lim == 0.f) {
#pragma unroll
            for (int e = 0; e < W; ++e) z1[e] *= s1.c;
        }
        if (s2.lim == 0.f) {
#pragma unroll
            for (int e = 0; e < W; ++e) z2[e] *= s2.c;
        }
    }
    const bool c1 = MODE == kScoreBounded || s1.lim != 0.f, c2 = MODE == kScoreBounded || s2.lim != 0.f;
    if (__all_sync(0xffffffffu, (!c1 || top1 <= s1.z_near) && (!c2 || top2 <= s2.z_near))) {
        if (c1) cap_near(z1, s1);
        if (c2) cap_near(z2, s2);
    } else if (__all_sync(0xffffffffu, (!c1 || top1 <= s1.z_mid) && (!c2 || top2 <= s2.z_mid))) {
        if (c1) cap_mid(z1, s1);
        if (c2) cap_mid(z2, s2);
    } else {
        if (c1) {
#pragma unroll
            for (int e = 0; e < W; ++e) z1[e] = score_far(z1[e], s1);
        }
        if (c2) {
#pragma unroll
            for (int e = 0; e < W; ++e) z2[e] = score_far(z2[e], s2);
        }
    }
}

// Finish of a row from its state in x units (c = 1, scale = ln 2) or in raw
// units (plain: scale = the softmax scale).  The difference of the two
// log-sum-exps is taken before they are rounded: KL is often far smaller than
// either.  `empty`: the row sees no key.
__device__ __forceinline__ void finish_scored(const RowState& s, float scale, bool empty, float& kl, float& lse1,
                                              float& lse2) {
    if (empty) {
        kl = 0.f;
        lse1 = lse2 = -INFINITY;
        return;
    }
    const float a = logf(s.l1), b = logf(s.l2), r = s.l2 / s.l1;
    lse1 = fmaf(scale, s.m1, a);
    lse2 = fmaf(scale, s.m2, b);
    const float d = r > 1e-30f && r < 1e30f ? logf(r) : b - a;
    kl = fmaf(scale, s.acc / s.l1 + (s.m2 - s.m1), d);
    if (!(s.l1 > 0.f && s.l2 > 0.f)) kl = lse1 = lse2 = __int_as_float(0x7fc00000);  // NaN or -inf scores alone
}

}  // namespace streamkl
