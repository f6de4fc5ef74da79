// score_fwd.cu -- forward of the score-modified divergence on sm_103a: capped
// and biased scores, a key range per query row.
//
//   score_fwd_tile_kernel    128 query rows x the key tiles that any of them sees
//   score_fwd_decode_kernel  Nq <= 16: keys on the MMA M side, the key range split
//   score_combine_kernel     merges the splits of a row
//
// Roles, rings and the five-scalar state are those of the unmodified forward;
// what differs is the update: z -> x (score.cuh), the range of each row, and for
// bounded scores a sum of 2^x without a running maximum.
//
// 8192 causal rows, 32 heads: plain scores 511 us (1.08 PFLOP/s), caps of 50 730
// us (0.75).  The update bounds both; with caps the FMA pipe is busy 62% of the
// cycles, issue slots 65%, the tensor pipe 33%.
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "score.cuh"

namespace streamkl {

namespace {

constexpr float kScoreTau = 8.0f;  // lazy rescale: running maxima up to 2^8 stale
// Update warpgroups of the tile kernel, each taking its share of a tile's columns.
// The cap's polynomial makes the update the slowest part, and its dependent steps
// need more warps to overlap (8K causal, 32 heads: 2 groups 985 us, 4 765); the
// plain update does better with the registers of 2 (8K tokens in documents: 197
// against 206 us).
constexpr int sf_groups(int mode) { return mode == kScorePlain ? 2 : 4; }
// warp 0 copies, warp 1 the S1 MMAs, the update warpgroups, the S2 MMAs, and the work items
constexpr int sf_threads(int mode) { return 64 + 128 * sf_groups(mode) + 64; }
constexpr int kSfNear = 4;   // key tiles left to issue when an item counts as nearly done
constexpr uint64_t kSfDrainNs = 200000000ull;  // in-flight copies and MMAs retire before a CTA exits

// A 128-row query tile of one head, and a share of its key tiles.
struct WorkItem {
    int bh, q0, split;
    int kt_begin, n_tiles;
    int valid;  // 0: no further items
    int pad[2];
};
static_assert(sizeof(WorkItem) == 32, "packed");

template <int D, int NST, int GROUPS>
struct ScoreTileSmem {
    static constexpr int kQBytes = kBlockQ * D * 2;
    static constexpr int kKBytes = kBlockK * D * 2;
    static constexpr int q1 = 0;
    static constexpr int q2 = kQBytes;
    static constexpr int k = 2 * kQBytes;  // stage s: K1 at k + 2*s*kKBytes, K2 right after
    static constexpr int bar_q = k + 2 * NST * kKBytes;
    static constexpr int bar_kfull = bar_q + 8;
    static constexpr int bar_kempty = bar_kfull + 8 * NST;
    static constexpr int bar_sfull = bar_kempty + 8 * NST;
    static constexpr int bar_sempty = bar_sfull + 16;
    static constexpr int bar_done = bar_sempty + 16;      // drain barriers of aborted MMA issuers (S1, S2)
    static constexpr int bar_qempty = bar_done + 16;
    static constexpr int bar_ifull = bar_qempty + 8;      // [2] work items
    static constexpr int bar_iempty = bar_ifull + 16;
    static constexpr int bar_clc = bar_iempty + 16;
    static constexpr int bar_near = bar_clc + 8;          // an item's copies are all but issued
    static constexpr int misc = bar_near + 8;             // tmem base, abort flag, items claimed (4 B each)
    static constexpr int clc = (misc + 16 + 15) / 16 * 16;  // [2] launch-control responses
    static constexpr int items = clc + 32;                // [2] WorkItem
    static constexpr int ranges = items + 64;             // [2][128] int2: the rows' key ranges
    static constexpr int red = ranges + 2 * kBlockQ * 8;  // [2][groups - 1][5][128] floats: the other groups' states
    static constexpr int kRed = (GROUPS - 1) * 5 * 128;
    static constexpr int total = red + 2 * kRed * 4;
    static constexpr int alloc = total + 1024;    // slack for 1024-byte alignment
};

__device__ __noinline__ bool score_drain(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > limit_ns) return false;
    }
    return true;
}

// The bias -slope |d0 - e| of column e.  Of a chunk that lies wholly before the
// warp's rows (where > 0) or behind them (where < 0) it is linear in e; its part
// without e is returned, for update_scored to add to the running maximum instead
// of to every score.
template <int W>
__device__ __forceinline__ float add_bias(float (&x)[W], float slope, float d0, int where) {
    if (where == 0) {
#pragma unroll
        for (int e = 0; e < W; ++e) x[e] = fmaf(-slope, fabsf(d0 - static_cast<float>(e)), x[e]);
        return 0.f;
    }
    const float s = where > 0 ? slope : -slope;
#pragma unroll
    for (int e = 0; e < W; e += 2) {
        const float2 v = __ffma2_rn(splat(s), make_float2(static_cast<float>(e), static_cast<float>(e + 1)),
                                    make_float2(x[e], x[e + 1]));
        x[e] = v.x;
        x[e + 1] = v.y;
    }
    return -s * d0;
}

// Hidden products become 0: whatever they were (NaN, infinities) has no effect,
// not even on the form that cap_scores takes.
template <int W>
__device__ __forceinline__ void hide(float (&z)[W], int first, int last) {
#pragma unroll
    for (int e = 0; e < W; ++e)
        if (e < first || e > last) z[e] = 0.f;
}

// Online update with columns [first, last] visible (the hidden ones finite).
// c = 1 when z holds x; the scores are z + base1 and z + base2 (kScoreBias).
template <int MODE, bool MASKED, int W>
__device__ __forceinline__ void update_scored(const float (&z1)[W], const float (&z2)[W], int first, int last,
                                              RowState& st, float c, float tau, float base1, float base2) {
    constexpr bool BOUNDED = MODE == kScoreBounded, BIAS = MODE == kScoreBias;
    float2 s1[2] = {splat(0.f), splat(0.f)}, s2[2] = {splat(0.f), splat(0.f)}, sa[2] = {splat(0.f), splat(0.f)};
    const float2 neg = splat(-1.f);
    if (BOUNDED) {
        st.m1 = st.m2 = 0.f;
    } else {
        float a1 = -INFINITY, b1 = -INFINITY, a2 = -INFINITY, b2 = -INFINITY;
#pragma unroll
        for (int e = 0; e < W; e += 4) {
            float v1[4], v2[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool vis = !MASKED || (e + k >= first && e + k <= last);
                v1[k] = vis ? z1[e + k] : -INFINITY;
                v2[k] = vis ? z2[e + k] : -INFINITY;
            }
            a1 = max3f(a1, v1[0], v1[1]);
            b1 = max3f(b1, v1[2], v1[3]);
            a2 = max3f(a2, v2[0], v2[1]);
            b2 = max3f(b2, v2[2], v2[3]);
        }
        const float cm1 = fmaxf(a1, b1) + (BIAS ? base1 : 0.f), cm2 = fmaxf(a2, b2) + (BIAS ? base2 : 0.f);
        if (cm1 > st.m1 + tau) {
            const float a = ex2(c * (st.m1 - cm1));  // 0 on the first visible chunk (m1 = -inf)
            st.l1 *= a;
            st.acc *= a;
            st.m1 = cm1;
        }
        if (cm2 > st.m2 + tau) {
            st.l2 *= ex2(c * (st.m2 - cm2));
            st.m2 = cm2;
        }
    }
    // a row that has seen no key yet keeps m = -inf: a reference of 0 makes its masked terms 2^-inf = 0
    float r1 = MASKED && st.m1 == -INFINITY ? 0.f : st.m1, r2 = MASKED && st.m2 == -INFINITY ? 0.f : st.m2;
    if (BIAS) {  // relative to the base; the running maximum itself stays as it is, so that a far base costs it no bits
        r1 -= base1;
        r2 -= base2;
    }
    const float2 cc = splat(c), n1 = splat(-c * r1), n2 = splat(-c * r2);
#pragma unroll
    for (int e = 0; e < W; e += 2) {
        const int k = (e >> 1) & 1;
        const float2 u1 = make_float2(z1[e], z1[e + 1]), u2 = make_float2(z2[e], z2[e + 1]);
        float2 x1 = BOUNDED ? u1 : __ffma2_rn(u1, cc, n1), x2 = BOUNDED ? u2 : __ffma2_rn(u2, cc, n2);
        const float2 df = __ffma2_rn(u2, neg, u1);
        if (MASKED) {
            const bool va = e >= first && e <= last, vb = e + 1 >= first && e + 1 <= last;
            x1 = make_float2(va ? x1.x : -INFINITY, vb ? x1.y : -INFINITY);
            x2 = make_float2(va ? x2.x : -INFINITY, vb ? x2.y : -INFINITY);
        }
        const float2 p1 = make_float2(ex2(x1.x), ex2(x1.y)), p2 = make_float2(ex2(x2.x), ex2(x2.y));
        s1[k] = __fadd2_rn(s1[k], p1);
        s2[k] = __fadd2_rn(s2[k], p2);
        sa[k] = __ffma2_rn(p1, df, sa[k]);
    }
    const float sum = (s1[0].x + s1[0].y) + (s1[1].x + s1[1].y);
    st.l1 += sum;
    st.l2 += (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
    st.acc += (sa[0].x + sa[0].y) + (sa[1].x + sa[1].y);
    if (BIAS) st.acc = fmaf(sum, base1 - base2, st.acc);
}

// States of one row over disjoint keys, merged at once.
template <int MODE, int N>
__device__ __forceinline__ RowState merge_groups(const RowState (&o)[N], float c) {
    RowState s = o[0];
#pragma unroll
    for (int g = 1; g < N; ++g) {
        s.m1 = fmaxf(s.m1, o[g].m1);
        s.m2 = fmaxf(s.m2, o[g].m2);
    }
    s.l1 = s.acc = s.l2 = 0.f;
#pragma unroll
    for (int g = 0; g < N; ++g) {  // a group that saw nothing has m = -inf and l = acc = 0
        const float w1 = MODE == kScoreBounded ? 1.f : o[g].m1 == -INFINITY ? 0.f : ex2(c * (o[g].m1 - s.m1));
        const float w2 = MODE == kScoreBounded ? 1.f : o[g].m2 == -INFINITY ? 0.f : ex2(c * (o[g].m2 - s.m2));
        s.l1 = fmaf(o[g].l1, w1, s.l1);
        s.acc = fmaf(o[g].acc, w1, s.acc);
        s.l2 = fmaf(o[g].l2, w2, s.l2);
    }
    return s;
}

__device__ __forceinline__ void store_scored(const FwdParams& p, size_t row, int split, const RowState& st, bool empty,
                                             bool failed) {
    if (p.num_splits == 1) {
        float kl, l1, l2;
        finish_scored(st, p.scale, empty, kl, l1, l2);
        if (failed) kl = l1 = l2 = __int_as_float(0x7fc00000);
        p.KL[row] = kl;
        p.LSE1[row] = l1;
        p.LSE2[row] = l2;
    } else {
        const size_t R = static_cast<size_t>(p.B) * p.H * p.Nq, S = static_cast<size_t>(p.num_splits);
        float v[5] = {st.m1, st.l1, st.acc, st.m2, st.l2};
        if (failed) v[1] = v[4] = __int_as_float(0x7fc00000);
#pragma unroll
        for (int f = 0; f < 5; ++f) p.part[(f * S + split) * R + row] = v[f];
    }
}

// Rows of the last two claimed work items: their outputs, or their split's parts
// of them, become NaN.
__device__ __noinline__ void mark_claimed(const FwdParams& p, const WorkItem* items, int claims) {
    const float nan = __int_as_float(0x7fc00000);
    for (int k = max(0, claims - 2); k < claims; ++k) {
        const WorkItem& item = items[k & 1];
        if (!item.valid) continue;
        for (int r = threadIdx.x; r < kBlockQ && item.q0 + r < p.Nq; r += blockDim.x)
            store_scored(p, static_cast<size_t>(item.bh) * p.Nq + item.q0 + r, item.split, RowState{nan, nan, nan, nan, nan},
                         false, true);
    }
}

// This split's share of key tiles [lo, hi).
__device__ __forceinline__ int2 split_tiles(int lo, int hi, int split, int num_splits) {
    const int n = max(0, hi - lo), per = (n + num_splits - 1) / num_splits;
    const int begin = lo + split * per;
    return make_int2(begin, max(0, min(hi, begin + per) - begin));
}

}  // namespace

// ---------------------------------------------------------------------------
// Tile forward.  A work item is a 128-row query tile of one head; a CTA starts
// with its own and then takes over CTAs that have not started, one after the
// other.  Short rows (documents, windows) make short items: their start (row
// ranges, first copies) and end (merge, outputs) run while the neighbouring items'
// tiles are computed.  Every role walks the same items:
//   the last warp fetches the items and works out the union of the rows' key ranges
//                 (only tiles inside it are visited)
//   warp 0        issues the copies
//   warp 1, S2    the MMAs (warp 1 owns TMEM)
//   the others    the update, one query row per thread
// Rings (key tiles, score buffers) run on through the items.  8192 tokens, 32
// heads, documents of 468 to 2741 tokens: one item per CTA 258 us, as here 174 us.
// ---------------------------------------------------------------------------
template <int D, int NST, int MODE>
__global__ void __launch_bounds__(sf_threads(MODE), 1)
    score_fwd_tile_kernel(const __grid_constant__ CUtensorMap tQ1, const __grid_constant__ CUtensorMap tK1,
                          const __grid_constant__ CUtensorMap tQ2, const __grid_constant__ CUtensorMap tK2,
                          const __grid_constant__ FwdParams p, const __grid_constant__ ScoreParams sp) {
    constexpr int kGroups = sf_groups(MODE), kUpdate = 128 * kGroups;
    constexpr int kS2Warp = 2 + kUpdate / 32, kItemWarp = kS2Warp + 1;
    using L = ScoreTileSmem<D, NST, kGroups>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::misc + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::misc);
    int* claims = reinterpret_cast<int*>(gbase + L::misc + 8);  // work items claimed
    WorkItem* items = reinterpret_cast<WorkItem*>(gbase + L::items);
    int2* ranges = reinterpret_cast<int2*>(gbase + L::ranges);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(base + L::bar_q, 1);
        mbar_init(base + L::bar_qempty, 2);  // both issuers' last MMAs of the item
        for (int s = 0; s < NST; ++s) {
            mbar_init(base + L::bar_kfull + 8 * s, 1);
            mbar_init(base + L::bar_kempty + 8 * s, 2);  // both issuers' MMAs have read the stage
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(base + L::bar_sfull + 8 * s, 2);  // S1 and S2 of the buffer are complete
            mbar_init(base + L::bar_sempty + 8 * s, kUpdate);
            mbar_init(base + L::bar_ifull + 8 * s, 1);
            mbar_init(base + L::bar_iempty + 8 * s, 3 + kUpdate / 32);  // the copies, the issuers, the update warps
        }
        mbar_init(base + L::bar_done, 1);
        mbar_init(base + L::bar_done + 8, 1);
        mbar_init(base + L::bar_clc, 1);
        mbar_init(base + L::bar_near, 1);
        *abort_flag = 0;
        *claims = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 1) tmem_alloc(base + L::misc, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wc{abort_flag, p.status, p.wait_ns};

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            prefetch_tensormap(&tQ1);
            prefetch_tensormap(&tK1);
            prefetch_tensormap(&tQ2);
            prefetch_tensormap(&tK2);
            const uint64_t keep = policy_evict_last();  // key tiles are read again by other query tiles
            int it = 0, n_q = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int slot = k & 1;
                if (!mbar_wait(base + L::bar_ifull + 8 * slot, (k >> 1) & 1, wc, kErrWaitOther)) break;
                const WorkItem item = items[slot];
                mbar_arrive(base + L::bar_iempty + 8 * slot);
                if (!item.valid) break;
                if (item.n_tiles == 0) {
                    mbar_arrive(base + L::bar_near);
                    continue;
                }
                const int b = item.bh / p.H, h = item.bh - b * p.H, hk = h / p.kv_group;
                // the previous item's last MMAs have read its query tiles
                if (!mbar_wait(base + L::bar_qempty, (n_q & 1) ^ 1, wc, kErrWaitQ)) break;
                mbar_arrive_expect_tx(base + L::bar_q, 2 * L::kQBytes);
#pragma unroll
                for (int c = 0; c < D / kSwizzleCols; ++c) {
                    tma_load_4d(base + L::q1 + c * kBlockQ * 128, &tQ1, base + L::bar_q, c * kSwizzleCols, item.q0, h, b);
                    tma_load_4d(base + L::q2 + c * kBlockQ * 128, &tQ2, base + L::bar_q, c * kSwizzleCols, item.q0, h, b);
                }
                ++n_q;
                for (int t = 0; t < item.n_tiles; ++t, ++it) {
                    if (t == max(0, item.n_tiles - kSfNear)) mbar_arrive(base + L::bar_near);
                    const int s = it % NST;
                    if (!(ok = mbar_wait(base + L::bar_kempty + 8 * s, ((it / NST) & 1) ^ 1, wc, kErrWaitK))) break;
                    const uint32_t fb = base + L::bar_kfull + 8 * s;
                    mbar_arrive_expect_tx(fb, 2 * L::kKBytes);
                    const int k0 = (item.kt_begin + t) * kBlockK;
                    const uint32_t k1s = base + L::k + 2 * s * L::kKBytes, k2s = k1s + L::kKBytes;
#pragma unroll
                    for (int c = 0; c < D / kSwizzleCols; ++c) {
                        tma_load_4d_hint(k1s + c * kBlockK * 128, &tK1, fb, c * kSwizzleCols, k0, hk, b, keep);
                        tma_load_4d_hint(k2s + c * kBlockK * 128, &tK2, fb, c * kSwizzleCols, k0, hk, b, keep);
                    }
                }
            }
            // every issued copy has landed, every stage was released
            if (n_q > 0) score_drain(base + L::bar_q, (n_q - 1) & 1, kSfDrainNs);
            for (int j = max(0, it - NST); j < it; ++j) {
                score_drain(base + L::bar_kfull + 8 * (j % NST), (j / NST) & 1, kSfDrainNs);
                if (!*abort_flag) score_drain(base + L::bar_kempty + 8 * (j % NST), (j / NST) & 1, kSfDrainNs);
            }
        }
    } else if (warp == kItemWarp) {
        // ------------------------------------------------------------ work items
        // The next item is asked for once every role has taken up the one before, so that its start
        // hides behind that one's tiles; of the last three items per SM only when that one is nearly
        // done, so that they go to the CTAs that end first (256 items of 4 to 16 tiles: 67 us when
        // always early, 53 us so; 2048 items of 1 to 23 tiles: 197 us when always late, 175 so).
        // These two waits last as long as whole items do: the limit of a wait is theirs per key tile.
        // After a give-up `claims` says which items the CTA answers for: the last one of them may be
        // one whose response came late and that no role has seen.
        int unit = blockIdx.x, last_tiles = 0, before_tiles = 0;
        bool gave_up = false;
        WaitCtx wi = wc;
        for (int k = 0;; ++k) {
            const int slot = k & 1;
            if (k > 0) {
                wi.limit_ns = max(p.wait_ns, min(p.wait_ns, 1ull << 38) * (1ull + last_tiles + before_tiles));
                if (!__all_sync(0xffffffffu, mbar_wait(base + L::bar_iempty + 8 * (slot ^ 1), ((k - 1) >> 1) & 1, wi, kErrWaitOther)))
                    break;
                const bool late = unit >= static_cast<int>(gridDim.x) - 3 * p.take_over;
                if (p.take_over && late &&
                    !__all_sync(0xffffffffu, mbar_wait(base + L::bar_near, (k - 1) & 1, wi, kErrWaitOther)))
                    break;
                unit = -1;
                if (p.take_over) {
                    const uint32_t response = base + L::clc + 16 * slot;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(base + L::bar_clc, 16);
                        clc_request(response, base + L::bar_clc);
                    }
                    gave_up = !__all_sync(0xffffffffu, mbar_wait(base + L::bar_clc, (k - 1) & 1, wc, kErrWaitOther));
                    if (gave_up && !__all_sync(0xffffffffu, score_drain(base + L::bar_clc, (k - 1) & 1, kSfDrainNs))) break;
                    unit = clc_response(response);
                    fence_proxy_async_smem();  // the response is read before its slot is written again
                    __syncwarp();
                }
            }
            WorkItem item{0, 0, 0, 0, 0, unit >= 0, {0, 0}};
            if (unit >= 0) {
                // Groups of heads, a few waves of CTAs each, so that CTAs running at a time share
                // key tiles through L2; in a group the last query tiles of every head, which see
                // the most keys under a causal mask, come first.
                const int u = unit / p.num_splits;
                const int2 at = grouped_order(u, p.num_q_tiles, p.B * p.H, p.order_group);
                const int b = at.x / p.H;
                item.bh = at.x;
                item.q0 = (p.num_q_tiles - 1 - at.y) * kBlockQ;
                item.split = unit - u * p.num_splits;
                int2 r[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) r[n] = row_range(sp, p.Nq, p.Nk, b, item.q0 + lane + 32 * n);
                int lo = INT32_MAX, hi = 0;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    ranges[slot * kBlockQ + lane + 32 * n] = r[n];
                    if (r[n].x < r[n].y) lo = min(lo, r[n].x), hi = max(hi, r[n].y);
                }
                lo = __reduce_min_sync(0xffffffffu, lo);
                hi = __reduce_max_sync(0xffffffffu, hi);
                if (lo < hi) {
                    const int2 mine = split_tiles(lo / kBlockK, (hi + kBlockK - 1) / kBlockK, item.split, p.num_splits);
                    item.kt_begin = mine.x;
                    item.n_tiles = mine.y;
                }
            }
            before_tiles = last_tiles;
            last_tiles = item.n_tiles;
            if (lane == 0) items[slot] = item, *claims = k + 1;
            __syncwarp();
            if (gave_up) break;
            if (lane == 0) mbar_arrive(base + L::bar_ifull + 8 * slot);
            if (unit < 0) break;
        }
    } else if (warp == 1 || warp == kS2Warp) {
        // ------------------------------------------------------------ MMA: S1 (warp 1), S2 (last warp)
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(kBlockQ, kBlockK);
            const bool second = warp != 1;
            const uint32_t done_bar = base + L::bar_done + (second ? 8 : 0);
            const uint32_t dhi = smem_desc_hi();
            const uint32_t q_lo = smem_desc_lo_k128(base + (second ? L::q2 : L::q1));
            const uint32_t k_lo0 = smem_desc_lo_k128(base + L::k) + (second ? (L::kKBytes >> 4) : 0u);
            constexpr uint32_t kStageLo = (2 * L::kKBytes) >> 4;
            const uint32_t dcol = second ? kBlockK : 0u;
            int it = 0, n_q = 0, s = 0;
            uint32_t kph = 0, k_lo = k_lo0;
            // test aid: a wait on a barrier that nothing arrives on gives up after wait_ns; the first item counts as
            // taken up, so that the CTA goes on to claim the next one
            const bool stall = p.inject_stall && blockIdx.x == 0 && !second;
            if (stall) mbar_arrive(base + L::bar_iempty);
            bool ok = !(stall && !mbar_wait(base + L::bar_done, 0, wc, kErrWaitOther));
            for (int k = 0; ok; ++k) {
                const int slot = k & 1;
                if (!mbar_wait(base + L::bar_ifull + 8 * slot, (k >> 1) & 1, wc, kErrWaitOther)) break;
                const int n_tiles = items[slot].n_tiles, valid = items[slot].valid;
                mbar_arrive(base + L::bar_iempty + 8 * slot);
                if (!valid) break;
                if (n_tiles == 0) continue;
                if (!mbar_wait(base + L::bar_q, n_q & 1, wc, kErrWaitQ)) break;
                ++n_q;
                tc_fence_after();
                for (int t = 0; t < n_tiles; ++t, ++it) {
                    const int buf = it & 1;
                    if (!(ok = mbar_wait(base + L::bar_kfull + 8 * s, kph, wc, kErrWaitK))) break;
                    if (!(ok = mbar_wait(base + L::bar_sempty + 8 * buf, ((it >> 1) & 1) ^ 1, wc, kErrWaitS))) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * 2 * kBlockK + dcol;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t qo = ((kk >> 2) * kBlockQ * 128 + (kk & 3) * 32) >> 4;
                        const uint32_t ko = ((kk >> 2) * kBlockK * 128 + (kk & 3) * 32) >> 4;
                        tc_mma_bf16_w(d, q_lo + qo, dhi, k_lo + ko, dhi, idesc, kk > 0);
                    }
                    tc_commit(base + L::bar_sfull + 8 * buf);
                    tc_commit(base + L::bar_kempty + 8 * s);
                    if (++s == NST) {
                        s = 0;
                        kph ^= 1;
                        k_lo = k_lo0;
                    } else {
                        k_lo += kStageLo;
                    }
                }
                if (ok) tc_commit(base + L::bar_qempty);
            }
            if (*abort_flag && it > 0) {  // let the issued MMAs retire before TMEM is freed
                tc_commit(done_bar);
                score_drain(done_bar, 0, kSfDrainNs);
            }
        }
    } else {
        // ------------------------------------------------------------ online update
        constexpr int kChunks = 4 / kGroups;  // 32-column chunks per group and tile
        const int wg = (warp - 2) >> 2;
        const int wq = warp & 3;
        const int row = wq * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float c = MODE == kScorePlain ? p.scale_log2e : 1.f;
        const float tau = kScoreTau / c;
        int it = 0;
        // All update warps leave together: each pass ends in one barrier that also says whether every warp goes on.
        for (int k = 0;; ++k) {
            const int slot = k & 1;
            bool ok = __all_sync(0xffffffffu, mbar_wait(base + L::bar_ifull + 8 * slot, (k >> 1) & 1, wc, kErrWaitOther));
            const WorkItem item = items[slot];
            const int2 range = ranges[slot * kBlockQ + row];
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(base + L::bar_iempty + 8 * slot);
            const bool live = ok && item.valid;
            const int n_tiles = live ? item.n_tiles : 0;
            const int bh = item.bh, b = bh / p.H, i = item.q0 + row;
            // keys [warp_lo, warp_hi) are seen by some row of the warp, [whole_lo, whole_hi) by all of them
            const int warp_lo = __reduce_min_sync(0xffffffffu, range.x < range.y ? range.x : INT32_MAX);
            const int warp_hi = __reduce_max_sync(0xffffffffu, range.y);
            const int whole_lo = __reduce_max_sync(0xffffffffu, range.x);
            const int whole_hi = __reduce_min_sync(0xffffffffu, range.y);
            int64_t pos = 0;
            float sl1 = 0.f, sl2 = 0.f;
            if (MODE == kScoreBias && live) {
                const int h = bh - b * p.H;
                pos = row_position(sp, p.Nq, p.Nk, b, i);
                if (sp.side[0].slopes) sl1 = sp.side[0].slopes[h] * kLog2e;
                if (sp.side[1].slopes) sl2 = sp.side[1].slopes[h] * kLog2e;
            }
            RowState st{-INFINITY, 0.f, 0.f, -INFINITY, 0.f};
            for (int t = 0; t < n_tiles; ++t, ++it) {
                const int buf = it & 1;
                if (!__all_sync(0xffffffffu, mbar_wait(base + L::bar_sfull + 8 * buf, (it >> 1) & 1, wc, kErrWaitS))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int j0 = (item.kt_begin + t) * kBlockK;
                const uint32_t t1 = tl + buf * 2 * kBlockK, t2 = t1 + kBlockK;
#pragma unroll 1
                for (int cc = 0; cc < kChunks; ++cc) {
                    const int ch = kChunks * wg + cc;
                    const int c0 = j0 + ch * 32;  // the chunk's first key
                    const bool any = c0 < warp_hi && c0 + 32 > warp_lo;
                    const bool whole = c0 >= whole_lo && c0 + 32 <= whole_hi;
                    if (!any) {
                        if (cc == kChunks - 1) {
                            tc_fence_before();
                            mbar_arrive(base + L::bar_sempty + 8 * buf);
                        }
                        continue;
                    }
                    float z1[32], z2[32];
                    tmem_ld32(t1 + ch * 32, z1);
                    tmem_ld32(t2 + ch * 32, z2);
                    tc_wait_ld();
                    if (cc == kChunks - 1) {
                        tc_fence_before();
                        mbar_arrive(base + L::bar_sempty + 8 * buf);
                    }
                    const int first = range.x - c0, last = range.y - 1 - c0;  // columns that the row sees
                    bool masked = false, take = true;
                    if (!whole) {
                        // Rows of two documents in one warp: each sees all of most chunks or nothing
                        // of them, which needs no mask, only the rows that take part.
                        take = first <= 0 && last >= 31;
                        const bool none = first > 31 || last < 0 || range.x >= range.y;
                        masked = !__all_sync(0xffffffffu, take || none);
                        if (masked) {
                            hide(z1, first, last);
                            hide(z2, first, last);
                            take = true;
                        }
                    }
                    cap_scores<MODE>(z1, z2, sp.side[0], sp.side[1], take);
                    float base1 = 0.f, base2 = 0.f;
                    if (MODE == kScoreBias) {
                        const int64_t away = pos - c0;  // distance of the chunk's first key
                        const int where = away - lane >= 31 ? 1 : away - lane + 31 <= 0 ? -1 : 0;
                        const float d0 = static_cast<float>(away);
                        if (sl1 != 0.f) base1 = add_bias(z1, sl1, d0, where);
                        if (sl2 != 0.f) base2 = add_bias(z2, sl2, d0, where);
                    }
                    if (masked)
                        update_scored<MODE, true>(z1, z2, first, last, st, c, tau, base1, base2);
                    else if (take)
                        update_scored<MODE, false>(z1, z2, 0, 31, st, c, tau, base1, base2);
                }
            }
            // the groups' states of a row; two buffers, so that one barrier per item keeps them apart
            float* red = reinterpret_cast<float*>(gbase + L::red) + slot * L::kRed;
            if (wg > 0) {
                float* r = red + (wg - 1) * 5 * 128;
                r[row] = st.m1;
                r[128 + row] = st.l1;
                r[256 + row] = st.acc;
                r[384 + row] = st.m2;
                r[512 + row] = st.l2;
            }
            const bool go_on = bar_sync_and(1, kUpdate, live && ok);
            if (wg == 0 && live) {
                RowState o[kGroups];
                o[0] = st;
#pragma unroll
                for (int g = 1; g < kGroups; ++g) {
                    const float* r = red + (g - 1) * 5 * 128;
                    o[g] = RowState{r[row], r[128 + row], r[256 + row], r[384 + row], r[512 + row]};
                }
                st = merge_groups<MODE>(o, c);
                if (i < p.Nq)
                    store_scored(p, static_cast<size_t>(bh) * p.Nq + i, item.split, st, range.x >= range.y,
                                 !go_on || *abort_flag);
            }
            if (!go_on) break;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // An item is claimed once every role has taken up the one before: after a give-up the unfinished ones
    // are among the last two, which are still in the ring.
    if (*abort_flag) mark_claimed(p, items, *claims);
}

// ---------------------------------------------------------------------------
// Decode forward, Nq <= 16: S^T = K Q^T with 128 keys on the TMEM lanes and up
// to 16 query columns (heads_per_cta heads of one key head x Nq rows), so a key
// byte is streamed once for all of them.  Bound by HBM: 4 caches of up to 131072
// keys, 8 key heads, caps of 50, 1.93 GB in 282 us with the combine.  Each split
// takes its share of the tiles that the CTA's rows see, not of the whole cache.
// ---------------------------------------------------------------------------
template <int D, int NST>
struct ScoreDecodeSmem {
    static constexpr int kQBytes = kDecodeMaxQ * D * 2;  // 16 rows
    static constexpr int kKBytes = kBlockK * D * 2;
    static constexpr int q1 = 0;
    static constexpr int q2 = ((kQBytes + 1023) / 1024) * 1024;
    static constexpr int k = q2 + q2;
    static constexpr int bar_q = k + 2 * NST * kKBytes;
    static constexpr int bar_kfull = bar_q + 8;
    static constexpr int bar_kempty = bar_kfull + 8 * NST;
    static constexpr int bar_sfull = bar_kempty + 8 * NST;
    static constexpr int bar_sempty = bar_sfull + 16;
    static constexpr int bar_done = bar_sempty + 16;
    static constexpr int misc = bar_done + 8;                       // tmem base, abort flag
    static constexpr int cols = (misc + 8 + 15) / 16 * 16;          // [16] columns: {begin, end, slope1, slope2}
    static constexpr int at = cols + kDecodeMaxQ * 16;              // [16] positions (int64)
    static constexpr int red = at + kDecodeMaxQ * 8;                // [4 warps][16 q][5] floats
    static constexpr int total = red + 4 * kDecodeMaxQ * 5 * 4;
    static constexpr int alloc = total + 1024;
};

template <int D, int NST, int MODE>
__global__ void __launch_bounds__(192, 1)
    score_fwd_decode_kernel(const __grid_constant__ CUtensorMap tQ1, const __grid_constant__ CUtensorMap tK1,
                            const __grid_constant__ CUtensorMap tQ2, const __grid_constant__ CUtensorMap tK2,
                            const __grid_constant__ FwdParams p, const __grid_constant__ ScoreParams sp) {
    using L = ScoreDecodeSmem<D, NST>;
    constexpr int NQ = kDecodeMaxQ;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::misc + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::misc);
    int4* cols = reinterpret_cast<int4*>(gbase + L::cols);
    int64_t* at = reinterpret_cast<int64_t*>(gbase + L::at);
    float* red = reinterpret_cast<float*>(gbase + L::red);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hp = p.heads_per_cta;
    const int nq = hp * p.Nq;  // packed query columns in use
    const int gi = blockIdx.x / p.num_splits;
    const int split = blockIdx.x - gi * p.num_splits;
    const int groups = p.H / hp;
    const int b = gi / groups, h0 = (gi - b * groups) * hp;
    const int hk = h0 / p.kv_group;  // key head shared by the packed query heads
    const size_t row0 = (static_cast<size_t>(b) * p.H + h0) * p.Nq;  // output row of column 0

    // the ranges of the columns: every warp works out the same bounds
    int lo = INT32_MAX, hi = 0, full_lo = 0, full_hi = INT32_MAX;
    if (lane < nq) {
        const int i = lane % p.Nq, h = h0 + lane / p.Nq;
        const int2 r = row_range(sp, p.Nq, p.Nk, b, i);
        if (r.x < r.y) lo = r.x, hi = r.y;
        full_lo = r.x, full_hi = r.y;
        if (warp == 0) {
            const float a1 = MODE == kScoreBias && sp.side[0].slopes ? sp.side[0].slopes[h] * kLog2e : 0.f;
            const float a2 = MODE == kScoreBias && sp.side[1].slopes ? sp.side[1].slopes[h] * kLog2e : 0.f;
            cols[lane] = make_int4(r.x, r.y, __float_as_int(a1), __float_as_int(a2));
            at[lane] = row_position(sp, p.Nq, p.Nk, b, i);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    full_lo = __reduce_max_sync(0xffffffffu, full_lo);  // keys [full_lo, full_hi) are seen by every column
    full_hi = __reduce_min_sync(0xffffffffu, full_hi);
    const int2 mine = lo < hi ? split_tiles(lo / kBlockK, (hi + kBlockK - 1) / kBlockK, split, p.num_splits)
                              : make_int2(0, 0);
    const int kt_begin = mine.x, n_tiles = mine.y;

    if (threadIdx.x == 0) {
        mbar_init(base + L::bar_q, 1);
        for (int s = 0; s < NST; ++s) {
            mbar_init(base + L::bar_kfull + 8 * s, 1);
            mbar_init(base + L::bar_kempty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(base + L::bar_sfull + 8 * s, 1);
            mbar_init(base + L::bar_sempty + 8 * s, 128);
        }
        mbar_init(base + L::bar_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    // unused query columns read zeros (the copies below fill only the first nq rows)
    for (int i = threadIdx.x; i < 2 * (D / kSwizzleCols) * (NQ - nq) * 8; i += blockDim.x) {
        const int chunk16 = i & 7, rr = i >> 3;
        const int r = nq + rr % (NQ - nq), tc = rr / (NQ - nq);  // tc: tensor * column blocks
        const uint32_t dst = base + (tc & 1 ? L::q2 : L::q1) + (tc >> 1) * NQ * 128 + r * 128 + chunk16 * 16;
        st_shared_v4(dst, 0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    if (warp == 1) tmem_alloc(base + L::misc, 64);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wc{abort_flag, p.status, p.wait_ns};

    if (warp == 0) {
        if (lane == 0 && n_tiles > 0) {
            prefetch_tensormap(&tQ1);
            prefetch_tensormap(&tK1);
            prefetch_tensormap(&tQ2);
            prefetch_tensormap(&tK2);
            const uint64_t stream_once = policy_evict_first();  // each key is read exactly once
            // one box = Nq rows x heads_per_cta heads, landing as nq consecutive rows
            mbar_arrive_expect_tx(base + L::bar_q, 2 * nq * D * 2);
#pragma unroll
            for (int c = 0; c < D / kSwizzleCols; ++c) {
                tma_load_4d(base + L::q1 + c * NQ * 128, &tQ1, base + L::bar_q, c * kSwizzleCols, 0, h0, b);
                tma_load_4d(base + L::q2 + c * NQ * 128, &tQ2, base + L::bar_q, c * kSwizzleCols, 0, h0, b);
            }
            int it = 0;
            for (; it < n_tiles; ++it) {
                const int s = it % NST;
                if (!mbar_wait(base + L::bar_kempty + 8 * s, ((it / NST) & 1) ^ 1, wc, kErrWaitK)) break;
                const uint32_t fb = base + L::bar_kfull + 8 * s;
                mbar_arrive_expect_tx(fb, 2 * L::kKBytes);
                const int k0 = (kt_begin + it) * kBlockK;
                const uint32_t k1s = base + L::k + 2 * s * L::kKBytes, k2s = k1s + L::kKBytes;
#pragma unroll
                for (int c = 0; c < D / kSwizzleCols; ++c) {
                    tma_load_4d_hint(k1s + c * kBlockK * 128, &tK1, fb, c * kSwizzleCols, k0, hk, b, stream_once);
                    tma_load_4d_hint(k2s + c * kBlockK * 128, &tK2, fb, c * kSwizzleCols, k0, hk, b, stream_once);
                }
            }
            score_drain(base + L::bar_q, 0, kSfDrainNs);  // the query tiles' copies have landed
            for (int j = max(0, it - NST); j < it; ++j) {
                score_drain(base + L::bar_kfull + 8 * (j % NST), (j / NST) & 1, kSfDrainNs);
                if (!*abort_flag) score_drain(base + L::bar_kempty + 8 * (j % NST), (j / NST) & 1, kSfDrainNs);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && n_tiles > 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(kBlockK, NQ);
            int issued = 0;
            // test aid: a wait on a barrier that nothing arrives on (bar_done is
            // only committed on the abort path below) gives up after wait_ns
            const bool stalled = p.inject_stall && blockIdx.x == 0 &&
                                 !mbar_wait(base + L::bar_done, 0, wc, kErrWaitOther);
            if (!stalled && mbar_wait(base + L::bar_q, 0, wc, kErrWaitQ)) {
                tc_fence_after();
                for (int it = 0; it < n_tiles; ++it) {
                    const int s = it % NST, buf = it & 1;
                    if (!mbar_wait(base + L::bar_kfull + 8 * s, (it / NST) & 1, wc, kErrWaitK)) break;
                    if (!mbar_wait(base + L::bar_sempty + 8 * buf, ((it >> 1) & 1) ^ 1, wc, kErrWaitS)) break;
                    tc_fence_after();
                    const uint32_t d1 = tmem + buf * 2 * NQ, d2 = d1 + NQ;
                    const uint32_t k1s = base + L::k + 2 * s * L::kKBytes, k2s = k1s + L::kKBytes;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t ko = (kk >> 2) * kBlockK * 128 + (kk & 3) * 32;
                        const uint32_t qo = (kk >> 2) * NQ * 128 + (kk & 3) * 32;
                        tc_mma_bf16(d1, smem_desc_k128(k1s + ko), smem_desc_k128(base + L::q1 + qo), idesc, kk > 0);
                    }
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t ko = (kk >> 2) * kBlockK * 128 + (kk & 3) * 32;
                        const uint32_t qo = (kk >> 2) * NQ * 128 + (kk & 3) * 32;
                        tc_mma_bf16(d2, smem_desc_k128(k2s + ko), smem_desc_k128(base + L::q2 + qo), idesc, kk > 0);
                    }
                    tc_commit(base + L::bar_sfull + 8 * buf);
                    tc_commit(base + L::bar_kempty + 8 * s);
                    ++issued;
                }
            }
            if (*abort_flag && issued > 0) {
                tc_commit(base + L::bar_done);
                score_drain(base + L::bar_done, 0, kSfDrainNs);
            }
        }
    } else {
        const int wq = warp & 3;
        const int krow = wq * 32 + lane;  // key within the tile = TMEM lane
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float c = MODE == kScorePlain ? p.scale_log2e : 1.f;
        const float tau = kScoreTau / c;
        RowState st[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) st[q] = RowState{-INFINITY, 0.f, 0.f, -INFINITY, 0.f};
        bool ok = true;
        for (int it = 0; it < n_tiles; ++it) {
            const int buf = it & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(base + L::bar_sfull + 8 * buf, (it >> 1) & 1, wc, kErrWaitS))) {
                ok = false;
                break;
            }
            tc_fence_after();
            float z1[NQ], z2[NQ];
            tmem_ld16(tl + buf * 2 * NQ, z1);
            tmem_ld16(tl + buf * 2 * NQ + NQ, z2);
            tc_wait_ld();
            tc_fence_before();
            mbar_arrive(base + L::bar_sempty + 8 * buf);
            const int j0 = (kt_begin + it) * kBlockK, j = j0 + krow;
            const bool whole = j0 >= full_lo && j0 + kBlockK <= full_hi;
            // bit q: column q sees this thread's key; hidden products become 0, so that
            // whatever they were has no effect, not even on the form of cap_scores
            uint32_t vis = 0xffffffffu;
            if (!whole) {
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    if (q < nq) {
                        const int2 range = *reinterpret_cast<const int2*>(&cols[q]);
                        if (j < range.x || j >= range.y) {
                            vis &= ~(1u << q);
                            z1[q] = z2[q] = 0.f;
                        }
                    }
                }
            }
            cap_scores<MODE>(z1, z2, sp.side[0], sp.side[1]);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                if (q < nq) {
                    float x1 = z1[q], x2 = z2[q];
                    if (MODE == kScoreBias) {
                        const float dist = fabsf(static_cast<float>(at[q] - j));
                        x1 = fmaf(-__int_as_float(cols[q].z), dist, x1);
                        x2 = fmaf(-__int_as_float(cols[q].w), dist, x2);
                    }
                    if ((vis >> q) & 1u) {
                        RowState& s = st[q];
                        if (MODE == kScoreBounded) {
                            s.m1 = s.m2 = 0.f;
                        } else {
                            if (x1 > s.m1 + tau) {
                                const float a = ex2(c * (s.m1 - x1));
                                s.l1 *= a;
                                s.acc *= a;
                                s.m1 = x1;
                            }
                            if (x2 > s.m2 + tau) {
                                s.l2 *= ex2(c * (s.m2 - x2));
                                s.m2 = x2;
                            }
                        }
                        const float p1 = ex2(c * (x1 - s.m1));
                        s.l1 += p1;
                        s.acc = fmaf(p1, x1 - x2, s.acc);
                        s.l2 += ex2(c * (x2 - s.m2));
                    }
                }
            }
        }
        // merge the 128 per-key states of every query: warp butterfly, then warps
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            if (q < nq) {
                RowState s = st[q];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    RowState t{__shfl_xor_sync(0xffffffffu, s.m1, o), __shfl_xor_sync(0xffffffffu, s.l1, o),
                               __shfl_xor_sync(0xffffffffu, s.acc, o), __shfl_xor_sync(0xffffffffu, s.m2, o),
                               __shfl_xor_sync(0xffffffffu, s.l2, o)};
                    merge_state(s, t, c);
                }
                if (lane == 0) {
                    float* r = red + (wq * NQ + q) * 5;
                    r[0] = s.m1;
                    r[1] = s.l1;
                    r[2] = s.acc;
                    r[3] = s.m2;
                    r[4] = s.l2;
                }
            }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");  // the four update warps only
        if (wq == 0 && lane < nq) {
            const int q = lane;
            RowState s{-INFINITY, 0.f, 0.f, -INFINITY, 0.f};
            for (int w = 0; w < 4; ++w) {
                const float* r = red + (w * NQ + q) * 5;
                RowState t{r[0], r[1], r[2], r[3], r[4]};
                merge_state(s, t, c);
            }
            store_scored(p, row0 + q, split, s, cols[q].x >= cols[q].y, !ok || *abort_flag);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
}

// ---------------------------------------------------------------------------
// One thread per row merges its partial states and finishes.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128) score_combine_kernel(const FwdParams p, const __grid_constant__ ScoreParams sp,
                                                            float c) {
    const size_t R = static_cast<size_t>(p.B) * p.H * p.Nq, S = static_cast<size_t>(p.num_splits);
    const size_t row = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (row >= R) return;
    RowState s{-INFINITY, 0.f, 0.f, -INFINITY, 0.f};
    for (size_t k = 0; k < S; ++k) {
        RowState t{p.part[(0 * S + k) * R + row], p.part[(1 * S + k) * R + row], p.part[(2 * S + k) * R + row],
                   p.part[(3 * S + k) * R + row], p.part[(4 * S + k) * R + row]};
        merge_state(s, t, c);
    }
    const size_t bh = row / p.Nq;
    const int2 r = row_range(sp, p.Nq, p.Nk, static_cast<int>(bh / p.H), static_cast<int>(row - bh * p.Nq));
    float kl, l1, l2;
    finish_scored(s, p.scale, r.x >= r.y, kl, l1, l2);
    p.KL[row] = kl;
    p.LSE1[row] = l1;
    p.LSE2[row] = l2;
}

namespace {

template <int D, int NST, int MODE>
cudaError_t launch_tile(const CUtensorMap* m, const FwdParams& p, const ScoreParams& sp, int ctas, cudaStream_t st) {
    constexpr int bytes = ScoreTileSmem<D, NST, sf_groups(MODE)>::alloc;
    static_assert(bytes <= 232448, "shared memory");
    auto k = score_fwd_tile_kernel<D, NST, MODE>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k<<<ctas, sf_threads(MODE), bytes, st>>>(m[0], m[1], m[2], m[3], p, sp);
    return cudaGetLastError();
}

template <int D, int NST, int MODE>
cudaError_t launch_decode(const CUtensorMap* m, const FwdParams& p, const ScoreParams& sp, int ctas, cudaStream_t st) {
    constexpr int bytes = ScoreDecodeSmem<D, NST>::alloc;
    static_assert(bytes <= 232448, "shared memory");
    auto k = score_fwd_decode_kernel<D, NST, MODE>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k<<<ctas, 192, bytes, st>>>(m[0], m[1], m[2], m[3], p, sp);
    return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_mode(int d, bool decode, const CUtensorMap* m, const FwdParams& p, const ScoreParams& sp, int ctas,
                        cudaStream_t st) {
    if (decode)
        return d == 128 ? launch_decode<128, 3, MODE>(m, p, sp, ctas, st) : launch_decode<64, 6, MODE>(m, p, sp, ctas, st);
    return d == 128 ? launch_tile<128, 2, MODE>(m, p, sp, ctas, st) : launch_tile<64, 4, MODE>(m, p, sp, ctas, st);
}

}  // namespace

cudaError_t launch_score_fwd(int d, int mode, bool decode, const CUtensorMap* maps, const FwdParams& p,
                             const ScoreParams& sp, int ctas, cudaStream_t stream) {
    cudaError_t e = mode == kScorePlain     ? launch_mode<kScorePlain>(d, decode, maps, p, sp, ctas, stream)
                    : mode == kScoreBounded ? launch_mode<kScoreBounded>(d, decode, maps, p, sp, ctas, stream)
                    : mode == kScoreGeneral ? launch_mode<kScoreGeneral>(d, decode, maps, p, sp, ctas, stream)
                                            : launch_mode<kScoreBias>(d, decode, maps, p, sp, ctas, stream);
    if (e != cudaSuccess || p.num_splits == 1) return e;
    const int64_t rows = int64_t(p.B) * p.H * p.Nq;
    score_combine_kernel<<<static_cast<unsigned>((rows + 127) / 128), 128, 0, stream>>>(
        p, sp, mode == kScorePlain ? p.scale_log2e : 1.f);
    return cudaGetLastError();
}

}  // namespace streamkl
