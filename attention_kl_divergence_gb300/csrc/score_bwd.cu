// score_bwd.cu -- backward of the score-modified divergence on sm_103a.
//
//   setting 1 (student trains): dS2 = g (P2 - P1)
//   setting 2 (teacher trains): dS1 = g P1 ((S1 - LSE1) - (S2 - LSE2) - KL)
//   dz_t = scale (1 - tanh^2(scale z_t / cap_t)) dS_t,  dQ_t = dz_t K_t,  dK_t = dz_t^T Q_t
//
// One key-tile kernel: 128 keys per CTA, the 64-row query tiles that see any of
// them streamed through; dK stays in tensor memory, dQ is added to float32 in
// L2 by bulk reductions.  Roles and rings are those of the unmodified fused
// backward; what differs is the recompute (score.cuh), the query tiles visited
// (from the rows' key ranges), the mask of a tile pair that is partly hidden, and
// the row constants, which a first kernel prepares and bulk copies fetch: worked
// out by the copying warp they took longer than a tile's matrix work.
//
// dS enters the gradient products as two bf16 terms (2^-17 of it is lost),
// whatever the gradients' type.  One term rounds each dS by up to 2^-8: what all
// keys have in common cancels in dQ, where the dS of a row sum to zero, and those
// roundings do not.  Keys with an offset of 16 beside a noise of 1 in an eighth of
// the channels: dQ off by 0.0085 of its norm with one term, by the output's own
// rounding, 0.0017, with two.  With one term the kernel took 1260 us instead of
// 1411; with two in dQ and one in dK as long as with two in both.
//
// 8192 causal rows, 32 heads on 8 key heads, caps of 50, bf16 gradients: prepare
// 21 us, gradients 1411 us, finish 30 us: about 3100 cycles of an SM per tile, and
// 2900 without caps.  Without caps the 32 MMAs of a tile (about 60 cycles each,
// whatever N <= 128 is) and their handoffs are the bound, with caps the update's
// dependent steps (the tensor pipe is busy half of the cycles; with one dS term
// twice the update warps or a second buffer for the scores changed nothing).
#include <algorithm>

#include "bwd_common.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "score.cuh"

namespace streamkl {

namespace {

// The backward's workspace, written by score_prepare_kernel:
//   rows   [B*H][q tiles][3][64] floats: -LSE1 (log2), -xb and g * scale of each row
//   keys   [B][q tiles] KeyBlock: the ranges of the tile's rows and their bounds
// Both are read by bulk copies of a tile's block.
struct KeyBlock {
    int32_t begin[kBwdTile], end[kBwdTile];
    int4 bounds[2];  // per half: lowest begin, highest end of a row with keys; highest begin, lowest end of all rows
};
constexpr int kRowBlockBytes = 3 * kBwdTile * 4;
static_assert(sizeof(KeyBlock) == 2 * kBwdTile * 4 + 32, "packed");

__device__ __forceinline__ bool has_nonfinite_bf16(uint32_t u) {
    return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t at) {
    uint32_t u;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(at) : "memory");
    return u;
}

// Zero every row with a NaN or an infinity among query rows [r0, r0 + 32) of
// the tile at `qt`, and this thread's row of the key tile at `kt`.  Several
// warps may find the same row: they all write zeros.
template <int D>
__device__ __forceinline__ void clear_nonfinite(uint32_t qt, int r0, uint32_t kt, int key_row, int lane) {
#pragma unroll 1
    for (int r = r0; r < r0 + 32; ++r) {
        bool bad = false;
#pragma unroll
        for (int c = 0; c < D / kSwizzleCols; ++c)
            bad |= has_nonfinite_bf16(ld_shared_u32(qt + c * kBwdTile * 128 + r * 128 + lane * 4));
        if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
            for (int c = 0; c < D / kSwizzleCols; ++c)
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(qt + c * kBwdTile * 128 + r * 128 + lane * 4), "r"(0u)
                             : "memory");
        }
    }
    bool bad = false;
#pragma unroll 1
    for (int k = 0; k < D / 2; ++k)
        bad |= has_nonfinite_bf16(ld_shared_u32(kt + (k >> 5) * kBlockK * 128 + key_row * 128 + (k & 31) * 4));
    if (bad) {
#pragma unroll 1
        for (int k = 0; k < D / 2; ++k)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(kt + (k >> 5) * kBlockK * 128 + key_row * 128 + (k & 31) * 4),
                         "r"(0u)
                         : "memory");
    }
    __syncwarp();
}

// One block per (64-row query tile, batch and head): the constants of its rows,
// the ranges of the tile (the first head's block) and zeros in its rows of dQ.
// A row that sees no key gets zero constants; an infinite LSE (from an infinite
// score) counts as NaN, as in its own softmax.
__global__ void __launch_bounds__(256) score_prepare_kernel(const __grid_constant__ BwdParams p,
                                                            const __grid_constant__ ScoreParams sp, int setting, int d) {
    const size_t block = blockIdx.x;
    const int bh = static_cast<int>(block / p.num_q_tiles), tile = static_cast<int>(block - static_cast<size_t>(bh) * p.num_q_tiles);
    const int b = bh / p.H, h = bh - b * p.H;
    const int rows = min(kBwdTile, p.Nq - tile * kBwdTile);
    float4* dq = reinterpret_cast<float4*>(p.dQacc + (static_cast<size_t>(bh) * p.Nq + tile * kBwdTile) * d);
    for (int k = threadIdx.x; k < rows * d / 4; k += blockDim.x) dq[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (threadIdx.x >= kBwdTile) return;
    const int r = threadIdx.x, i = tile * kBwdTile + r;
    const int2 keys = row_range(sp, p.Nq, p.Nk, b, i);
    const bool live = keys.x < keys.y;
    float la = 0.f, xb = 0.f, g = 0.f;
    if (live) {
        const size_t row = static_cast<size_t>(bh) * p.Nq + i;
        const float l1 = p.LSE1[row], l2 = p.LSE2[row], nan = __int_as_float(0x7fc00000);
        const float other = fabsf(l2) < INFINITY ? l2 : nan;
        la = fabsf(l1) < INFINITY ? l1 * kLog2e : nan;
        xb = setting == 1 ? other * kLog2e : (l1 - other) + p.KL[row];
        g = p.g[row];
    }
    float* out = sp.rows + block * (3 * kBwdTile);
    out[r] = -la;
    out[kBwdTile + r] = -xb;
    out[2 * kBwdTile + r] = g * p.scale;  // the softmax scale of both gradients
    if (h != 0) return;
    KeyBlock& kb = static_cast<KeyBlock*>(sp.keys)[static_cast<size_t>(b) * p.num_q_tiles + tile];
    kb.begin[r] = keys.x;
    kb.end[r] = keys.y;
    const int lo = __reduce_min_sync(0xffffffffu, live ? keys.x : INT32_MAX), hi = __reduce_max_sync(0xffffffffu, keys.y);
    const int in_lo = __reduce_max_sync(0xffffffffu, live ? keys.x : INT32_MAX), in_hi = __reduce_min_sync(0xffffffffu, keys.y);
    if ((r & 31) == 0) kb.bounds[r >> 5] = make_int4(lo, hi, in_lo, in_hi);
}

// After a give-up: NaN in this CTA's rows of dK (or of its part) and in the dQ
// rows of iterations [m0, m0 + n), the query tiles [t0, t0 + per_head) of each of
// the key head's query heads in turn.  Other CTAs' reductions keep a NaN.
__device__ __forceinline__ void mark_gradients(const BwdParams& p, const ScoreParams& sp, int d, int b, int hk, int n0,
                                               int split, int t0, int per_head, int64_t m0, int64_t n) {
    const float nan = __int_as_float(0x7fc00000);
    const size_t row = (static_cast<size_t>(b) * p.H_kv + hk) * p.Nk + n0;
    const int keys = min(kBlockK, p.Nk - n0) * d;
    float* part = sp.dk_parts + static_cast<size_t>(split) * p.B * p.H_kv * p.Nk * d + row * d;
    for (int e = threadIdx.x; e < keys; e += blockDim.x) {
        if (p.num_splits > 1)
            part[e] = nan;
        else if (p.grad_bf16)
            static_cast<uint16_t*>(p.dK)[row * d + e] = 0x7fc0;
        else
            static_cast<float*>(p.dK)[row * d + e] = nan;
    }
    for (int64_t m = m0; m < m0 + n; ++m) {
        const int h = hk * p.kv_group + static_cast<int>(m / per_head), r0 = (t0 + static_cast<int>(m % per_head)) * kBwdTile;
        float* dq = p.dQacc + ((static_cast<size_t>(b) * p.H + h) * p.Nq + r0) * d;
        for (int e = threadIdx.x; e < min(kBwdTile, p.Nq - r0) * d; e += blockDim.x) dq[e] = nan;
    }
}

// ---------------------------------------------------------------------------
// CTA = 128 keys; 64-row query tiles.  Warps: 0 copies, 1 TMEM +
// score MMAs, 2-9 recompute/dS (two warpgroups, one key per thread, each taking
// 32 of the tile's 64 query rows), 10-13 dQ^T accumulator -> bulk reduce-add into
// global dQ, 14 gradient MMAs.  TMEM: K1|K2 as the A operand of the score MMAs
// (cols 0-127), S1^T|S2^T (128-255), dK (256-383), dQ^T of the hi|lo halves of dS
// (384-511).
// ---------------------------------------------------------------------------
template <int D, int NST>
struct ScoreKvSmem {
    static constexpr int kKBytes = kBlockK * D * 2;    // 128 keys
    static constexpr int kQBytes = kBwdTile * D * 2;   // 64 query rows of one tensor
    static constexpr int kDsBytes = kBlockK * kBwdTile * 2;
    // Three rings: the trainable side's query tiles (read by the score and the
    // dK MMAs, so freed after dK), the other side's (read by the score MMAs
    // only, so freed right after them: half as deep does), and the per-row
    // constants (freed once the update warps have read them).
    static constexpr int kQt = NST, kQn = NST / 2, kNv = NST >= 8 ? 4 : 2;
    static constexpr int k1 = 0;
    static constexpr int k2 = kKBytes;
    static constexpr int qt = 2 * kKBytes;
    static constexpr int qn = qt + kQt * kQBytes;
    static constexpr int kNumDs = 2;                   // dS buffers (hi + lo each)
    static constexpr int ds = qn + kQn * kQBytes;      // buffer b: hi at ds + 2*b*kDsBytes, lo right after
    // d = 64: a zero 64-feature atom pads the dQ^T MMA's A operand (K_t^T) to M = 128
    static constexpr int zero = ds + 2 * kNumDs * kDsBytes;
    static constexpr int kZeroBytes = D < 128 ? kBlockK * 128 : 0;
    static constexpr int vec = zero + kZeroBytes;      // [kNv][3][64] floats
    static constexpr int keys = vec + kNv * kRowBlockBytes;  // [kNv] KeyBlock
    static constexpr int bars = keys + kNv * static_cast<int>(sizeof(KeyBlock));
    static constexpr int bar_k = bars;
    static constexpr int bar_qtfull = bar_k + 8;
    static constexpr int bar_qtempty = bar_qtfull + 8 * kQt;
    static constexpr int bar_qnfull = bar_qtempty + 8 * kQt;
    static constexpr int bar_qnempty = bar_qnfull + 8 * kQn;
    static constexpr int bar_vfull = bar_qnempty + 8 * kQn;
    static constexpr int bar_vempty = bar_vfull + 8 * kNv;
    static constexpr int bar_sfull = bar_vempty + 8 * kNv;
    static constexpr int bar_sempty = bar_sfull + 8;
    static constexpr int bar_dsfull = bar_sempty + 8;
    static constexpr int bar_dsempty = bar_dsfull + 8 * kNumDs;
    static constexpr int bar_dqfull = bar_dsempty + 8 * kNumDs;
    static constexpr int bar_dqempty = bar_dqfull + 8;
    static constexpr int bar_done = bar_dqempty + 8;
    static constexpr int bar_drain = bar_done + 8;  // the score issuer's own drain on abort
    static constexpr int misc = bar_drain + 8;    // tmem base, abort flag, first and last query tile
    static constexpr int total = misc + 16;
    static constexpr int alloc = total;  // no slack: the kernel checks the base is 1024-byte aligned
};

constexpr int kSbThreads = 480;

template <int D, int NST, int SETTING, int MODE>
__global__ void __launch_bounds__(kSbThreads, 1)
    score_bwd_kernel(const __grid_constant__ CUtensorMap tQ1, const __grid_constant__ CUtensorMap tK1,
                     const __grid_constant__ CUtensorMap tQ2, const __grid_constant__ CUtensorMap tK2,
                     const __grid_constant__ BwdParams p, const __grid_constant__ ScoreParams sp) {
    using L = ScoreKvSmem<D, NST>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // The layout uses every byte it asked for, so the dynamic shared memory
    // base itself must be 1024-byte aligned (128-byte swizzle atoms); if it is
    // not, report it and leave (below) before touching any barrier or tensor memory.
    const uint32_t base = smem_u32(smem_raw);
    uint8_t* gbase = smem_raw;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::misc + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::misc);
    int* tile_span = reinterpret_cast<int*>(gbase + L::misc + 8);
    float* vec = reinterpret_cast<float*>(gbase + L::vec);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kGradWarp = kSbThreads / 32 - 1;  // issues the gradient MMAs

    // Groups of key heads, a few waves of CTAs each, so that resident CTAs share query
    // tiles through L2; in a group the first key tiles of every head, which the most
    // rows see under a causal mask, come first.  (A key head serves kv_group query
    // heads: the CTA visits every query tile of each of them, so dK sums the group's
    // gradients without a second pass.)
    const int unit = blockIdx.x / p.num_splits, split = blockIdx.x - unit * p.num_splits;
    const int2 at = grouped_order(unit, p.num_k_tiles, p.B * p.H_kv, p.order_group);
    const int bkv = at.x, nt = at.y;  // flat (batch, key head), key tile
    const int b = bkv / p.H_kv, hk = bkv - b * p.H_kv;
    const int n0 = nt * kBlockK;
    const uint32_t kt_tile = base + (SETTING == 1 ? L::k2 : L::k1);  // trainable keys
    if (base & 1023u) {
        if (threadIdx.x == 0 && p.status) atomicOr(p.status, kErrSmemAlign);
        mark_gradients(p, sp, D, b, hk, n0, split, 0, p.num_q_tiles, 0, static_cast<int64_t>(p.num_q_tiles) * p.kv_group);
        return;
    }

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tK1);
        prefetch_tensormap(&tK2);
        prefetch_tensormap(&tQ1);
        prefetch_tensormap(&tQ2);
        mbar_init(base + L::bar_k, 1);
        for (int s = 0; s < L::kQt; ++s) {
            mbar_init(base + L::bar_qtfull + 8 * s, 1);
            mbar_init(base + L::bar_qtempty + 8 * s, 1);
        }
        for (int s = 0; s < L::kQn; ++s) {
            mbar_init(base + L::bar_qnfull + 8 * s, 1);
            mbar_init(base + L::bar_qnempty + 8 * s, 1);
        }
        for (int s = 0; s < L::kNv; ++s) {
            mbar_init(base + L::bar_vfull + 8 * s, 1);
            mbar_init(base + L::bar_vempty + 8 * s, 256);
        }
        for (int s = 0; s < L::kNumDs; ++s) {
            mbar_init(base + L::bar_dsfull + 8 * s, 256);
            mbar_init(base + L::bar_dsempty + 8 * s, 1);
        }
        mbar_init(base + L::bar_sfull, 1);
        mbar_init(base + L::bar_sempty, 256);
        mbar_init(base + L::bar_dqfull, 1);
        mbar_init(base + L::bar_dqempty, 128);
        mbar_init(base + L::bar_done, 1);
        mbar_init(base + L::bar_drain, 1);
        *abort_flag = 0;
        tile_span[0] = INT32_MAX;
        tile_span[1] = -1;
        fence_barrier_init();
        fence_proxy_async_smem();
        // the key tiles are on their way while the query tiles are looked up
        mbar_arrive_expect_tx(base + L::bar_k, 2 * L::kKBytes);
#pragma unroll
        for (int c = 0; c < D / kSwizzleCols; ++c) {
            tma_load_4d(base + L::k1 + c * kBlockK * 128, &tK1, base + L::bar_k, c * kSwizzleCols, n0, hk, b);
            tma_load_4d(base + L::k2 + c * kBlockK * 128, &tK2, base + L::bar_k, c * kSwizzleCols, n0, hk, b);
        }
    }
    if (L::kZeroBytes > 0) {
        for (int k = threadIdx.x; k < L::kZeroBytes / 16; k += blockDim.x)
            st_shared_v4(base + L::zero + 16 * k, 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();  // the tensor core reads it through the async proxy
    }
    if (warp == 1) tmem_alloc(base + L::misc, 512);
    // the query tiles with a row that sees one of these keys: from the first to the last of them
    {
        const KeyBlock* blocks = static_cast<const KeyBlock*>(sp.keys) + static_cast<size_t>(b) * p.num_q_tiles;
        int first = INT32_MAX, last = -1;
        for (int t = threadIdx.x; t < p.num_q_tiles; t += kSbThreads) {
            const int4 a = blocks[t].bounds[0], c = blocks[t].bounds[1];
            const int lo = min(a.x, c.x), hi = max(a.y, c.y);
            if (lo < hi && lo - kBlockK < n0 && hi > n0) {
                first = min(first, t);
                last = max(last, t);
            }
        }
        first = __reduce_min_sync(0xffffffffu, first);
        last = __reduce_max_sync(0xffffffffu, last);
        __syncthreads();  // tile_span is set up
        if (lane == 0 && last >= 0) {
            atomicMin(&tile_span[0], first);
            atomicMax(&tile_span[1], last);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wc{abort_flag, p.status, p.wait_ns};
    const int m_start = tile_span[1] >= 0 ? tile_span[0] : 0;
    const int per_head = tile_span[1] - m_start + 1;  // query tiles of one query head that see this key tile
    // this split's share of the key tile's iterations, counted from m0
    const int64_t all_tiles = static_cast<int64_t>(per_head) * p.kv_group;
    const int m0 = static_cast<int>(all_tiles * split / p.num_splits);
    const int n_tiles = static_cast<int>(all_tiles * (split + 1) / p.num_splits) - m0;
    // iteration m -> (query head, query tile)
    auto qhead = [&](int m) { return p.kv_group == 1 ? hk : hk * p.kv_group + (m0 + m) / per_head; };
    auto qtile = [&](int m) { return m_start + (p.kv_group == 1 ? m0 + m : (m0 + m) % per_head); };

    if (warp == 0) {
        // ------------------------------------------------ copies
        if (lane == 0 && n_tiles > 0) {
            const uint64_t keep = policy_evict_last();
            const CUtensorMap* tqt = SETTING == 1 ? &tQ2 : &tQ1;  // the trainable side's queries
            const CUtensorMap* tqn = SETTING == 1 ? &tQ1 : &tQ2;
            const KeyBlock* blocks = static_cast<const KeyBlock*>(sp.keys) + static_cast<size_t>(b) * p.num_q_tiles;
            int n_qt = 0, n_qn = 0, n_v = 0;  // tiles whose copies were issued, per ring
            int st = 0, sn = 0, sv = 0;
            uint32_t pt = 0, pn = 0, pv = 0;
            int h = qhead(0), t = qtile(0);
            for (int m = 0; m < n_tiles; ++m) {
                const int r0 = t * kBwdTile;
                if (!mbar_wait(base + L::bar_qtempty + 8 * st, pt ^ 1, wc, kErrWaitOther)) break;
                const uint32_t fq = base + L::bar_qtfull + 8 * st, dq = base + L::qt + st * L::kQBytes;
                mbar_arrive_expect_tx(fq, L::kQBytes);
#pragma unroll
                for (int c = 0; c < D / kSwizzleCols; ++c)
                    tma_load_4d_hint(dq + c * kBwdTile * 128, tqt, fq, c * kSwizzleCols, r0, h, b, keep);
                ++n_qt;
                if (!mbar_wait(base + L::bar_qnempty + 8 * sn, pn ^ 1, wc, kErrWaitOther)) break;
                const uint32_t fn = base + L::bar_qnfull + 8 * sn, dn = base + L::qn + sn * L::kQBytes;
                mbar_arrive_expect_tx(fn, L::kQBytes);
#pragma unroll
                for (int c = 0; c < D / kSwizzleCols; ++c)
                    tma_load_4d_hint(dn + c * kBwdTile * 128, tqn, fn, c * kSwizzleCols, r0, h, b, keep);
                ++n_qn;
                if (!mbar_wait(base + L::bar_vempty + 8 * sv, pv ^ 1, wc, kErrWaitOther)) break;
                const uint32_t fv = base + L::bar_vfull + 8 * sv;
                mbar_arrive_expect_tx(fv, kRowBlockBytes + static_cast<uint32_t>(sizeof(KeyBlock)));
                const size_t row_block = (static_cast<size_t>(b) * p.H + h) * p.num_q_tiles + t;
                bulk_load(base + L::vec + sv * kRowBlockBytes, sp.rows + row_block * (3 * kBwdTile), kRowBlockBytes, fv);
                bulk_load(base + L::keys + sv * static_cast<uint32_t>(sizeof(KeyBlock)), blocks + t, sizeof(KeyBlock), fv);
                ++n_v;
                if (++st == L::kQt) st = 0, pt ^= 1;
                if (++sn == L::kQn) sn = 0, pn ^= 1;
                if (++sv == L::kNv) sv = 0, pv ^= 1;
                if (++t == m_start + per_head) {
                    t = m_start;
                    ++h;
                }
            }
            // every issued copy has landed (and, unless aborting, been consumed)
            for (int j = max(0, n_qt - L::kQt); j < n_qt; ++j) {
                const uint32_t bo = 8 * (j % L::kQt), ph = (j / L::kQt) & 1;
                drain_wait_b(base + L::bar_qtfull + bo, ph, kDrainNs);
                if (!*abort_flag) drain_wait_b(base + L::bar_qtempty + bo, ph, kDrainNs);
            }
            for (int j = max(0, n_qn - L::kQn); j < n_qn; ++j) {
                const uint32_t bo = 8 * (j % L::kQn), ph = (j / L::kQn) & 1;
                drain_wait_b(base + L::bar_qnfull + bo, ph, kDrainNs);
                if (!*abort_flag) drain_wait_b(base + L::bar_qnempty + bo, ph, kDrainNs);
            }
            for (int j = max(0, n_v - L::kNv); j < n_v; ++j) {
                const uint32_t bo = 8 * (j % L::kNv), ph = (j / L::kNv) & 1;
                drain_wait_b(base + L::bar_vfull + bo, ph, kDrainNs);
                if (!*abort_flag) drain_wait_b(base + L::bar_vempty + bo, ph, kDrainNs);
            }
        }
        if (lane == 0) drain_wait_b(base + L::bar_k, 0, kDrainNs);
    } else if (warp == 1) {
        // ------------------------------------------------ score MMAs
        // Two threads issue the MMAs: this one the scores of tile m, the
        // gradient warp's first thread the dK / dQ^T MMAs of earlier tiles.  A
        // thread waiting on a barrier or committing leaves the tensor pipe to
        // the other's queued work, and neither waits on the other's barriers.
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_bf16_f32(kBlockK, kBwdTile);
            const uint32_t t_k = tmem, t_s = tmem + 128;
            bool started = false;
            // test aid: a wait on a barrier that nothing arrives on before the end
            const bool stalled = p.inject_stall && blockIdx.x == 0 &&
                                 !mbar_wait(base + L::bar_done, 0, wc, kErrWaitOther);
            if (!stalled && n_tiles > 0 && mbar_wait(base + L::bar_k, 0, wc, kErrWaitK)) {
                tc_fence_after();
                // the CTA's key tiles become the A operand of every score MMA
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t ko = (kk >> 2) * kBlockK * 128 + (kk & 3) * 32;
                    tc_cp_128x256b(t_k + kk * 8, smem_desc_k128(base + L::k1 + ko));
                    tc_cp_128x256b(t_k + D / 2 + kk * 8, smem_desc_k128(base + L::k2 + ko));
                }
                started = true;
                // descriptor low words advance by compile-time offsets (the high word is
                // one constant); ring positions are counters rather than divisions
                const uint32_t dhi = smem_desc_hi();
                constexpr uint32_t kSlotLo = L::kQBytes >> 4;
                const uint32_t qt_lo0 = smem_desc_lo_k128(base + L::qt), qn_lo0 = smem_desc_lo_k128(base + L::qn);
                int st = 0, sn = 0;
                uint32_t pt = 0, pn = 0, qt_lo = qt_lo0, qn_lo = qn_lo0;
                for (int m = 0; m < n_tiles; ++m) {
                    if (!mbar_wait(base + L::bar_qtfull + 8 * st, pt, wc, kErrWaitQ)) break;
                    if (!mbar_wait(base + L::bar_qnfull + 8 * sn, pn, wc, kErrWaitQ)) break;
                    if (!mbar_wait(base + L::bar_sempty, (m & 1) ^ 1, wc, kErrWaitS)) break;
                    tc_fence_after();
                    const uint32_t q1_lo = SETTING == 1 ? qn_lo : qt_lo, q2_lo = SETTING == 1 ? qt_lo : qn_lo;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t qo = ((kk >> 2) * kBwdTile * 128 + (kk & 3) * 32) >> 4;
                        tc_mma_bf16_ta_w(t_s, t_k + kk * 8, q1_lo + qo, dhi, id_s, kk > 0);
                    }
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t qo = ((kk >> 2) * kBwdTile * 128 + (kk & 3) * 32) >> 4;
                        tc_mma_bf16_ta_w(t_s + 64, t_k + D / 2 + kk * 8, q2_lo + qo, dhi, id_s, kk > 0);
                    }
                    tc_commit(base + L::bar_sfull);
                    tc_commit(base + L::bar_qnempty + 8 * sn);  // the other side's tile is done with
                    if (++st == L::kQt) {
                        st = 0;
                        pt ^= 1;
                        qt_lo = qt_lo0;
                    } else {
                        qt_lo += kSlotLo;
                    }
                    if (++sn == L::kQn) {
                        sn = 0;
                        pn ^= 1;
                        qn_lo = qn_lo0;
                    } else {
                        qn_lo += kSlotLo;
                    }
                }
            }
            if (*abort_flag && started) {  // let the issued copies and MMAs retire before TMEM is freed
                tc_commit(base + L::bar_drain);
                drain_wait_b(base + L::bar_drain, 0, kDrainNs);
            }
        }
    } else if (warp == kGradWarp) {
        // ------------------------------------------------ gradient MMAs
        // tile m's dS (from the update warps) -> dK += dS^T Q_t, and
        // [dQ^T_hi | dQ^T_lo] = K_t^T [dS^T_hi | dS^T_lo]; then the tile's dS buffer
        // and query stage are released.  (Tile m's scores finished before its dS
        // existed, so these commits also cover the score MMAs that read the stage.)
        if (lane == 0) {
            constexpr uint32_t id_dk = idesc_bf16_f32(kBlockK, D, 0, 1);
            constexpr uint32_t id_dq = idesc_bf16_f32(128, 2 * kBwdTile, 1, 1);  // M = 128 features (d = 64: padded)
            // A = K_t^T as 64-feature atoms: the tile's second block, or the zero atom when d = 64
            const uint32_t a_atom = D == 128 ? kBlockK * 128 : base + L::zero - kt_tile;
            const uint32_t t_dk = tmem + 256, t_dq = tmem + 384;
            const uint32_t dhi = smem_desc_hi();
            constexpr uint32_t kSlotLo = L::kQBytes >> 4, kDsLo = (2 * L::kDsBytes) >> 4;
            const uint32_t qt_lo0 = smem_desc_lo_mn128(base + L::qt, kBwdTile * 128);
            const uint32_t ds_lo0 = smem_desc_lo_k128(base + L::ds);
            const uint32_t dsmn_lo0 = smem_desc_lo_mn128(base + L::ds, L::kDsBytes);
            const uint32_t kt_lo = smem_desc_lo_mn128(kt_tile, a_atom);
            int issued = 0, s2 = 0, dsb = 0;
            uint32_t dsph = 0, qt_lo = qt_lo0;
            // the key tiles (A of dQ^T) have landed before any dS exists; the wait states it
            if (n_tiles > 0 && mbar_wait(base + L::bar_k, 0, wc, kErrWaitK)) {
                for (int m = 0; m < n_tiles; ++m) {
                    if (!mbar_wait(base + L::bar_dsfull + 8 * dsb, dsph, wc, kErrWaitOther)) break;
                    tc_fence_after();
                    const uint32_t ds_lo = ds_lo0 + (dsb ? kDsLo : 0u);
                    // dK += dS^T Q_t : A = dS^T (K-major over queries), B = Q_t (MN-major); dS = hi + lo
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int kk = 0; kk < kBwdTile / 16; ++kk)
                            tc_mma_bf16_w(t_dk, ds_lo + ((part * L::kDsBytes + kk * 32) >> 4), dhi,
                                          qt_lo + ((kk * 16 * 128) >> 4), dhi, id_dk, (kk | part | m) != 0);
                    {
                        // A = K_t (MN-major), B = the hi and lo tiles as two 64-query atoms of one
                        // N = 128 operand, K = 128 keys
                        if (!mbar_wait(base + L::bar_dqempty, (m & 1) ^ 1, wc, kErrWaitOther)) break;
                        tc_fence_after();
                        const uint32_t dsmn_lo = dsmn_lo0 + (dsb ? kDsLo : 0u);
#pragma unroll
                        for (int kk = 0; kk < kBlockK / 16; ++kk)
                            tc_mma_bf16_w(t_dq, kt_lo + ((kk * 16 * 128) >> 4), dhi, dsmn_lo + ((kk * 16 * 128) >> 4),
                                          dhi, id_dq, kk > 0);
                        tc_commit(base + L::bar_dqfull);
                    }
                    tc_commit(base + L::bar_dsempty + 8 * dsb);
                    tc_commit(base + L::bar_qtempty + 8 * s2);
                    dsph ^= dsb;  // a buffer's phase flips each time it comes round again
                    dsb ^= 1;
                    if (++s2 == L::kQt) {
                        s2 = 0;
                        qt_lo = qt_lo0;
                    } else {
                        qt_lo += kSlotLo;
                    }
                    ++issued;
                }
                if (issued == n_tiles) tc_commit(base + L::bar_done);
            }
            if (*abort_flag && issued > 0) {  // let the issued MMAs retire before TMEM is freed
                tc_commit(base + L::bar_done);
                drain_wait_b(base + L::bar_done, 0, kDrainNs);
            }
        }
    } else if (warp < 10) {
        // ------------------------------------------------ recompute + dS^T
        // Two warpgroups: warps 2-5 take query rows 0-31 of every tile, warps
        // 6-9 rows 32-63; one key per thread.
        const int wg = (warp - 2) >> 2;
        const int wq = warp & 3;
        const int row = wq * 32 + lane;
        const int j = n0 + row;  // key index
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float c = p.scale_log2e;
        const float2 cc = make_float2(c, c), sc2 = make_float2(p.scale, p.scale);
        const bool key_ok = j < p.Nk;
        bool ok = true;
        for (int m = 0; m < n_tiles; ++m) {
            const int sv = m % L::kNv;
            if (!wait_all(base + L::bar_sfull, m & 1, wc, kErrWaitS) ||
                !wait_all(base + L::bar_vfull + 8 * sv, (m / L::kNv) & 1, wc, kErrWaitQ)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int r0 = qtile(m) * kBwdTile + wg * 32;  // first query row of this chunk
            const uint32_t t1 = tl + 128 + wg * 32, t2 = t1 + 64;
            const int dsb = m % L::kNumDs;
            const uint32_t dss = base + L::ds + 2 * dsb * L::kDsBytes;
            float z1[32], z2[32];
            tmem_ld32(t1, z1);
            tmem_ld32(t2, z2);
            tc_wait_ld();
            tc_fence_before();
            mbar_arrive(base + L::bar_sempty);  // the next score tile may overwrite S now
            const KeyBlock& kb = reinterpret_cast<const KeyBlock*>(gbase + L::keys)[sv];
            const int4 bounds = kb.bounds[wg];
            const bool whole = bounds.z <= n0 && bounds.w >= n0 + kBlockK;  // every row sees every key
            // bit e: query row r0 + e sees this thread's key
            uint32_t vis = 0xffffffffu;
            bool bad = false;
            if (!whole) {
                vis = 0u;
                const int4* lo4 = reinterpret_cast<const int4*>(kb.begin + wg * 32);
                const int4* hi4 = reinterpret_cast<const int4*>(kb.end + wg * 32);
#pragma unroll
                for (int e4 = 0; e4 < 8; ++e4) {
                    const int4 lo = lo4[e4], hi = hi4[e4];
                    const int los[4] = {lo.x, lo.y, lo.z, lo.w}, his[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int e = 4 * e4 + k;
                        if (j >= los[k] && j < his[k]) {
                            vis |= 1u << e;
                        } else {
                            bad |= !(fabsf(SETTING == 1 ? z2[e] : z1[e]) < INFINITY);
                            z1[e] = z2[e] = 0.f;  // no effect on the form of cap_scores
                        }
                    }
                }
            }
            cap_scores<MODE>(z1, z2, sp.side[0], sp.side[1]);
            float sl1 = 0.f, sl2 = 0.f, d0 = 0.f;
            if (MODE == kScoreBias) {
                const int h = qhead(m);
                if (sp.side[0].slopes) sl1 = -kLog2e * sp.side[0].slopes[h];
                if (sp.side[1].slopes) sl2 = -kLog2e * sp.side[1].slopes[h];
                d0 = static_cast<float>(row_position(sp, p.Nq, p.Nk, b, r0) - j);
            }
            // per-query constants of this chunk: 128-bit broadcast loads
            const float4* v4 = reinterpret_cast<const float4*>(vec + sv * 3 * kBwdTile + wg * 32);
            float dsv[32];
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
                const float4 a = v4[e4], x = v4[kBwdTile / 4 + e4], gg = v4[kBwdTile / 2 + e4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int e = 4 * e4 + 2 * k;
                    const float2 nla = k ? make_float2(a.z, a.w) : make_float2(a.x, a.y);
                    const float2 nxb = k ? make_float2(x.z, x.w) : make_float2(x.x, x.y);
                    const float2 gs = k ? make_float2(gg.z, gg.w) : make_float2(gg.x, gg.y);
                    const float2 u1 = make_float2(z1[e], z1[e + 1]), u2 = make_float2(z2[e], z2[e + 1]);
                    float2 d;
                    if (MODE == kScorePlain) {
                        d = dscore2<SETTING>(u1, u2, cc, sc2, nla, nxb, gs);
                    } else {
                        float2 x1 = u1, x2 = u2;
                        if (MODE == kScoreBias) {
                            const float2 away = make_float2(fabsf(d0 + static_cast<float>(e)),
                                                            fabsf(d0 + static_cast<float>(e + 1)));
                            x1 = __ffma2_rn(away, splat(sl1), x1);
                            x2 = __ffma2_rn(away, splat(sl2), x2);
                        }
                        // dS, then the slope of the cap 1 - tanh^2, tanh = x / lim before the bias
                        d = dscore2<SETTING>(x1, x2, splat(1.f), splat(kLn2), nla, nxb, gs);
                        const float2 th = __fmul2_rn(SETTING == 1 ? u2 : u1, splat(sp.side[SETTING == 1].inv_lim));
                        d = __fmul2_rn(d, __ffma2_rn(th, make_float2(-th.x, -th.y), splat(1.f)));
                    }
                    dsv[e] = d.x;
                    dsv[e + 1] = d.y;
                }
            }
            mbar_arrive(base + L::bar_vempty + 8 * sv);  // this tile's row constants are read
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (!((vis >> e) & 1u)) dsv[e] = 0.f;
                // A zero dS does not hide a NaN or an infinity in the operand it meets in the
                // gradient MMAs: rows with one, of either operand, become zero rows (where such a
                // row is visible, dS is NaN and the gradient with it).
                if (__any_sync(0xffffffffu, bad))
                    clear_nonfinite<D>(base + L::qt + (m % L::kQt) * L::kQBytes, wg * 32, kt_tile, row, lane);
            }
            if (!wait_all(base + L::bar_dsempty + 8 * dsb, ((m / L::kNumDs) & 1) ^ 1, wc, kErrWaitOther)) {
                ok = false;
                break;
            }
            store_ds_chunk(dss, dss + L::kDsBytes, row, wg * 4, dsv);
            fence_proxy_async_smem();
            mbar_arrive(base + L::bar_dsfull + 8 * dsb);
        }
        // epilogue: dK row = scale * accumulator; each warpgroup writes half the columns
        if (ok && (n_tiles == 0 || wait_all(base + L::bar_done, 0, wc, kErrWaitOther))) {
            tc_fence_after();
            // one split: the output; several: this split's float32 part of it, summed by score_finish_kernel
            const size_t at_row = static_cast<size_t>(bkv) * p.Nk + j;
            const bool parts = p.num_splits > 1, bf16 = !parts && p.grad_bf16 != 0;
            void* out = parts ? static_cast<void*>(sp.dk_parts + (static_cast<size_t>(split) * p.B * p.H_kv * p.Nk + at_row) * D)
                              : static_cast<void*>(reinterpret_cast<uint8_t*>(p.dK) + at_row * D * (bf16 ? 2 : 4));
#pragma unroll 1
            for (int c0 = wg * (D / 2); c0 < (wg + 1) * (D / 2); c0 += 32) {
                float v[32];
                tmem_ld32(tl + 256 + c0, v);
                tc_wait_ld();
                if (n_tiles == 0) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;  // no row sees these keys: nothing was accumulated
                }
                if (key_ok) store_grad32(out, c0, v, 1.0f, bf16);  // the scale is in dS
            }
        }
    } else {
        // ------------------------------------------------ dQ^T -> bulk L2 reduction into dQ
        // Each tile's 64 x d float32 block of dQ is staged in shared memory as
        // 64 contiguous rows (the non-trainable key tile's space: that tile
        // only fed the copy into tensor memory) and added to global dQ by bulk
        // reduce-adds, one per 32-row half, so that staging one half overlaps
        // the reduction still reading the other.
        const int wq = warp & 3;
        const int f = wq * 32 + lane;  // feature = TMEM lane
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t stage = base + (SETTING == 1 ? L::k1 : L::k2);
        const bool leader = warp == 10 && lane == 0;
        bool other_pending = false;  // the last bulk group issued was the other half's
        for (int m = 0; m < n_tiles; ++m) {
            // the four epilogue warps decide together, so none is left at a named barrier
            if (!bar_sync_and(3, 128, wait_all(base + L::bar_dqfull, m & 1, wc, kErrWaitOther))) break;
            tc_fence_after();
            float v0[32], v1[32];
            if (wq * 32 < D) {  // d = 64: TMEM lanes 64-127 hold the zero padding
                tmem_ld32(tl + 384, v0);  // hi, query rows 0-31
                tmem_ld32(tl + 416, v1);  // and 32-63
                tc_wait_ld();
                float lo[32];
                tmem_ld32(tl + 448, lo);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 t = __fadd2_rn(make_float2(v0[e], v0[e + 1]), make_float2(lo[e], lo[e + 1]));
                    v0[e] = t.x;
                    v0[e + 1] = t.y;
                }
                tmem_ld32(tl + 480, lo);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 t = __fadd2_rn(make_float2(v1[e], v1[e + 1]), make_float2(lo[e], lo[e + 1]));
                    v1[e] = t.x;
                    v1[e + 1] = t.y;
                }
            }
            tc_fence_before();
            mbar_arrive(base + L::bar_dqempty);
            const int r0 = qtile(m) * kBwdTile;
            const int nrow = min(kBwdTile, p.Nq - r0);
            float* dst = p.dQacc + ((static_cast<size_t>(b) * p.H + qhead(m)) * p.Nq + r0) * D;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t sh = stage + hf * 32 * (D * 4);
                // the reduction that last read this half has finished reading; when the
                // other half's reduction was the last one issued it may still run
                if (leader) {
                    if (other_pending)
                        bulk_wait_read_1();
                    else
                        bulk_wait_read_all();
                }
                asm volatile("bar.sync 2, 128;" ::: "memory");
                if (f < D) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(sh + e * (D * 4) + f * 4), "f"(hf ? v1[e] : v0[e])
                                     : "memory");
                }
                fence_proxy_async_smem();
                asm volatile("bar.sync 2, 128;" ::: "memory");
                const int rows = min(32, nrow - 32 * hf);
                other_pending = rows > 0;
                if (leader && rows > 0) {
                    bulk_reduce_add_f32(dst + hf * 32 * D, sh, static_cast<uint32_t>(rows * D * 4));
                    bulk_commit();
                }
            }
        }
        if (leader) bulk_wait_all();  // every reduction has landed before the CTA exits
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (*abort_flag) mark_gradients(p, sp, D, b, hk, n0, split, m_start, per_head, m0, n_tiles);
}

// 8 elements of dQ (float32 -> bf16, when asked for) or of dK (the sum of its
// splits' parts, in order) per thread and step.
__global__ void __launch_bounds__(256) score_finish_kernel(const float4* dq, uint4* dq_out, size_t nq8, const float4* dk_parts,
                                                           void* dk_out, size_t nk8, int splits, bool bf16) {
    for (size_t k = blockIdx.x * size_t(blockDim.x) + threadIdx.x; k < nq8 + nk8; k += size_t(gridDim.x) * blockDim.x) {
        if (k < nq8) {
            const float4 a = dq[2 * k], b = dq[2 * k + 1];
            dq_out[k] = make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
            continue;
        }
        const size_t e = k - nq8;
        float4 a = dk_parts[2 * e], b = dk_parts[2 * e + 1];
        for (int s = 1; s < splits; ++s) {
            const float4 u = dk_parts[2 * (s * nk8 + e)], v = dk_parts[2 * (s * nk8 + e) + 1];
            a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
            b.x += v.x, b.y += v.y, b.z += v.z, b.w += v.w;
        }
        if (bf16) {
            static_cast<uint4*>(dk_out)[e] =
                make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
        } else {
            static_cast<float4*>(dk_out)[2 * e] = a;
            static_cast<float4*>(dk_out)[2 * e + 1] = b;
        }
    }
}

template <int D, int SETTING, int MODE>
cudaError_t launch_impl(const CUtensorMap* m, const BwdParams& p, const ScoreParams& sp, int ctas, cudaStream_t st) {
    constexpr int NST = D == 128 ? 4 : 8;  // trainable-side query ring; the other side's is half as deep
    constexpr int bytes = ScoreKvSmem<D, NST>::alloc;
    static_assert(bytes <= 232448, "shared memory");
    auto k = score_bwd_kernel<D, NST, SETTING, MODE>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k<<<ctas, kSbThreads, bytes, st>>>(m[0], m[1], m[2], m[3], p, sp);
    return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_mode(int d, int setting, const CUtensorMap* m, const BwdParams& p, const ScoreParams& sp, int ctas,
                        cudaStream_t st) {
    if (d == 128)
        return setting == 1 ? launch_impl<128, 1, MODE>(m, p, sp, ctas, st) : launch_impl<128, 2, MODE>(m, p, sp, ctas, st);
    return setting == 1 ? launch_impl<64, 1, MODE>(m, p, sp, ctas, st) : launch_impl<64, 2, MODE>(m, p, sp, ctas, st);
}

}  // namespace

size_t score_bwd_row_bytes(int64_t bh, int q_tiles) { return static_cast<size_t>(bh) * q_tiles * kRowBlockBytes; }
size_t score_bwd_key_bytes(int64_t batch, int q_tiles) { return static_cast<size_t>(batch) * q_tiles * sizeof(KeyBlock); }

cudaError_t launch_score_bwd(int d, int setting, int mode, const CUtensorMap* maps, const BwdParams& p,
                             const ScoreParams& sp, int ctas, int sms, cudaStream_t stream) {
    score_prepare_kernel<<<static_cast<unsigned>(p.B * p.H) * p.num_q_tiles, 256, 0, stream>>>(p, sp, setting, d);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = mode == kScorePlain     ? launch_mode<kScorePlain>(d, setting, maps, p, sp, ctas, stream)
        : mode == kScoreBounded ? launch_mode<kScoreBounded>(d, setting, maps, p, sp, ctas, stream)
        : mode == kScoreGeneral ? launch_mode<kScoreGeneral>(d, setting, maps, p, sp, ctas, stream)
                                : launch_mode<kScoreBias>(d, setting, maps, p, sp, ctas, stream);
    const bool parts = p.num_splits > 1;
    if (e != cudaSuccess || !(parts || p.grad_bf16)) return e;
    const size_t nq8 = p.grad_bf16 ? static_cast<size_t>(p.B) * p.H * p.Nq * d / 8 : 0;
    const size_t nk8 = parts ? static_cast<size_t>(p.B) * p.H_kv * p.Nk * d / 8 : 0;
    const size_t blocks = std::min<size_t>((nq8 + nk8 + 255) / 256, static_cast<size_t>(sms) * 16);
    score_finish_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        reinterpret_cast<const float4*>(p.dQacc), static_cast<uint4*>(p.dQ), nq8,
        reinterpret_cast<const float4*>(sp.dk_parts), p.dK, nk8, p.num_splits, p.grad_bf16 != 0);
    return cudaGetLastError();
}

}  // namespace streamkl
