// attn_bwd.cu -- gradients of the attention over whole prompts on sm_103a.
//
//   P = exp(S - LSE),  dV = P^T dO,  dP = dO V^T,  D_i = sum(dO_i O_i)
//   dS = scale P (dP - D),  dQ = dS K,  dK = dS^T Q
//
// One key-tile kernel: 128 keys per CTA, the 64-row query tiles that see any of
// them streamed through, of every query head of the key head; dK and dV stay in
// tensor memory, dQ is added to float32 in L2 by bulk reductions.  Row constants
// and key ranges are prepared by a first kernel.
//
// P enters dV rounded to bf16; dS enters dQ and dK as two bf16 terms.  A row's dS sum
// to zero, and so what its keys have in common cancels in dQ; one term's roundings
// (2^-8 of each dS) do not.  For dQ the MMA that takes both terms as one operand of
// twice the columns takes as long as with one.  D is a product with O and what its
// rounding left (`rest`), for the same reason: an error of D is a multiple of the
// row's mean key in dQ.
//
// A zero P or dS does not hide a NaN or an infinity in the operand that it meets in an MMA.
// Rows that see none of such a token must not get it: keys that hold one become zero rows
// before the first gradient MMA, query rows in tiles where somebody does not see them.
// Where they are seen, P and dS are NaN, or dQ gets its NaN apart.
//
// Bound by the tensor core: the issuing thread never waits for more than a barrier's own
// latency, and is held back by 36 MMAs a tile of 65 to 82 cycles each, 2600 of about 3200.
// The scores' have N = 64 and take 73, no less than those with N = 128 (d = 64: 28 MMAs,
// 2100 of 2830 cycles, with half the operations).  8192 causal rows, 32 heads on 8,
// d = 128: 1575 us, 873 TFLOP/s of the five products, and 56 + 27 us for the first and the
// last kernel, which are bound by HBM (without the search for tokens that are not finite, whose
// registers spill 24 bytes: 1568 and 55).  Reductions into dQ out of registers, without the
// stage in shared memory, took 1660 us for the three where these take 1653 (d = 64: 1524,
// 1420).  128-row query tiles, with P and dS as operands in
// tensor memory and dQ in dP's place there, took 3357 us: no space is left for a second tile,
// and the steps of one stand in a chain.
#include <algorithm>

#include "attn.cuh"
#include "bwd_common.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "ptx.cuh"
#include "score.cuh"

namespace streamkl {

namespace {

constexpr int kAbRowBytes = 2 * kBwdTile * 4;  // a tile's row constants

// One block per (64-row query tile, batch and head), a warp per row at a time: the
// row's constants, the ranges of the tile (the first head's block) and zeros in its
// rows of dQ.  A row that sees no key gets zero constants; an infinite LSE (from an
// infinite score) counts as NaN, as in its own softmax, and so does the LSE of a row
// whose dO has a NaN or an infinity: the key-tile kernel may clear that row of dO, and
// its P has to carry it into dV.
template <int D>
__global__ void __launch_bounds__(256) attn_prepare_kernel(const __grid_constant__ AttnBwdParams p,
                                                           const __grid_constant__ ScoreParams sp) {
    const size_t block = blockIdx.x;
    const int bh = static_cast<int>(block / p.num_q_tiles), tile = static_cast<int>(block - static_cast<size_t>(bh) * p.num_q_tiles);
    const int b = bh / p.H, h = bh - b * p.H, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = min(kBwdTile, p.Nq - tile * kBwdTile);
    float4* dq = reinterpret_cast<float4*>(p.dQacc + (static_cast<size_t>(bh) * p.Nq + tile * kBwdTile) * D);
    for (int k = threadIdx.x; k < rows * D / 4; k += blockDim.x) dq[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    // a half warp per row, D / 16 values a lane
    constexpr int W = D / 32;  // words of two
    float* out = p.rows + block * (2 * kBwdTile);
    const int half = lane >> 4, at = (lane & 15) * (D / 16);
    float sums[4];
    bool broken[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = 8 * warp + 2 * k + half, i = tile * kBwdTile + r;
        float s = 0.f;
        bool found = false;
        if (i < p.Nq) {
            const uint32_t* g = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.dO) + (b * p.g_b + h * p.g_h + i * p.g_n) + at);
            const uint32_t* o = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.O) + (b * p.o_b + h * p.o_h + i * p.o_n) + at);
            const uint32_t* e = p.rest ? reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.rest) + (static_cast<size_t>(bh) * p.Nq + i) * D + at) : nullptr;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const uint32_t ug = g[w], uo = o[w], ue = e ? e[w] : 0u;
                found |= has_nonfinite_bf16(ug);
                s = fmaf(__uint_as_float(ug << 16), __uint_as_float(uo << 16) + __uint_as_float(ue << 16), s);
                s = fmaf(__uint_as_float(ug & 0xffff0000u), __uint_as_float(uo & 0xffff0000u) + __uint_as_float(ue & 0xffff0000u), s);
            }
        }
        sums[k] = s;
        broken[k] = (__ballot_sync(0xffffffffu, found) >> (lane & 16) & 0xffffu) != 0u;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sums[k] += __shfl_xor_sync(0xffffffffu, sums[k], o);
        const int r = 8 * warp + 2 * k + half, i = tile * kBwdTile + r;
        if ((lane & 15) == 0) {
            const int2 keys = row_range(sp, p.Nq, p.Nk, b, i);
            float nl = 0.f, nd = 0.f;
            if (keys.x < keys.y) {
                const float l = p.LSE[static_cast<size_t>(bh) * p.Nq + i];
                nl = fabsf(l) < INFINITY && !broken[k] ? -l * kLog2e : __int_as_float(0x7fc00000);
                nd = -p.scale * sums[k];
            }
            out[r] = nl;
            out[kBwdTile + r] = nd;
        }
    }
    if (h != 0 || threadIdx.x >= kBwdTile) return;
    const int r = threadIdx.x;
    const int2 keys = row_range(sp, p.Nq, p.Nk, b, tile * kBwdTile + r);
    const bool live = keys.x < keys.y;
    KeyBlock& kb = static_cast<KeyBlock*>(p.keys)[static_cast<size_t>(b) * p.num_q_tiles + tile];
    kb.begin[r] = keys.x;
    kb.end[r] = keys.y;
    const int lo = __reduce_min_sync(0xffffffffu, live ? keys.x : INT32_MAX), hi = __reduce_max_sync(0xffffffffu, keys.y);
    const int in_lo = __reduce_max_sync(0xffffffffu, live ? keys.x : INT32_MAX), in_hi = __reduce_min_sync(0xffffffffu, keys.y);
    if ((r & 31) == 0) kb.bounds[r >> 5] = make_int4(lo, hi, in_lo, in_hi);
}

// After a give-up: NaN in this CTA's rows of dK and dV (or of its parts) and in the
// dQ rows of iterations [m0, m0 + n), the query tiles [t0, t0 + per_head) of each of
// the key head's query heads in turn.  Other CTAs' reductions keep a NaN.
__device__ __noinline__ void mark_attn_gradients(const AttnBwdParams& p, int d, int b, int hk, int n0, int split, int t0,
                                                 int per_head, int64_t m0, int64_t n) {
    const float nan = __int_as_float(0x7fc00000);
    const size_t row = (static_cast<size_t>(b) * p.H_kv + hk) * p.Nk + n0, all = static_cast<size_t>(p.B) * p.H_kv * p.Nk * d;
    const int keys = min(kBlockK, p.Nk - n0) * d;
    for (int e = threadIdx.x; e < keys; e += blockDim.x) {
        if (p.num_splits > 1) {
            p.parts[split * all + row * d + e] = nan;
            p.parts[(p.num_splits + split) * all + row * d + e] = nan;
        } else {
            static_cast<uint16_t*>(p.dK)[row * d + e] = 0x7fc0;
            static_cast<uint16_t*>(p.dV)[row * d + e] = 0x7fc0;
        }
    }
    for (int64_t m = m0; m < m0 + n; ++m) {
        const int h = hk * p.group + static_cast<int>(m / per_head), r0 = (t0 + static_cast<int>(m % per_head)) * kBwdTile;
        float* dq = p.dQacc + ((static_cast<size_t>(b) * p.H + h) * p.Nq + r0) * d;
        for (int e = threadIdx.x; e < min(kBwdTile, p.Nq - r0) * d; e += blockDim.x) dq[e] = nan;
    }
}

// ---------------------------------------------------------------------------
// CTA = 128 keys; 64-row query tiles.  Warps: 0 copies, 1 TMEM + the MMAs, 2-9 P and
// dS (two warpgroups, one key per thread, each taking 32 of the tile's 64 query
// rows), 10-13 dQ^T accumulator -> bulk reduce-add into global dQ.  TMEM: S^T | dP^T (cols 0-127), dK (128-255), dV (256-383), dQ^T
// of the hi | lo halves of dS (384-511).
// ---------------------------------------------------------------------------
template <int D>
struct AttnKvSmem {
    static constexpr int kKBytes = kBlockK * D * 2;    // 128 keys
    static constexpr int kQBytes = kBwdTile * D * 2;   // 64 query rows
    static constexpr int kDsBytes = kBlockK * kBwdTile * 2;
    static constexpr int kStageBytes = 32 * D * 4;     // 32 rows of dQ
    static constexpr int kNst = D == 128 ? 3 : 6;      // query and dO tiles
    static constexpr int kNv = 2;                      // row constants and key ranges
    static constexpr int k = 0;
    static constexpr int v = kKBytes;
    static constexpr int q = 2 * kKBytes;
    static constexpr int g = q + kNst * kQBytes;       // dO
    static constexpr int ds = g + kNst * kQBytes;      // hi, lo
    static constexpr int pt = ds + 2 * kDsBytes;       // P^T
    static constexpr int stage = pt + kDsBytes;
    // d = 64: a zero 64-feature atom pads the dQ^T MMA's A operand (K^T) to M = 128
    static constexpr int zero = stage + kStageBytes;
    static constexpr int kZeroBytes = D < 128 ? kBlockK * 128 : 0;
    static constexpr int vec = zero + kZeroBytes;      // [kNv][2][64] floats
    static constexpr int keys = vec + kNv * kAbRowBytes;  // [kNv] KeyBlock
    static constexpr int bar_k = keys + kNv * static_cast<int>(sizeof(KeyBlock));
    static constexpr int bar_full = bar_k + 8;         // [kNst]
    static constexpr int bar_empty = bar_full + 8 * kNst;
    static constexpr int bar_vfull = bar_empty + 8 * kNst;
    static constexpr int bar_vempty = bar_vfull + 8 * kNv;
    static constexpr int bar_sfull = bar_vempty + 8 * kNv;
    static constexpr int bar_sempty = bar_sfull + 8;
    static constexpr int bar_dsfull = bar_sempty + 8;
    static constexpr int bar_dsempty = bar_dsfull + 8;
    static constexpr int bar_dqfull = bar_dsempty + 8;
    static constexpr int bar_dqempty = bar_dqfull + 8;
    static constexpr int bar_done = bar_dqempty + 8;
    static constexpr int bar_drain = bar_done + 8;     // the issuer's own drain on abort
    static constexpr int misc = bar_drain + 8;         // tmem base, abort flag, first and last query tile
    static constexpr int alloc = misc + 16;            // no slack: the kernel checks the base is 1024-byte aligned
};

constexpr int kAbThreads = 448;

// Whether key `row` of the 128-key tile at `kt` holds a NaN or an infinity.
template <int D>
__device__ __forceinline__ bool key_row_broken(const uint8_t* kt, int row) {
    bool found = false;
#pragma unroll
    for (int c = 0; c < D / kSwizzleCols; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint4 u = *reinterpret_cast<const uint4*>(kt + c * kBlockK * 128 + row * 128 + ((k ^ (row & 7)) << 4));
            found |= has_nonfinite_bf16(u.x) | has_nonfinite_bf16(u.y) | has_nonfinite_bf16(u.z) | has_nonfinite_bf16(u.w);
        }
    return found;
}

// NaN in the features that are not finite in the broken key j, of the dQ rows of the wg-th halves of iterations
// [m0, m0 + n) (see mark_attn_gradients) that see it: what a dS of 0 times it is, without what the tile's other rows
// would get of it from the MMA.
__device__ __noinline__ void poison_rows(const AttnBwdParams& p, int d, int b, int hk, int j, int wg, int t0, int per_head, int m0, int n) {
    const uint16_t* key = static_cast<const uint16_t*>(p.K) + (b * p.k_b + hk * p.k_h + static_cast<int64_t>(j) * p.k_n);
    const KeyBlock* blocks = static_cast<const KeyBlock*>(p.keys) + static_cast<size_t>(b) * p.num_q_tiles;
    for (int m = m0; m < m0 + n; ++m) {
        const int h = hk * p.group + m / per_head, t = t0 + m % per_head;
        for (int r = 32 * wg; r < 32 * wg + 32; ++r) {
            if (j < blocks[t].begin[r] || j >= blocks[t].end[r]) continue;
            float* dq = p.dQacc + ((static_cast<size_t>(b) * p.H + h) * p.Nq + t * kBwdTile + r) * d;
            for (int f = 0; f < d; ++f)
                if (has_nonfinite_bf16(key[f])) red_add_f32(dq + f, __int_as_float(0x7fc00000));
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kAbThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
                    const __grid_constant__ CUtensorMap tV, const __grid_constant__ CUtensorMap tG,
                    const __grid_constant__ AttnBwdParams p) {
    using L = AttnKvSmem<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    uint8_t* gbase = smem_raw;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::misc + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::misc);
    int* tile_span = reinterpret_cast<int*>(gbase + L::misc + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // groups of key heads, a few waves of CTAs each, so that resident CTAs share query tiles through L2; in a
    // group the first key tiles of every head, which the most rows see under a causal mask, come first
    const int unit = blockIdx.x / p.num_splits, split = blockIdx.x - unit * p.num_splits;
    const int2 at = grouped_order(unit, p.num_k_tiles, p.B * p.H_kv, p.order_group);
    const int bkv = at.x, b = bkv / p.H_kv, hk = bkv - b * p.H_kv, n0 = at.y * kBlockK;
    if (base & 1023u) {
        if (threadIdx.x == 0 && p.status) atomicOr(p.status, kErrSmemAlign);
        mark_attn_gradients(p, D, b, hk, n0, split, 0, p.num_q_tiles, 0, static_cast<int64_t>(p.num_q_tiles) * p.group);
        return;
    }

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tK);
        prefetch_tensormap(&tV);
        prefetch_tensormap(&tQ);
        prefetch_tensormap(&tG);
        mbar_init(base + L::bar_k, 1);
        for (int s = 0; s < L::kNst; ++s) {
            mbar_init(base + L::bar_full + 8 * s, 1);
            mbar_init(base + L::bar_empty + 8 * s, 1);
        }
        for (int s = 0; s < L::kNv; ++s) {
            mbar_init(base + L::bar_vfull + 8 * s, 1);
            mbar_init(base + L::bar_vempty + 8 * s, 256);
        }
        mbar_init(base + L::bar_dsfull, 256);
        mbar_init(base + L::bar_dsempty, 1);
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
        // the key and value tiles are on their way while the query tiles are looked up
        mbar_arrive_expect_tx(base + L::bar_k, 2 * L::kKBytes);
#pragma unroll
        for (int c = 0; c < D / kSwizzleCols; ++c) {
            tma_load_4d(base + L::k + c * kBlockK * 128, &tK, base + L::bar_k, c * kSwizzleCols, n0, hk, b);
            tma_load_4d(base + L::v + c * kBlockK * 128, &tV, base + L::bar_k, c * kSwizzleCols, n0, hk, b);
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
        const KeyBlock* blocks = static_cast<const KeyBlock*>(p.keys) + static_cast<size_t>(b) * p.num_q_tiles;
        int first = INT32_MAX, last = -1;
        for (int t = threadIdx.x; t < p.num_q_tiles; t += kAbThreads) {
            const int4 x = blocks[t].bounds[0], y = blocks[t].bounds[1];
            const int lo = min(x.x, y.x), hi = max(x.y, y.y);
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
    const int64_t all_tiles = static_cast<int64_t>(per_head) * p.group;
    const int m0 = static_cast<int>(all_tiles * split / p.num_splits);
    const int n_tiles = static_cast<int>(all_tiles * (split + 1) / p.num_splits) - m0;
    // iteration m -> (query head, query tile)
    auto qhead = [&](int m) { return p.group == 1 ? hk : hk * p.group + (m0 + m) / per_head; };
    auto qtile = [&](int m) { return m_start + (p.group == 1 ? m0 + m : (m0 + m) % per_head); };

    if (warp == 0) {
        // ------------------------------------------------ copies
        if (lane == 0 && n_tiles > 0) {
            const uint64_t keep = policy_evict_last();
            const KeyBlock* blocks = static_cast<const KeyBlock*>(p.keys) + static_cast<size_t>(b) * p.num_q_tiles;
            int n_q = 0, n_v = 0;  // tiles whose copies were issued, per ring
            int h = qhead(0), t = qtile(0);
            for (int m = 0; m < n_tiles; ++m) {
                const int st = m % L::kNst, sv = m % L::kNv;
                if (!mbar_wait(base + L::bar_empty + 8 * st, ((m / L::kNst) & 1) ^ 1, wc, kErrWaitOther)) break;
                const uint32_t fq = base + L::bar_full + 8 * st;
                mbar_arrive_expect_tx(fq, 2 * L::kQBytes);
#pragma unroll
                for (int c = 0; c < D / kSwizzleCols; ++c) {
                    tma_load_4d_hint(base + L::q + st * L::kQBytes + c * kBwdTile * 128, &tQ, fq, c * kSwizzleCols, t * kBwdTile, h, b, keep);
                    tma_load_4d_hint(base + L::g + st * L::kQBytes + c * kBwdTile * 128, &tG, fq, c * kSwizzleCols, t * kBwdTile, h, b, keep);
                }
                ++n_q;
                if (!mbar_wait(base + L::bar_vempty + 8 * sv, ((m / L::kNv) & 1) ^ 1, wc, kErrWaitOther)) break;
                const uint32_t fv = base + L::bar_vfull + 8 * sv;
                mbar_arrive_expect_tx(fv, kAbRowBytes + static_cast<uint32_t>(sizeof(KeyBlock)));
                const size_t row_block = (static_cast<size_t>(b) * p.H + h) * p.num_q_tiles + t;
                bulk_load(base + L::vec + sv * kAbRowBytes, p.rows + row_block * (2 * kBwdTile), kAbRowBytes, fv);
                bulk_load(base + L::keys + sv * static_cast<uint32_t>(sizeof(KeyBlock)), blocks + t, sizeof(KeyBlock), fv);
                ++n_v;
                if (++t == m_start + per_head) {
                    t = m_start;
                    ++h;
                }
            }
            // every issued copy has landed (and, unless aborting, been consumed)
            for (int j = max(0, n_q - L::kNst); j < n_q; ++j) {
                drain_wait_b(base + L::bar_full + 8 * (j % L::kNst), (j / L::kNst) & 1, kDrainNs);
                if (!*abort_flag) drain_wait_b(base + L::bar_empty + 8 * (j % L::kNst), (j / L::kNst) & 1, kDrainNs);
            }
            for (int j = max(0, n_v - L::kNv); j < n_v; ++j) {
                drain_wait_b(base + L::bar_vfull + 8 * (j % L::kNv), (j / L::kNv) & 1, kDrainNs);
                if (!*abort_flag) drain_wait_b(base + L::bar_vempty + 8 * (j % L::kNv), (j / L::kNv) & 1, kDrainNs);
            }
        }
        if (lane == 0) drain_wait_b(base + L::bar_k, 0, kDrainNs);
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs
        // Scores of tile m: S^T = K Q^T, dP^T = V dO^T.  Gradients of tile m: dV += P^T dO, dK += dS^T Q and
        // [dQ^T_hi | dQ^T_lo] = K^T [dS^T_hi | dS^T_lo].  One thread issues them in the order in which they are wanted:
        // the scores of tile m + 2 behind the gradients of tile m, for whose end the update warps wait with P and dS of
        // tile m + 1.  (Issued by a thread of their own they got between the gradients: 8192 causal rows, 32 heads on
        // 8, 1713 us for the three kernels where one thread takes 1652; 16 heads, full, 1729 and 1557.)
        if (lane == 0 && n_tiles > 0) {
            constexpr uint32_t id_s = idesc_bf16_f32(kBlockK, kBwdTile);
            constexpr uint32_t id_dk = idesc_bf16_f32(kBlockK, D, 0, 1);
            constexpr uint32_t id_dq = idesc_bf16_f32(128, 2 * kBwdTile, 1, 1);  // M = 128 features (d = 64: padded)
            // A = K^T as 64-feature atoms: the tile's second block, or the zero atom when d = 64
            const uint32_t a_atom = D == 128 ? kBlockK * 128 : L::zero - L::k;
            const uint32_t t_dk = tmem + 128, t_dv = tmem + 256, t_dq = tmem + 384;
            const uint32_t dhi = smem_desc_hi();
            const uint32_t k_lo = smem_desc_lo_k128(base + L::k), v_lo = smem_desc_lo_k128(base + L::v);
            const uint32_t ds_lo = smem_desc_lo_k128(base + L::ds), p_lo = smem_desc_lo_k128(base + L::pt);
            const uint32_t dsmn_lo = smem_desc_lo_mn128(base + L::ds, L::kDsBytes);
            const uint32_t kt_lo = smem_desc_lo_mn128(base + L::k, a_atom);
            int issued = 0;
            auto scores = [&](int m) {
                const int st = m % L::kNst;
                if (!mbar_wait(base + L::bar_full + 8 * st, (m / L::kNst) & 1, wc, kErrWaitQ)) return false;
                if (!mbar_wait(base + L::bar_sempty, (m & 1) ^ 1, wc, kErrWaitS)) return false;
                tc_fence_after();
                const uint32_t q_lo = smem_desc_lo_k128(base + L::q + st * L::kQBytes), g_lo = smem_desc_lo_k128(base + L::g + st * L::kQBytes);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t ko = ((kk >> 2) * kBlockK * 128 + (kk & 3) * 32) >> 4, qo = ((kk >> 2) * kBwdTile * 128 + (kk & 3) * 32) >> 4;
                    tc_mma_bf16_w(tmem, k_lo + ko, dhi, q_lo + qo, dhi, id_s, kk > 0);
                }
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t ko = ((kk >> 2) * kBlockK * 128 + (kk & 3) * 32) >> 4, qo = ((kk >> 2) * kBwdTile * 128 + (kk & 3) * 32) >> 4;
                    tc_mma_bf16_w(tmem + 64, v_lo + ko, dhi, g_lo + qo, dhi, id_s, kk > 0);
                }
                tc_commit(base + L::bar_sfull);
                ++issued;
                return true;
            };
            auto gradients = [&](int m) {
                const int st = m % L::kNst;
                if (!mbar_wait(base + L::bar_dsfull, m & 1, wc, kErrWaitOther)) return false;
                tc_fence_after();
                const uint32_t q_lo = smem_desc_lo_mn128(base + L::q + st * L::kQBytes, kBwdTile * 128);
                const uint32_t g_lo = smem_desc_lo_mn128(base + L::g + st * L::kQBytes, kBwdTile * 128);
#pragma unroll
                for (int kk = 0; kk < kBwdTile / 16; ++kk)
                    tc_mma_bf16_w(t_dv, p_lo + ((kk * 32) >> 4), dhi, g_lo + ((kk * 16 * 128) >> 4), dhi, id_dk, (kk | m) != 0);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < kBwdTile / 16; ++kk)
                        tc_mma_bf16_w(t_dk, ds_lo + ((part * L::kDsBytes + kk * 32) >> 4), dhi, q_lo + ((kk * 16 * 128) >> 4), dhi, id_dk,
                                      (kk | part | m) != 0);
                ++issued;
                if (!mbar_wait(base + L::bar_dqempty, (m & 1) ^ 1, wc, kErrWaitOther)) return false;
                tc_fence_after();
                // B = the hi and lo tiles as two 64-query atoms of one N = 128 operand, K = 128 keys
#pragma unroll
                for (int kk = 0; kk < kBlockK / 16; ++kk)
                    tc_mma_bf16_w(t_dq, kt_lo + ((kk * 16 * 128) >> 4), dhi, dsmn_lo + ((kk * 16 * 128) >> 4), dhi, id_dq, kk > 0);
                tc_commit(base + L::bar_dsempty);
                tc_commit(base + L::bar_dqfull);
                tc_commit(base + L::bar_empty + 8 * st);
                if (m + 1 == n_tiles) tc_commit(base + L::bar_done);
                return true;
            };
            // test aid: a wait on a barrier that nothing arrives on before the end
            bool ok = !(p.inject_stall && blockIdx.x == 0 && !mbar_wait(base + L::bar_done, 0, wc, kErrWaitOther));
            ok = ok && mbar_wait(base + L::bar_k, 0, wc, kErrWaitK) && scores(0) && (n_tiles == 1 || scores(1));
            for (int m = 0; ok && m < n_tiles; ++m) ok = gradients(m) && (m + 2 >= n_tiles || scores(m + 2));
            if (*abort_flag && issued > 0) {  // let the issued MMAs retire before TMEM is freed
                tc_commit(base + L::bar_drain);
                drain_wait_b(base + L::bar_drain, 0, kDrainNs);
            }
        }
    } else if (warp < 10) {
        // ------------------------------------------------ P^T, dS^T
        // warps 2-5 take query rows 0-31 of every tile, warps 6-9 rows 32-63; one key per thread
        const int wg = (warp - 2) >> 2, wq = warp & 3, row = wq * 32 + lane;
        const int j = n0 + row;  // key index
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float2 cc = splat(p.c), sc = splat(p.scale);
        // Keys with a NaN or an infinity become zero rows before the first gradient MMA: a dS of 0 would not hide them from
        // rows that do not see them.  The first tiles' scores may be under way and see part of the zeros: for such a key
        // scores do not count (see below).  The barrier: both threads of a key have read it.
        bool ok = n_tiles == 0 || wait_all(base + L::bar_k, 0, wc, kErrWaitK);
        const bool broken = ok && n_tiles > 0 && key_row_broken<D>(gbase + L::k, row);
        if (bar_sync_or(1, 256, broken)) clear_key_row<D>(base + L::k, row);
        for (int m = 0; ok && m < n_tiles; ++m) {
            const int sv = m % L::kNv;
            if (!wait_all(base + L::bar_sfull, m & 1, wc, kErrWaitS) ||
                !wait_all(base + L::bar_vfull + 8 * sv, (m / L::kNv) & 1, wc, kErrWaitQ)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float z[32], dp[32];
            tmem_ld32(tl + wg * 32, z);
            tmem_ld32(tl + 64 + wg * 32, dp);
            tc_wait_ld();
            tc_fence_before();
            mbar_arrive(base + L::bar_sempty);  // the next tile's scores may overwrite them now
            const KeyBlock& kb = reinterpret_cast<const KeyBlock*>(gbase + L::keys)[sv];
            const int4 bounds = kb.bounds[wg];
            const bool whole = bounds.z <= n0 && bounds.w >= n0 + kBlockK;  // every row sees every key
            if (__any_sync(0xffffffffu, broken)) {  // a finite LSE means that the row's score with a broken key is -inf; a NaN in LSE stays
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (broken) z[e] = -INFINITY;
            }
            uint32_t vis = 0xffffffffu;  // bit e: query row e of the half sees this thread's key
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
                        const bool finite = fabsf(z[e]) < INFINITY && fabsf(dp[e]) < INFINITY;
                        if (j >= los[k] && j < his[k])
                            vis |= 1u << e;
                        else
                            bad |= !finite;
                    }
                }
            }
            const float4* v4 = reinterpret_cast<const float4*>(gbase + L::vec + sv * kAbRowBytes) + wg * 8;
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
                const float4 a = v4[e4], x = v4[kBwdTile / 4 + e4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int e = 4 * e4 + 2 * k;
                    const float2 y = __ffma2_rn(make_float2(z[e], z[e + 1]), cc, k ? make_float2(a.z, a.w) : make_float2(a.x, a.y));
                    const float2 pr = make_float2(ex2(y.x), ex2(y.y));
                    const float2 d = __fmul2_rn(pr, __ffma2_rn(make_float2(dp[e], dp[e + 1]), sc, k ? make_float2(x.z, x.w) : make_float2(x.x, x.y)));
                    z[e] = pr.x;
                    z[e + 1] = pr.y;
                    dp[e] = d.x;
                    dp[e + 1] = d.y;
                }
            }
            mbar_arrive(base + L::bar_vempty + 8 * sv);  // this tile's row constants are read
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (!((vis >> e) & 1u)) z[e] = dp[e] = 0.f;
                // A zero P or dS does not hide a NaN or an infinity in the operand it meets in the gradient MMAs:
                // query rows with one become zero rows.  (Where such a row is visible, P and dS are NaN.)
                if (__any_sync(0xffffffffu, bad)) {
                    const int st = m % L::kNst;
                    clear_query_rows<D>(base + L::q + st * L::kQBytes, wg * 32, lane);
                    clear_query_rows<D>(base + L::g + st * L::kQBytes, wg * 32, lane);
                }
            }
            if (!wait_all(base + L::bar_dsempty, (m & 1) ^ 1, wc, kErrWaitOther)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int cc4 = 0; cc4 < 4; ++cc4) {  // P^T as one bf16 term, laid out like dS^T
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = pack_bf16(z[8 * cc4 + 2 * k], z[8 * cc4 + 2 * k + 1]);
                st_shared_v4(base + L::pt + row * 128 + (((wg * 4 + cc4) ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
            store_ds_chunk(base + L::ds, base + L::ds + L::kDsBytes, row, wg * 4, dp);
            fence_proxy_async_smem();
            mbar_arrive(base + L::bar_dsfull);
        }
        if (broken) poison_rows(p, D, b, hk, j, wg, m_start, per_head, m0, n_tiles);
        __syncwarp();
        // epilogue: the first warpgroup writes dK, the second dV
        if (ok && (n_tiles == 0 || wait_all(base + L::bar_done, 0, wc, kErrWaitOther))) {
            tc_fence_after();
            const size_t at_row = static_cast<size_t>(bkv) * p.Nk + j;
            const bool parts = p.num_splits > 1;
            const size_t all = static_cast<size_t>(p.B) * p.H_kv * p.Nk;
            void* out = parts ? static_cast<void*>(p.parts + ((static_cast<size_t>(wg) * p.num_splits + split) * all + at_row) * D)
                              : static_cast<void*>(static_cast<uint16_t*>(wg ? p.dV : p.dK) + at_row * D);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                float v[32];
                tmem_ld32(tl + 128 + wg * 128 + c0, v);
                tc_wait_ld();
                if (n_tiles == 0) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;  // no row sees these keys: nothing was accumulated
                }
                if (j < p.Nk) store_grad32(out, c0, v, 1.0f, !parts);
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------ dQ^T -> bulk L2 reduction into dQ
        // Each half (32 rows) of a tile's block of dQ is staged in shared memory as contiguous float32 rows and
        // added to global dQ by a bulk reduce-add.
        const int wq = warp & 3;
        const int f = wq * 32 + lane;  // feature = TMEM lane
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const bool leader = warp == 10 && lane == 0;
        for (int m = 0; m < n_tiles; ++m) {
            // the four epilogue warps decide together, so none is left at a named barrier
            if (!bar_sync_and(3, 128, wait_all(base + L::bar_dqfull, m & 1, wc, kErrWaitOther))) break;
            tc_fence_after();
            float v[2][32];
            if (wq * 32 < D) {  // d = 64: TMEM lanes 64-127 hold the zero padding
                float lo[32];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    tmem_ld32(tl + 384 + 32 * hf, v[hf]);
                    tmem_ld32(tl + 448 + 32 * hf, lo);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 t = __fadd2_rn(make_float2(v[hf][e], v[hf][e + 1]), make_float2(lo[e], lo[e + 1]));
                        v[hf][e] = t.x;
                        v[hf][e + 1] = t.y;
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(base + L::bar_dqempty);
            const int r0 = qtile(m) * kBwdTile;
            const int nrow = min(kBwdTile, p.Nq - r0);
            float* dst = p.dQacc + ((static_cast<size_t>(b) * p.H + qhead(m)) * p.Nq + r0) * D;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                if (leader) bulk_wait_read_all();  // the last reduction has read the stage
                asm volatile("bar.sync 2, 128;" ::: "memory");
                if (f < D) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + L::stage + e * (D * 4) + f * 4), "f"(v[hf][e]) : "memory");
                }
                fence_proxy_async_smem();
                asm volatile("bar.sync 2, 128;" ::: "memory");
                const int rows = min(32, nrow - 32 * hf);
                if (leader && rows > 0) {
                    bulk_reduce_add_f32(dst + hf * 32 * D, base + L::stage, static_cast<uint32_t>(rows * D * 4));
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
    if (*abort_flag) mark_attn_gradients(p, D, b, hk, n0, split, m_start, per_head, m0, n_tiles);
}

// 8 elements of dQ (float32 -> bf16), or of dK and dV (the sum of their splits'
// parts, in order), per thread and step.
__global__ void __launch_bounds__(256) attn_finish_kernel(const float4* dq, uint4* dq_out, size_t nq8, const float4* parts,
                                                          uint4* dk_out, uint4* dv_out, size_t nk8, int splits) {
    for (size_t k = blockIdx.x * size_t(blockDim.x) + threadIdx.x; k < nq8 + 2 * nk8; k += size_t(gridDim.x) * blockDim.x) {
        float4 a, b;
        uint4* out;
        if (k < nq8) {
            a = dq[2 * k], b = dq[2 * k + 1];
            out = dq_out + k;
        } else {
            const bool second = k - nq8 >= nk8;
            const size_t e = k - nq8 - (second ? nk8 : 0);
            const float4* q = parts + (second ? 2 * splits * nk8 : 0);
            a = q[2 * e], b = q[2 * e + 1];
            for (int s = 1; s < splits; ++s) {
                const float4 u = q[2 * (s * nk8 + e)], v = q[2 * (s * nk8 + e) + 1];
                a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
                b.x += v.x, b.y += v.y, b.z += v.z, b.w += v.w;
            }
            out = (second ? dv_out : dk_out) + e;
        }
        *out = make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
    }
}

template <int D>
cudaError_t launch_attn_bwd_d(const CUtensorMap* m, const AttnBwdParams& p, const ScoreParams& sp, int ctas, int sms, cudaStream_t st) {
    constexpr int bytes = AttnKvSmem<D>::alloc;
    static_assert(bytes <= 232448, "shared memory");
    auto k = attn_bwd_kernel<D>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(k, bytes, &done);
    if (e != cudaSuccess) return e;
    attn_prepare_kernel<D><<<static_cast<unsigned>(p.B * p.H) * p.num_q_tiles, 256, 0, st>>>(p, sp);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k<<<ctas, kAbThreads, bytes, st>>>(m[0], m[1], m[2], m[3], p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const size_t nq8 = static_cast<size_t>(p.B) * p.H * p.Nq * D / 8;
    const size_t nk8 = p.num_splits > 1 ? static_cast<size_t>(p.B) * p.H_kv * p.Nk * D / 8 : 0;
    const size_t blocks = std::min<size_t>((nq8 + 2 * nk8 + 255) / 256, static_cast<size_t>(sms) * 16);
    attn_finish_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(
        reinterpret_cast<const float4*>(p.dQacc), static_cast<uint4*>(p.dQ), nq8, reinterpret_cast<const float4*>(p.parts),
        static_cast<uint4*>(p.dK), static_cast<uint4*>(p.dV), nk8, p.num_splits);
    return cudaGetLastError();
}

}  // namespace

size_t attn_bwd_row_bytes(int64_t bh, int q_tiles) { return static_cast<size_t>(bh) * q_tiles * kAbRowBytes; }
size_t attn_bwd_key_bytes(int64_t batch, int q_tiles) { return static_cast<size_t>(batch) * q_tiles * sizeof(KeyBlock); }

cudaError_t launch_attn_bwd(int d, const CUtensorMap* maps, const AttnBwdParams& p, const ScoreParams& sp, int ctas, int sms,
                            cudaStream_t stream) {
    return d == 128 ? launch_attn_bwd_d<128>(maps, p, sp, ctas, sms, stream) : launch_attn_bwd_d<64>(maps, p, sp, ctas, sms, stream);
}

}  // namespace streamkl
