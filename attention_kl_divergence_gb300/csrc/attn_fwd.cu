// attn_fwd.cu -- attention over whole prompts on sm_103a, forward.
//
//   O_i = sum_j 2^(x_ij - m_i) v_j / l_i,  l_i = sum_j 2^(x_ij - m_i),  x = log2(e) scale q k
//
// over the keys of row i's range, one pass over the keys.  The probabilities enter
// the product with V as one bf16 term, or, where the backward is to follow (`rest` is
// asked for), as two: the backward's row sums of dO O take O as that of exact
// probabilities, and an error of theirs is a multiple of the row's mean key in dQ.  m_i is a
// running maximum that may stay up to 2^8 behind.
//
// A CTA takes a pair of 128-row tiles that read the same keys (two heads of a key head, or
// neighbouring rows): each key and value tile that TMA brings serves both, and while the
// softmax of one runs the tensor core has the other's products.  A key tile takes a pair
// about 3450 cycles, of which its MMAs need 2515 at the measured peak.  32768 causal rows,
// 8 heads, d = 128: 1594 us, 1379 TFLOP/s.  8192 causal rows, 32 heads on 8, with rest:
// 592 us, 929 TFLOP/s, and half as much again for the second term.  8192 rows in documents:
// 191 us, 720 TFLOP/s; a CTA spends about 13000 cycles on its start and end there and 33000
// on its key tiles.  At the 96 registers that 19 warps leave a thread the kernels spill 48 to 60
// bytes.  One token over 4 caches of up to 65536 keys: 160 us, 5.9 TB/s.
#include "attn.cuh"
#include "bwd_common.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "ptx.cuh"
#include "score.cuh"

namespace streamkl {

namespace {

constexpr float kAttnTau = 8.f;  // m may stay this far (log2) below the largest score
// warps 0-15 softmax (two warpgroups per tile of the pair: a thread has half of a row's
// scores), 16 copies, 17 MMAs, 18 looks for NaN and infinities in values that some row must
// not see (two such warps: 8192 causal rows, 32 heads on 8, with rest 613 us, one 592).  One warpgroup per tile, a row per thread, left its latencies
// bare: 1912 us where two took 1757, 32768 causal rows, 8 heads.
constexpr int kAfThreads = 608;

template <int D>
struct AttnSmem {
    static constexpr int kNst = D == 128 ? 5 : 8;      // ring of key and value tiles, alternating
    static constexpr int kTile = kBlockQ * D * 2;      // 128 rows of q, k or v
    static constexpr int q = 0;                        // the pair's query tiles
    static constexpr int kv = 2 * kTile;
    static constexpr int bar_q = kv + kNst * kTile;    // [2]
    static constexpr int bar_full = bar_q + 16;        // [kNst]
    static constexpr int bar_empty = bar_full + 8 * kNst;
    static constexpr int bar_clean = bar_empty + 8 * kNst;  // [kNst] checks, in turn
    static constexpr int bar_s = bar_clean + 8 * kNst;      // [2] scores complete
    static constexpr int bar_p = bar_s + 16;                // [2] probabilities stored
    static constexpr int bar_o = bar_p + 16;                // [2] output complete
    static constexpr int bar_done = bar_o + 16;             // drain of an aborted issuer
    static constexpr int misc = bar_done + 8;               // tmem base, abort flag
    static constexpr int spans = (misc + 8 + 15) / 16 * 16; // [2] int4: union and common range of a tile's rows
    static constexpr int bad = spans + 32;                  // [kNst][4] keys whose values are not finite
    static constexpr int tops = bad + 16 * kNst;            // [2][2][128] maxima of the halves of the rows, their sums at the end
    static constexpr int alloc = tops + 2048;               // no slack: the kernel checks the base is 1024-byte aligned
    static constexpr int stage = q;                         // outputs at the end, when the query tiles are done with
};

// The key tiles [lo, hi) of a range of keys.
__device__ __forceinline__ int2 tiles_of(int4 span) {
    return span.x < span.y ? make_int2(span.x / kBlockK, (span.y + kBlockK - 1) / kBlockK) : make_int2(0, 0);
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }

// 2^(z c - ref) of 16 scores, from FROM on, as 8 words of bf16 pairs, and with two terms what they lack as 8 more.
// Their float32 sums are added to la, lb.
template <int TERMS, int FROM>
__device__ __forceinline__ void exp_part(const float (&z)[32], float c, float ref, float2& la, float2& lb, uint32_t (&w)[8],
                                         uint32_t (&less)[8]) {
    const float2 cc = splat(c), nr = splat(-ref), minus = splat(-1.f);
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
        const int e = FROM + k;
        const float2 a = __ffma2_rn(make_float2(z[e], z[e + 1]), cc, nr), b = __ffma2_rn(make_float2(z[e + 2], z[e + 3]), cc, nr);
        const float2 pa = make_float2(ex2(a.x), ex2(a.y)), pb = make_float2(ex2(b.x), ex2(b.y));
        la = __fadd2_rn(la, pa);
        lb = __fadd2_rn(lb, pb);
        w[k / 2] = pack_bf16(pa.x, pa.y);
        w[k / 2 + 1] = pack_bf16(pb.x, pb.y);
        if (TERMS == 2) {
            const float2 da = __ffma2_rn(unpack_bf16(w[k / 2]), minus, pa), db = __ffma2_rn(unpack_bf16(w[k / 2 + 1]), minus, pb);
            less[k / 2] = pack_bf16(da.x, da.y);
            less[k / 2 + 1] = pack_bf16(db.x, db.y);
        }
    }
}

__device__ __forceinline__ float max_chunk(const float (&z)[32]) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = max3f(m[k], z[e + 2 * k], z[e + 2 * k + 1]);
    }
    return fmaxf(max3f(m[0], m[1], m[2]), m[3]);
}

// 0 x + sum of two bf16.
__device__ __forceinline__ uint32_t zero_times(uint32_t x, uint32_t sum) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(sum));
    return r;
}

// Hidden scores become -inf.
__device__ __forceinline__ void hide_chunk(float (&z)[32], int first, int last) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (e < first || e > last) z[e] = -INFINITY;
}

template <int D>
__device__ __noinline__ void mark_row(const AttnFwdParams& p, int split, int sub, int b, int h, int i) {
    const float nan = __int_as_float(0x7fc00000);
    const size_t R = static_cast<size_t>(p.B) * p.H * p.Nq, flat = (static_cast<size_t>(b) * p.H + h) * p.Nq + i;
    if (p.parts > 1) {
        const size_t at = (p.dual ? 2 * split + sub : split) * R + flat;
        p.part_ml[at] = make_float2(0.f, nan);
        for (int k = 0; k < D; ++k) p.part[at * D + k] = nan;
        return;
    }
    uint16_t* out = static_cast<uint16_t*>(p.O) + (b * p.o_b + h * p.o_h + static_cast<int64_t>(i) * p.o_n);
    for (int k = 0; k < D; ++k) {
        out[k] = 0x7fc0;
        if (p.rest) static_cast<uint16_t*>(p.rest)[flat * D + k] = 0x7fc0;
    }
    p.LSE[flat] = nan;
}

// n columns of O at t_o times f.
__device__ __noinline__ void rescale(uint32_t t_o, int n, float f) {
#pragma unroll 1
    for (int k = 0; k < n; k += 32) {
        float v[32];
        tmem_ld32(t_o + k, v);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= f;
        tmem_st32(t_o + k, v);
    }
    tc_wait_st();
}

// A lane's row of 16 CH words -> memory at `out` (null: not written), through shared memory: what a lane holds are 64 CH
// bytes of a row of its own, and the lanes of a store cover whole rows.
template <int CH>
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t (&w)[CH][16], uint8_t* out, int lane) {
    constexpr int kLanes = 4 * CH;  // of a row
    auto at = [&](int row, int piece) { return stage + row * (64 * CH) + ((piece ^ (CH == 2 ? row & 7 : row >> 1 & 3)) << 4); };
#pragma unroll
    for (int k = 0; k < kLanes; ++k)
        *reinterpret_cast<uint4*>(at(lane, k)) = make_uint4(w[k / 4][k % 4 * 4], w[k / 4][k % 4 * 4 + 1], w[k / 4][k % 4 * 4 + 2], w[k / 4][k % 4 * 4 + 3]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
        const int row = k * (32 / kLanes) + lane / kLanes, piece = lane % kLanes;
        uint8_t* to = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), row));
        const uint4 u = *reinterpret_cast<const uint4*>(at(row, piece));
        if (to) *reinterpret_cast<uint4*>(to + 16 * piece) = u;
    }
    __syncwarp();
}

}  // namespace

template <int D, int TERMS>
__global__ void __launch_bounds__(kAfThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
                    const __grid_constant__ CUtensorMap tV, const __grid_constant__ AttnFwdParams p,
                    const __grid_constant__ ScoreParams sp) {
    using L = AttnSmem<D>;
    constexpr int NST = L::kNst;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    uint8_t* gbase = smem_raw;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::misc + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::misc);
    int4* spans = reinterpret_cast<int4*>(gbase + L::spans);
    uint32_t* bad = reinterpret_cast<uint32_t*>(gbase + L::bad);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the pair's tiles; in a group of heads the last query tiles of every head come first
    const int unit = p.by_splits.of(blockIdx.x), split = blockIdx.x - unit * p.num_splits;
    const int og = p.order_units.of(unit), first_head = og * p.order_group.d, rest_units = unit - first_head * p.units_q;
    const bool last_group = first_head + static_cast<int>(p.order_group.d) >= p.B * p.H_kv * p.units_h;
    const int from_end = last_group ? p.order_last.of(rest_units) : p.order_group.of(rest_units);
    const int head = first_head + rest_units - from_end * static_cast<int>(last_group ? p.order_last.d : p.order_group.d);
    const int bkv = p.by_units_h.of(head), hb = head - bkv * p.units_h, qu = p.units_q - 1 - from_end;
    const int b = p.by_H_kv.of(bkv), hk = bkv - b * p.H_kv;
    auto block_of = [&](int s) { return p.pair_heads ? 2 * hb + s : hb; };
    auto qtile_of = [&](int s) { return p.pair_heads || p.dual ? qu : 2 * qu + s; };
    auto exists = [&](int s) { return block_of(s) < p.blocks && qtile_of(s) < p.q_tiles; };

    // a softmax thread's row: its keys, and whether there is such a row; the thread has 64 of a tile's columns
    const int sub = (warp >> 3) & 1, side = (warp >> 2) & 1, wq = warp & 3, row = wq * 32 + lane;
    const int in_block = p.by_rows.of(row), i = qtile_of(sub) * kBlockQ + row - in_block * p.rows;
    const bool valid = warp < 16 && exists(sub) && in_block < p.heads && i < p.Nq;
    const int2 range = valid ? row_range(sp, p.Nq, p.Nk, b, i) : make_int2(0, 0);
    if (base & 1023u) {  // reported, not expected: every row becomes NaN
        if (threadIdx.x == 0 && p.status) atomicOr(p.status, kErrSmemAlign);
        if (valid && side == 0) mark_row<D>(p, split, sub, b, hk * p.group + block_of(sub) * p.heads + in_block, i);
        return;
    }

    if (threadIdx.x == 512) {
        prefetch_tensormap(&tQ);
        prefetch_tensormap(&tK);
        prefetch_tensormap(&tV);
        for (int s = 0; s < 2; ++s) {
            mbar_init(base + L::bar_q + 8 * s, 1);
            mbar_init(base + L::bar_s + 8 * s, 1);
            mbar_init(base + L::bar_p + 8 * s, 256);
            mbar_init(base + L::bar_o + 8 * s, 1);
            spans[s] = make_int4(INT32_MAX, 0, 0, INT32_MAX);
        }
        for (int s = 0; s < NST; ++s) {
            mbar_init(base + L::bar_full + 8 * s, 1);
            mbar_init(base + L::bar_empty + 8 * s, 2);  // the MMAs and the checking warp
            mbar_init(base + L::bar_clean + 8 * s, 1);
        }
        mbar_init(base + L::bar_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
        // the query tiles are on their way while the rows' ranges are looked up
        for (int s = 0; s < 2; ++s) {
            if (!exists(s)) continue;
            const uint32_t fb = base + L::bar_q + 8 * s, dst = base + L::q + s * L::kTile;
            mbar_arrive_expect_tx(fb, static_cast<uint32_t>(p.heads * p.rows) * D * 2);  // the rows that a copy writes
#pragma unroll
            for (int c = 0; c < D / kSwizzleCols; ++c)
                tma_load_4d(dst + c * kBlockQ * 128, &tQ, fb, c * kSwizzleCols, qtile_of(s) * kBlockQ,
                            hk * p.group + block_of(s) * p.heads, b);
        }
    }
    if (warp == 17) tmem_alloc(base + L::misc, 512);
    __syncthreads();
    // keys that some row of the warp sees, and those that all of its rows see
    int4 mine = make_int4(0, 0, 0, 0);
    if (warp < 16) {
        const bool live = range.x < range.y;
        mine.x = __reduce_min_sync(0xffffffffu, live ? range.x : INT32_MAX);
        mine.y = __reduce_max_sync(0xffffffffu, live ? range.y : 0);
        mine.z = __reduce_max_sync(0xffffffffu, !valid ? 0 : live ? range.x : INT32_MAX);
        mine.w = __reduce_min_sync(0xffffffffu, valid ? range.y : INT32_MAX);
        if (lane == 0) {
            int* s = reinterpret_cast<int*>(spans + sub);
            atomicMin(s, mine.x);
            atomicMax(s + 1, mine.y);
            atomicMax(s + 2, mine.z);
            atomicMin(s + 3, mine.w);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wc{abort_flag, p.status, p.wait_ns};

    // key tiles: this split's share [t0, t1) of the pair's, and each tile's own part of it
    const int2 ta = tiles_of(spans[0]), tb = tiles_of(spans[1]);
    int t0, t1;
    {
        const int lo = ta.x < ta.y ? (tb.x < tb.y ? min(ta.x, tb.x) : ta.x) : tb.x, hi = max(ta.y, tb.y);
        const int n = max(0, hi - lo), per = (n + p.num_splits - 1) / p.num_splits;
        t0 = lo + split * per;
        t1 = max(t0, min(hi, t0 + per));
    }
    auto active = [&](int s, int t) {
        return (s == 0 ? t >= ta.x && t < ta.y : t >= tb.x && t < tb.y) && !(p.dual && ((t - t0) & 1) != s);
    };
    // a value tile is checked when some row of an active tile does not see all of its keys
    const int2 wa = make_int2((spans[0].z - 1) / kBlockK + (spans[0].z > 0), spans[0].w / kBlockK);  // tiles that all rows see all of
    const int2 wb = make_int2((spans[1].z - 1) / kBlockK + (spans[1].z > 0), spans[1].w / kBlockK);
    auto checked = [&](int t) { return (active(0, t) && !(t >= wa.x && t < wa.y)) || (active(1, t) && !(t >= wb.x && t < wb.y)); };

    if (warp == 16) {
        // ------------------------------------------------------------ copies
        if (lane == 0 && t1 > t0) {
            const uint64_t keep = policy_evict_last();  // key and value tiles are read again by other query tiles
            int n = 0;
            for (; n < 2 * (t1 - t0); ++n) {  // key tile, value tile, key tile, ...
                const int s = n % NST;
                if (!mbar_wait(base + L::bar_empty + 8 * s, ((n / NST) & 1) ^ 1, wc, kErrWaitK)) break;
                const uint32_t fb = base + L::bar_full + 8 * s, dst = base + L::kv + s * L::kTile;
                mbar_arrive_expect_tx(fb, L::kTile);
#pragma unroll
                for (int c = 0; c < D / kSwizzleCols; ++c)
                    tma_load_4d_hint(dst + c * kBlockK * 128, n & 1 ? &tV : &tK, fb, c * kSwizzleCols,
                                     (t0 + (n >> 1)) * kBlockK, hk, b, keep);
            }
            // every issued copy has landed, every stage was released
            for (int j = max(0, n - NST); j < n; ++j) {
                drain_wait_b(base + L::bar_full + 8 * (j % NST), (j / NST) & 1, kDrainNs);
                if (!*abort_flag) drain_wait_b(base + L::bar_empty + 8 * (j % NST), (j / NST) & 1, kDrainNs);
            }
        }
        for (int s = 0; lane == 0 && s < 2; ++s)
            if (exists(s)) drain_wait_b(base + L::bar_q + 8 * s, 0, kDrainNs);
    } else if (warp == 17) {
        // ------------------------------------------------------------ MMAs
        // S_s(t) = Q_s K(t)^T, then O_s += P_s(t) V(t) with P_s over S_s in tensor memory.  While one tile's
        // softmax runs, the tensor core works for the other.  The MMAs of a thread run in order: S_s(t + 1)
        // does not overwrite P_s(t) before O_s has taken it, and S_s(t + 1) complete means that O_s is too.
        // (A thread for each tile: 2223 us where one takes 1745, 32768 causal rows, 8 heads: the MMAs of two
        // threads get in each other's way.)
        if (lane == 0 && t1 > t0) {
            constexpr uint32_t id_s = idesc_bf16_f32(kBlockQ, kBlockK), id_o = idesc_bf16_f32(kBlockQ, D, 0, 1);
            constexpr uint32_t kTileLo = L::kTile >> 4;
            const uint32_t dhi = smem_desc_hi();
            const uint32_t q_lo = smem_desc_lo_k128(base + L::q), k_lo0 = smem_desc_lo_k128(base + L::kv);
            const uint32_t v_lo0 = smem_desc_lo_mn128(base + L::kv, kBlockK * 128);
            int issued = 0;
            uint32_t n_p[2] = {0, 0};
            bool ok = !(p.inject_stall && blockIdx.x == 0 && !mbar_wait(base + L::bar_done, 0, wc, kErrWaitOther));
            auto scores = [&](int s, int st) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * kBlockQ * 128 + (kk & 3) * 32) >> 4;
                    tc_mma_bf16_w(tmem + s * 128, q_lo + s * kTileLo + o, dhi, k_lo0 + st * kTileLo + o, dhi, id_s, kk > 0);
                }
                tc_commit(base + L::bar_s + 8 * s);
                ++issued;
            };
            auto values = [&](int s, int st) {
                const uint32_t v_lo = v_lo0 + st * kTileLo;
#pragma unroll
                for (int kk = 0; kk < TERMS * kBlockK / 16; ++kk)  // columns: see the softmax
                    tc_mma_bf16_ta_w(tmem + 256 + s * 128, tmem + s * 128 + (kk >> 1 & 3) * 32 + (kk >> 3) * 16 + (kk & 1) * 8,
                                     v_lo + (((kk & 7) * 16 * 128) >> 4), dhi, id_o, (n_p[s] | kk) != 0);
                ++n_p[s];
            };
            // ring positions: K(t) and V(t) stand in stages 2 (t - t0) and 2 (t - t0) + 1, modulo NST
            int sk = 0, sv = 1;
            uint32_t pk = 0, pv = 0;
            auto landed = [&](int st, uint32_t phase) { return mbar_wait(base + L::bar_full + 8 * st, phase, wc, kErrWaitK); };
            auto step = [](int& st, uint32_t& phase, int by) {
                st += by;
                if (st >= NST) st -= NST, phase ^= 1;
            };
            if (p.dual) {  // the tile's rows twice: every second key tile each
                for (int s = 0; ok && s < 2 && t0 + s < t1; ++s) {
                    if (!(ok = mbar_wait(base + L::bar_q + 8 * s, 0, wc, kErrWaitQ) && landed(sk, pk))) break;
                    tc_fence_after();
                    scores(s, sk);
                    tc_commit(base + L::bar_empty + 8 * sk);
                    step(sk, pk, 2);
                }
                for (int t = t0; ok && t < t1; ++t) {
                    const int s = (t - t0) & 1;
                    if (!(ok = landed(sv, pv) && mbar_wait(base + L::bar_p + 8 * s, n_p[s] & 1, wc, kErrWaitS))) break;
                    tc_fence_after();
                    values(s, sv);
                    tc_commit(base + L::bar_empty + 8 * sv);
                    step(sv, pv, 2);
                    if (t + 2 >= t1) {
                        tc_commit(base + L::bar_o + 8 * s);
                        continue;
                    }
                    if (!(ok = landed(sk, pk))) break;
                    tc_fence_after();
                    scores(s, sk);
                    tc_commit(base + L::bar_empty + 8 * sk);
                    step(sk, pk, 2);
                }
            } else {
                // the tiles' key tiles [lo, hi)
                const int lo[2] = {max(ta.x, t0), max(tb.x, t0)}, hi[2] = {min(ta.y, t1), min(tb.y, t1)};
                for (int s = 0; ok && s < 2; ++s)
                    if (lo[s] < hi[s]) ok = mbar_wait(base + L::bar_q + 8 * s, 0, wc, kErrWaitQ);
                if ((ok = ok && landed(sk, pk))) {
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        if (lo[s] == t0 && t0 < hi[s]) scores(s, sk);
                    tc_commit(base + L::bar_empty + 8 * sk);
                    step(sk, pk, 2);
                }
                for (int t = t0; ok && t < t1; ++t) {
                    const bool more = t + 1 < t1;
                    if (!(ok = landed(sv, pv) && (!more || landed(sk, pk)))) break;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (t >= lo[s] && t < hi[s]) {
                            if (!(ok = mbar_wait(base + L::bar_p + 8 * s, n_p[s] & 1, wc, kErrWaitS))) break;
                            tc_fence_after();
                            values(s, sv);
                            if (t + 1 == hi[s]) tc_commit(base + L::bar_o + 8 * s);
                        }
                        if (t + 1 >= lo[s] && t + 1 < hi[s]) scores(s, sk);
                    }
                    if (!ok) break;
                    tc_commit(base + L::bar_empty + 8 * sv);
                    step(sv, pv, 2);
                    if (more) {
                        tc_commit(base + L::bar_empty + 8 * sk);
                        step(sk, pk, 2);
                    }
                }
            }
            if (*abort_flag && issued > 0) {  // let the issued MMAs retire before TMEM is freed
                tc_commit(base + L::bar_done);
                drain_wait_b(base + L::bar_done, 0, kDrainNs);
            }
        }
    } else if (warp == 18) {
        // ------------------------------------------------------------ value check
        // A probability of 0 does not hide a NaN or an infinity in the value that it meets in the MMA.  In tiles
        // that some row does not see all of, keys with such values get zeros, and rows that see them become NaN.
        // The warp waits for every copy of the ring in turn and releases every stage with the MMAs: a wait that skipped
        // a stage's use would take the use before it for its own.  The k-th check uses slot k % NST: the ring holds
        // fewer value tiles than there are slots.
        int k_check = 0;
        for (int n = 0; n < 2 * (t1 - t0); ++n) {
            const int st = n % NST, t = t0 + (n >> 1);
            if (!wait_all(base + L::bar_full + 8 * st, (n / NST) & 1, wc, kErrWaitK)) break;
            if (!(n & 1) || !checked(t)) {
                if (lane == 0) mbar_arrive(base + L::bar_empty + 8 * st);
                continue;
            }
            const int slot = k_check++ % NST;
            const uint8_t* tile = gbase + L::kv + st * L::kTile;
#pragma unroll 1
            for (int r0 = 0; r0 < kBlockK; r0 += 32) {
                const int r = r0 + lane;
                uint32_t sum = 0u;  // 0 x: NaN where x is not finite
#pragma unroll 2
                for (int c = 0; c < D / kSwizzleCols; ++c)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint4 u = *reinterpret_cast<const uint4*>(tile + c * kBlockK * 128 + r * 128 + ((k ^ (lane & 7)) << 4));
                        sum = zero_times(u.x, zero_times(u.y, zero_times(u.z, zero_times(u.w, sum))));
                    }
                const bool any = has_nonfinite_bf16(sum);
                const uint32_t rows = __ballot_sync(0xffffffffu, any);
                if (lane == 0) bad[4 * slot + (r0 >> 5)] = rows;
                if (any) {
#pragma unroll 1
                    for (int c = 0; c < D / kSwizzleCols; ++c)
#pragma unroll 1
                        for (int k = 0; k < 8; ++k)
                            st_shared_v4(base + L::kv + st * L::kTile + c * kBlockK * 128 + r * 128 + 16 * k, 0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(base + L::bar_clean + 8 * slot);
                mbar_arrive(base + L::bar_empty + 8 * st);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t t_s = tl + sub * 128 + 64 * side, t_o = tl + 256 + sub * 128;
        const float c = p.c;
        float ref = -INFINITY;     // m, the same on both sides of a row
        float l = 0.f;             // sum of the probabilities of this side
        float* tops = reinterpret_cast<float*>(gbase + L::tops) + sub * 256 + row;
        bool broken = false;
        bool ok = true;
        int n = 0, k_check = 0;
        for (int t = t0; t < t1; ++t) {
            const bool check = checked(t);
            const int slot = k_check % NST, phase = (k_check / NST) & 1;
            k_check += check;
            if (!active(sub, t)) continue;
            ok = ok && wait_all(base + L::bar_s + 8 * sub, n & 1, wc, kErrWaitS);
            tc_fence_after();
            const int j0 = t * kBlockK + 64 * side;
            const int first = range.x - j0, last = range.y - 1 - j0;  // columns that the row sees
            const bool whole = j0 >= mine.z && j0 + 64 <= mine.w;
            const bool any0 = j0 < mine.y && j0 + 32 > mine.x, any1 = j0 + 32 < mine.y && j0 + 64 > mine.x;
            // the largest score; the second 32 columns stay, the first are read once more
            float z[32];
            float top = -INFINITY;
            if (any0) {
                tmem_ld32(t_s, z);
                tc_wait_ld();
                if (!whole) hide_chunk(z, first, last);
                top = max_chunk(z);
            }
            if (any1) {
                tmem_ld32(t_s + 32, z);
                tc_wait_ld();
                if (!whole) hide_chunk(z, first - 32, last - 32);
                top = fmaxf(top, max_chunk(z));
            }
            top *= c;
            if (bar_sync_or(1 + sub, 256, (valid && top > ref + kAttnTau) || !ok)) {
                // some row's m rises (or a wait gave up): both sides of the rows take the larger of their maxima
                tops[128 * side] = top;
                if (!(ok = bar_sync_and(1 + sub, 256, ok))) break;
                top = fmaxf(top, tops[128 * (side ^ 1)]);
                const bool raise = valid && top > ref + kAttnTau;
                const float f = raise ? ex2(ref - top) : 1.f;
                l *= f;
                if (raise) ref = top;
                if (n > 0 && __any_sync(0xffffffffu, raise)) rescale(t_o + side * (D / 2), D / 2, f);
            }
            // 32 scores make room for their probabilities: 16 columns of (first) terms, 16 of second terms
            const float r = ref == -INFINITY ? 0.f : ref;
            float2 la = splat(0.f), lb = la;
            uint32_t w[8], less[8];
#pragma unroll
            for (int q = 1; q >= 0; --q) {
                const uint32_t t_q = t_s + 32 * q;
                if (q ? any1 : any0) {
                    if (q == 0) {
                        tmem_ld32(t_s, z);
                        tc_wait_ld();
                        if (!whole) hide_chunk(z, first, last);
                    }
                    exp_part<TERMS, 0>(z, c, r, la, lb, w, less);
                    tmem_st8(t_q, w);
                    if (TERMS == 2) tmem_st8(t_q + 16, less);
                    exp_part<TERMS, 16>(z, c, r, la, lb, w, less);
                    tmem_st8(t_q + 8, w);
                    if (TERMS == 2) tmem_st8(t_q + 24, less);
                } else {  // no row of the warp sees any of these keys
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0u;
#pragma unroll
                    for (int k = 0; k < 2 * TERMS; ++k) tmem_st8(t_q + 8 * k, w);
                }
            }
            l += (la.x + la.y) + (lb.x + lb.y);
            if (check) ok = wait_all(base + L::bar_clean + 8 * slot, phase, wc, kErrWaitOther);
            if (check && ok) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t u = bad[4 * slot + 2 * side + k];
                    if (u) {
                        const int from = max(first - 32 * k, 0), to = min(last - 32 * k, 31);
                        if (from <= to) broken |= ((u >> from) << from & (0xffffffffu >> (31 - to))) != 0u;
                    }
                }
                __syncwarp();
            }
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(base + L::bar_p + 8 * sub);
            ++n;
        }
        if (ok && n > 0) ok = wait_all(base + L::bar_o + 8 * sub, 0, wc, kErrWaitOther);
        tc_fence_after();
        // both sides' sums, which are not below 0: the sign says that a value which the row sees is broken.  Its outputs are
        // NaN then; LSE has no values in it.
        ok = bar_sync_and(1 + sub, 256, ok);
        tops[128 * side] = broken ? -l : l;
        ok = bar_sync_and(1 + sub, 256, ok);
        const float theirs = tops[128 * (side ^ 1)];
        l += fabsf(theirs);
        broken |= signbit(theirs);
        if (ok && exists(sub)) ok = wait_all(base + L::bar_q + 8 * sub, 0, wc, kErrWaitQ);  // the stage's bytes
        const float nan = __int_as_float(0x7fc00000);
        const bool fail = __any_sync(0xffffffffu, !ok || *abort_flag);
        const int h = hk * p.group + block_of(sub) * p.heads + in_block;
        const size_t flat = (static_cast<size_t>(b) * p.H + h) * p.Nq + i;
        if (fail) l = nan;
        const bool empty = range.x >= range.y;
        if (p.parts == 1) {
            const float inv = empty ? 0.f : broken ? nan : 1.f / l;
            uint32_t w[D / 64][16], less[D / 64][16];
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                float v[32];
                if (n > 0 && !fail) {
                    tmem_ld32(t_o + side * (D / 2) + 32 * k, v);
                    tc_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float x = empty ? 0.f : n > 0 && !fail ? v[e] * inv : nan, y = empty ? 0.f : n > 0 && !fail ? v[e + 1] * inv : nan;
                    const uint32_t u = pack_bf16(x, y);
                    w[k][e / 2] = u;
                    if (TERMS == 2) less[k][e / 2] = pack_bf16(x - __uint_as_float(u << 16), y - __uint_as_float(u & 0xffff0000u));
                }
            }
            uint8_t* out = valid ? static_cast<uint8_t*>(p.O) + 2 * (b * p.o_b + h * p.o_h + static_cast<int64_t>(i) * p.o_n) + side * D : nullptr;
            uint8_t* rest = valid ? static_cast<uint8_t*>(p.rest) + flat * (2 * D) + side * D : nullptr;
            uint8_t* stage = gbase + L::stage + sub * L::kTile + (4 * side + wq) * (32 * D);
            if (!fail) {
                store_rows<D / 64>(stage, w, out, lane);
                if (TERMS == 2) store_rows<D / 64>(stage, less, rest, lane);
            } else if (valid) {  // the query tile may still be on its way
#pragma unroll 1
                for (int k = 0; k < D; k += 16) {
                    *reinterpret_cast<uint4*>(out + k) = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
                    if (TERMS == 2) *reinterpret_cast<uint4*>(rest + k) = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
                }
            }
            if (valid && side == 0) p.LSE[flat] = empty ? -INFINITY : fmaf(ref, kLn2, logf(l));
        } else {
            const size_t R = static_cast<size_t>(p.B) * p.H * p.Nq, at_row = (p.dual ? 2 * split + sub : split) * R + flat;
#pragma unroll 1
            for (int k = side * (D / 2); k < (side + 1) * (D / 2); k += 32) {
                float v[32];
                if (n > 0 && !fail) {
                    tmem_ld32(t_o + k, v);
                    tc_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                if (valid) store_grad32(p.part + at_row * D, k, v, broken ? nan : 1.f, false);
                __syncwarp();
            }
            if (valid && side == 0) p.part_ml[at_row] = make_float2(ref, l);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// One warp per row: the splits' sums, brought to the largest m.
template <int D>
__global__ void __launch_bounds__(256) attn_combine_kernel(const __grid_constant__ AttnFwdParams p,
                                                           const __grid_constant__ ScoreParams sp) {
    const size_t R = static_cast<size_t>(p.B) * p.H * p.Nq;
    const size_t row = blockIdx.x * size_t(8) + (threadIdx.x >> 5);
    if (row >= R) return;
    const int lane = threadIdx.x & 31, V = D / 32;
    const int i = static_cast<int>(row % p.Nq), h = static_cast<int>(row / p.Nq % p.H), b = static_cast<int>(row / p.Nq / p.H);
    const int2 range = row_range(sp, p.Nq, p.Nk, b, i);
    float m = -INFINITY;
    for (int s = lane; s < p.parts; s += 32) m = fmaxf(m, p.part_ml[s * R + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // a lane weighs a part each, then all lanes add up the parts; the loads of several are under way at a time
    float l = 0.f, v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.f;
    for (int s0 = 0; s0 < p.parts; s0 += 32) {
        const float2 ml = s0 + lane < p.parts ? p.part_ml[(s0 + lane) * R + row] : make_float2(-INFINITY, 0.f);
        const float mine = ml.x == -INFINITY ? 1.f : ex2(ml.x - m);  // 1: zeros, all of whose keys are hidden, or NaN
        l = fmaf(ml.y, mine, l);
        const float* part = p.part + (s0 * R + row) * D + lane * V;
        const int n = min(32, p.parts - s0);
#pragma unroll 8
        for (int s = 0; s < n; ++s, part += R * D) {
            const float f = __shfl_sync(0xffffffffu, mine, s);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = fmaf(part[e], f, v[e]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const bool empty = range.x >= range.y;
    const float inv = empty ? 0.f : 1.f / l;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.O) + (b * p.o_b + h * p.o_h + i * p.o_n) + lane * V);
    uint32_t* rest = p.rest ? reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.rest) + row * D + lane * V) : nullptr;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
        const float a = empty ? 0.f : v[e] * inv, c = empty ? 0.f : v[e + 1] * inv;
        const uint32_t u = pack_bf16(a, c);
        out[e / 2] = u;
        if (rest) rest[e / 2] = pack_bf16(a - __uint_as_float(u << 16), c - __uint_as_float(u & 0xffff0000u));
    }
    if (lane == 0) p.LSE[row] = empty ? -INFINITY : fmaf(m, kLn2, logf(l));
}

namespace {
template <int D, int TERMS>
cudaError_t launch_attn_d(const CUtensorMap* m, const AttnFwdParams& p, const ScoreParams& sp, int ctas, cudaStream_t st) {
    constexpr int bytes = AttnSmem<D>::alloc;
    static_assert(bytes <= 232448, "shared memory");
    auto k = attn_fwd_kernel<D, TERMS>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(k, bytes, &done);
    if (e != cudaSuccess) return e;
    k<<<ctas, kAfThreads, bytes, st>>>(m[0], m[1], m[2], p, sp);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.parts == 1) return e;
    const int64_t rows = int64_t(p.B) * p.H * p.Nq;
    attn_combine_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, st>>>(p, sp);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_attn_fwd(int d, const CUtensorMap* maps, const AttnFwdParams& p, const ScoreParams& sp, int ctas,
                            cudaStream_t stream) {
    if (p.rest)  // for training: see the second term's use above
        return d == 128 ? launch_attn_d<128, 2>(maps, p, sp, ctas, stream) : launch_attn_d<64, 2>(maps, p, sp, ctas, stream);
    return d == 128 ? launch_attn_d<128, 1>(maps, p, sp, ctas, stream) : launch_attn_d<64, 1>(maps, p, sp, ctas, stream);
}

}  // namespace streamkl
