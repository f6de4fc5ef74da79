// attn.cuh -- parameter blocks of the attention over whole prompts (attn_fwd.cu,
// attn_bwd.cu).
#pragma once

#include <cstdint>

#include "common.cuh"
#include "score.cuh"

namespace streamkl {

// Division of 0 <= n < 2^31 by a number that the host knows, by Granlund and Montgomery's method (Division by Invariant
// Integers using Multiplication, 1994): with 2^s >= d the smallest such power and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (n m / 2^32 + n) / 2^s, all rounded down.  A CTA's first steps are a chain of
// six of them (the smallest call, in a graph: 8.2 us with the compiler's, 7.8 with these).
struct FastDiv {
    uint32_t d, m;
    int s;
    static FastDiv by(int64_t d) {
        FastDiv f{static_cast<uint32_t>(d), 0, 0};
        while ((int64_t(1) << f.s) < d) ++f.s;
        f.m = static_cast<uint32_t>((uint64_t(1) << 32) * static_cast<uint64_t>((int64_t(1) << f.s) - d) / static_cast<uint64_t>(d) + 1);
        return f;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int of(int n) const {
        const uint32_t t = __umulhi(static_cast<uint32_t>(n), m);
        return static_cast<int>(s == 0 ? n : (t + ((n - t) >> 1)) >> (s - 1));
    }
#endif
};

// Forward.  A 128-row tile holds `heads` query heads of one key head with `rows`
// rows each (few rows: several heads share a tile; else one head and 128 rows).  A
// work item is a pair of tiles that read the same keys: two head blocks, or two
// neighbouring query tiles.
struct AttnFwdParams {
    int B, H, H_kv, Nq, Nk;
    int group;               // query heads per key head
    int heads, rows;         // of a tile
    int blocks, q_tiles;     // tiles of a key head: head blocks x query tiles
    int pair_heads;          // a pair is two head blocks (else two query tiles)
    int units_h, units_q;    // pairs of a key head
    int dual;                // a tile without another to pair with stands twice, each with every second key tile
    int num_splits;
    int parts;               // of a row: num_splits, twice that if dual; 1: outputs
    // units in groups of heads, tiles slow and heads fast in a group (see grouped_order): heads of a group, of the last
    // one, and units of a group
    FastDiv order_group, order_last, order_units;
    FastDiv by_splits, by_units_h, by_H_kv, by_rows;
    float c;                 // softmax scale * log2(e)
    void* O;                 // bf16, strided
    int64_t o_b, o_h, o_n;
    void* rest;              // bf16 [B, H, Nq, d] or null: O before its rounding, less O
    float* LSE;              // [B, H, Nq]
    float* part;             // several parts: [parts][B*H*Nq][d] sums of 2^(x - m) v
    float2* part_ml;         // [parts][B*H*Nq]: m (log2) and the sum of 2^(x - m)
    unsigned int* status;
    unsigned long long wait_ns;
    int inject_stall;
};

// Backward.  Query tiles of 64 rows, key tiles of 128.
struct AttnBwdParams {
    int B, H, H_kv, Nq, Nk;
    int group;
    int num_q_tiles, num_k_tiles;
    int num_splits;          // CTAs that share a key tile's query tiles
    int order_group;
    float scale, c;          // softmax scale; times log2(e)
    const void* K;           // bf16, strided; for keys that are not finite
    int64_t k_b, k_h, k_n;
    const void* dO;          // bf16, strided
    int64_t g_b, g_h, g_n;
    const void* O;           // bf16, strided
    int64_t o_b, o_h, o_n;
    const void* rest;        // bf16 [B, H, Nq, d] or null
    const float* LSE;
    void* dQ;                // bf16 [B, H, Nq, d]
    void* dK;                // bf16 [B, H_kv, Nk, d]
    void* dV;
    float* dQacc;            // float32 [B, H, Nq, d]: the key tiles' terms are added here
    float* rows;             // [B*H][q tiles][2][64]: -LSE (log2) and -scale sum(dO O) of each row
    void* keys;              // [B][q tiles] KeyBlock
    float* parts;            // several splits: [2 (dK, dV)][splits][B*H_kv*Nk][d]
    unsigned int* status;
    unsigned long long wait_ns;
    int inject_stall;
};

}  // namespace streamkl
