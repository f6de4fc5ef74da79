// cache8.cuh -- parameter blocks of the 8-bit cache (cache8.cu, cache8_attn.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace streamkl {

constexpr int kCacheLeastExponent = -100;  // of a page's scale

// Pages of T tokens: values [pages, H_kv, T, d] in e4m3, scales [pages, H_kv].
// Token j of sequence b stands in page table[b][j / T], row j % T.
struct CacheView {
    uint8_t* values[2];  // keys, values
    float* scales[2];
    int pages, H_kv, T, d;
    int log_T;               // T is a power of two
    const int32_t* table;    // [B, M]
    const int32_t* lengths;  // [B]
    int B, M;
};

struct CacheAppendParams {
    CacheView c;
    const void* x[2];      // new tokens [B, H_kv, N, d] bf16
    int64_t x_b[2], x_h[2], x_n[2];
    int N;
    const int32_t* counts;  // [B] or null: N
};

struct CacheReadParams {
    CacheView c;
    void* y[2];            // [B, H_kv, N, d] bf16
    int64_t y_b[2], y_h[2], y_n[2];
    int N;
};

struct CacheAttnParams {
    CacheView c;
    int H, Nq, group;
    int tile_rows;         // 8 (one tile holds a key head's group x Nq rows) or 16
    int row_groups;        // of up to kCacheTeams tiles, of those rows
    int teams;             // tiles that a CTA works on at a time: 1, 2, 4 or 8
    int spread;            // CTAs take equal shares of all chunks, and parts are combined; else a cluster per segment
    int cluster;           // its CTAs, each with a share of the segment's chunks
    const void* Q;         // [B, H, Nq, d] bf16
    int64_t q_b, q_h, q_n;
    void* O;               // [B, H, Nq, d] bf16
    int64_t o_b, o_h, o_n;
    float* LSE;            // [B, H, Nq]
    float scale_log2e;
    float* part;           // spread: [CTAs][2][tile_rows teams][d] sums and
    unsigned int* status;
    unsigned long long wait_ns;
    int inject_stall;
    float4* part_state;    // [CTAs][2][tile_rows teams] their references
};

constexpr int kCacheTeams = 8;

}  // namespace streamkl
