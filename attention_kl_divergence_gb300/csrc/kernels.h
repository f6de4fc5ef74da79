// kernels.h -- host-side launchers of the CUDA kernels (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "attn.cuh"
#include "cache8.cuh"
#include "common.cuh"
#include "score.cuh"

namespace streamkl {

// maps = {Q1, K1, Q2, K2}; Q maps use 128-row boxes (tile) or 16-row boxes (decode).
cudaError_t launch_fwd_tile(int d, const CUtensorMap* maps, const FwdParams& p, int ctas, cudaStream_t stream);
cudaError_t launch_fwd_decode(int d, const CUtensorMap* maps, const FwdParams& p, int ctas, cudaStream_t stream);
cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream);
int fwd_tile_stages(int d);

// Backward.  bwd_q maps: Q boxes of 128 rows, K boxes of 64 rows; bwd_kv maps:
// Q boxes of 64 rows, K boxes of 128 rows.
cudaError_t launch_bwd_q(int d, int setting, const CUtensorMap* maps, const BwdParams& p, int ctas,
                         cudaStream_t stream);
cudaError_t launch_to_bf16(const float* in, void* out, size_t n, int sms, cudaStream_t stream);
cudaError_t launch_bwd_kv(int d, int setting, bool fused, const CUtensorMap* maps, const BwdParams& p, int ctas,
                          cudaStream_t stream);
// Key-split backward for at most 16 query rows per key head: Q maps with boxes
// of Nq rows x kv_group heads, K maps with 128-row boxes; p.num_splits set.
// Joint backward (both sides from one recompute of the scores per kernel):
// qmaps as for bwd_q, kvmaps as for bwd_kv; p.dQ/p.dK take the teacher's
// gradients, p.dQb/p.dKb the student's.
cudaError_t launch_bwd_joint(int d, const CUtensorMap* qmaps, const CUtensorMap* kvmaps, const BwdParams& pq,
                             const BwdParams& pkv, int ctas_q, int ctas_kv, cudaStream_t stream);
cudaError_t launch_bwd_decode(int d, int setting, const CUtensorMap* maps, const BwdParams& p, int ctas,
                              cudaStream_t stream);

// Score-modified divergence; mode: kScore* of score.cuh.  Maps as for fwd_tile /
// fwd_decode, and as for bwd_kv.
cudaError_t launch_score_fwd(int d, int mode, bool decode, const CUtensorMap* maps, const FwdParams& p,
                             const ScoreParams& sp, int ctas, cudaStream_t stream);
size_t score_bwd_row_bytes(int64_t bh, int q_tiles);     // workspace of sp.rows and
size_t score_bwd_key_bytes(int64_t batch, int q_tiles);  // of sp.keys
cudaError_t launch_score_bwd(int d, int setting, int mode, const CUtensorMap* maps, const BwdParams& p,
                             const ScoreParams& sp, int ctas, int sms, cudaStream_t stream);

// Attention over whole prompts.  maps = {Q, K, V}: Q boxes of p.rows rows x
// p.heads heads, K and V boxes of 128 rows.
cudaError_t launch_attn_fwd(int d, const CUtensorMap* maps, const AttnFwdParams& p, const ScoreParams& sp, int ctas,
                            cudaStream_t stream);

// Its gradients.  maps = {Q, K, V, dO}: Q and dO boxes of 64 rows, K and V boxes of 128.
size_t attn_bwd_row_bytes(int64_t bh, int q_tiles);     // workspace of p.rows and
size_t attn_bwd_key_bytes(int64_t batch, int q_tiles);  // of p.keys
cudaError_t launch_attn_bwd(int d, const CUtensorMap* maps, const AttnBwdParams& p, const ScoreParams& sp, int ctas, int sms,
                            cudaStream_t stream);

// 8-bit cache: new tokens in, tokens out, and attention of a few new tokens over it.
cudaError_t launch_cache8_append(const CacheAppendParams& p, cudaStream_t stream);
cudaError_t launch_cache8_read(const CacheReadParams& p, cudaStream_t stream);
// maps = {keys, values}: the pool's rows of d bytes, boxes of 16 rows.
cudaError_t launch_cache8_attn(const CUtensorMap* maps, const CacheAttnParams& p, int ctas, cudaStream_t stream);

cudaError_t launch_key_ranges(const KeyRangeParams& p, cudaStream_t stream);

// Norm and rotation of query and key heads.  norm_rope_bwd_ctas plans the
// gradient pass: its CTAs, and how many of them take the query heads.
cudaError_t launch_norm_rope_fwd(int d, const NormRopeParams& p, cudaStream_t stream);
void norm_rope_bwd_ctas(const NormRopeParams& p, int sms, int* ctas_q, int* ctas);
cudaError_t launch_norm_rope_bwd(int d, const NormRopeParams& p, int ctas, cudaStream_t stream);
cudaError_t launch_rope_table(const double* inv_freq, int64_t rows, int half, float* table, int sms,
                              cudaStream_t stream);

}  // namespace streamkl
