// host.h -- argument checks, launch planning and tensor maps shared by the
// entry points of the C ABI (defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/streamkl.h"

namespace streamkl {

constexpr int kMaxSplits = 64;
constexpr int64_t kDefaultWaitNs = 2000000000LL;

bool aligned16(const void* p);
streamkl_status check_shape(const streamkl_shape* s, int causal);
int kv_heads(const streamkl_shape* s);
streamkl_status device_sms(int* sms);
int choose_splits(int64_t units, int k_tiles, int slots);
int decode_splits(int64_t units, int k_tiles, int sms);
int order_group(int64_t heads, int tiles, int sms);
int bwd_splits(int64_t units, int64_t iterations, int sms);
bool make_map(CUtensorMap* m, const void* ptr, const streamkl_shape* s, bool is_q, int box_rows, int box_heads = 1);
bool make_map_strided(CUtensorMap* m, const void* ptr, int d, int64_t N, int heads, int B, const streamkl_strides& st,
                      int box_rows, int box_heads = 1);
bool make_map_bytes(CUtensorMap* m, const void* ptr, int d, int64_t rows);
// The dynamic shared memory that a kernel asks for, set once per device (the call costs a small launch a tenth of its
// host time).  `done`: one word per kernel, bit k for device k.
template <typename Kernel>
cudaError_t allow_smem(Kernel k, int bytes, std::atomic<uint64_t>* done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (e != cudaSuccess || (done->load(std::memory_order_relaxed) & bit)) return e;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
    return e;
}
float resolve_scale(float scale, int d);
int64_t wait_limit(const streamkl_options* opt);

}  // namespace streamkl
