// host.h -- argument checks, launch planning and tensor maps shared by the
// entry points of the C ABI (defined in api.cu).
#pragma once

#include <cuda.h>
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
bool make_map(CUtensorMap* m, const void* ptr, const streamkl_shape* s, bool is_q, int box_rows, int box_heads = 1);
float resolve_scale(float scale, int d);
int64_t wait_limit(const streamkl_options* opt);

}  // namespace streamkl
