// key_ranges.cu -- the key range of each query row from causal, window, prefix,
// document and length masks.  One thread per row; a few bytes per row.
#include "common.cuh"
#include "kernels.h"

namespace streamkl {

__global__ void __launch_bounds__(256) key_ranges_kernel(const KeyRangeParams p) {
    const int b = blockIdx.y;
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    const int kl = p.k_lengths ? min(max(p.k_lengths[b], 0), p.Nk) : p.Nk;
    const int ql = p.q_lengths ? min(max(p.q_lengths[b], 0), p.Nq) : p.Nq;
    if (i == 0) p.offset[b] = kl - ql;
    if (i >= p.Nq) return;
    const int64_t pos = static_cast<int64_t>(i) + kl - ql;
    int64_t lo = 0, hi = kl;
    if (p.causal) hi = min(hi, pos + 1);
    if (p.window > 0) {
        lo = max(lo, pos - p.window + 1);
        hi = min(hi, pos + p.window);
    }
    if (p.prefix) hi = max(hi, static_cast<int64_t>(min(p.prefix[b], kl)));
    if (p.docs) {  // the document with docs[m] <= pos < docs[m + 1]
        const int32_t* d = p.docs + static_cast<size_t>(b) * p.doc_stride;
        int lower = 0, upper = p.num_docs;  // number of bounds <= pos
        while (lower < upper) {
            const int mid = (lower + upper) / 2;
            if (d[mid] <= pos)
                lower = mid + 1;
            else
                upper = mid;
        }
        if (lower == 0 || lower == p.num_docs) {
            hi = 0;
        } else {
            lo = max(lo, static_cast<int64_t>(d[lower - 1]));
            hi = min(hi, static_cast<int64_t>(d[lower]));
        }
    }
    const bool any = i < ql && lo < hi;
    const size_t r = static_cast<size_t>(b) * p.Nq + i;
    p.begin[r] = any ? static_cast<int32_t>(lo) : 0;
    p.end[r] = any ? static_cast<int32_t>(hi) : 0;
}

cudaError_t launch_key_ranges(const KeyRangeParams& p, cudaStream_t stream) {
    key_ranges_kernel<<<dim3((p.Nq + 255) / 256, p.B), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace streamkl
