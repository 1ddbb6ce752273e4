// attention_spans.cu -- the key intervals of packed documents, as the
// attention kernels take them.
#include <cuda_runtime.h>

#include "bounds.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace {

__global__ void __launch_bounds__(256) spans_kernel(const int32_t* __restrict__ offsets, int64_t documents,
                                                    const int32_t* __restrict__ prefix, int causal, int64_t tokens,
                                                    int2* __restrict__ spans, const Extent xs) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= tokens) return;
    // the document of token i: the last offset at or below i (empty documents
    // share their offset with the next one, which is then the last)
    int64_t a = -1, b = documents;   // offsets[a] <= i < offsets[b], with offsets[-1] = -inf
    while (b - a > 1) {
        const int64_t m = (a + b) >> 1;
        if (offsets[m] <= i) a = m;
        else b = m;
    }
    int2 s = make_int2(0, 0);
    if (a >= 0 && i < offsets[a + 1]) {
        const int64_t start = offsets[a], end = offsets[a + 1] < tokens ? offsets[a + 1] : tokens;
        int64_t hi = end;
        if (causal) {
            hi = i + 1;
            if (prefix) {
                const int64_t to = start + prefix[a];
                hi = to > hi ? to : hi;
                hi = hi > end ? end : hi;
            }
        }
        s = make_int2((int)(start < 0 ? 0 : start), (int)hi);
    }
    store_out(spans + i, s, xs);
}

}  // namespace

cudaError_t launch_attention_spans(const int32_t* offsets, int64_t documents, const int32_t* prefix, bool causal,
                                   int64_t tokens, int32_t* spans, cudaStream_t stream) {
    spans_kernel<<<(unsigned)((tokens + 255) / 256), 256, 0, stream>>>(offsets, documents, prefix, causal ? 1 : 0, tokens,
                                                                       reinterpret_cast<int2*>(spans),
                                                                       extent_of(spans, tokens * 8));
    return cudaGetLastError();
}

cudaError_t attention_spans_bounds_read_and_clear(uint64_t* n) { return bounds_read_and_clear_local(n); }

}  // namespace nvfp4
