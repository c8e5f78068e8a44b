// Host entry of the kernels that kvo_paged_chunk_attn takes for a few new tokens of each request.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "kvo.h"

namespace kvo {

constexpr int FEW_ROWS = 16;       // tokens x query heads of a group

size_t paged_few_workspace(const kvo_paged_cache* c, int r, int64_t max_new, int64_t max_len);
// The maps' boxes are 16 rows of the pools.
cudaError_t launch_paged_few(const kvo_paged_cache* c, const CUtensorMap& mk, const CUtensorMap& mv, const void* q, int64_t q_stride,
                             int64_t total, int r, const int32_t* cu, const int32_t* lens, int64_t max_new, int64_t max_len, void* o,
                             float* lse, void* workspace, int32_t* status, cudaStream_t s);

}  // namespace kvo
