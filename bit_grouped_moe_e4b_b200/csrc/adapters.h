// Host-side launchers of the adapter path's kernels, used by the C-ABI layer
// (api.cu): token rows by expert and back (csrc/rows.cu), the gated activation
// on stored rows (csrc/glu.cu) and the grouped low-rank adapters (csrc/lora.cu,
// csrc/lora_tc.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "e4b.h"

namespace e4b {

// bf16 rows in global memory: row i at p + i * ld.
struct RowsIn {
  const uint16_t* p;
  int64_t ld;
};
struct RowsOut {
  uint16_t* p;
  int64_t ld;
};

cudaError_t launch_permute(RowsIn x, int64_t T, int64_t H, const int32_t* perm, int32_t top_k,
                           const int64_t* offsets, int32_t E, int64_t R_max, RowsOut xs, cudaStream_t st, int sms);
// y[t] = bf16(sum_j w_j rows[inv[t * top_k + j]]), w_j = gates[t * top_k + j], or 1 without gates.
cudaError_t launch_sum_slots(RowsIn rows, int64_t R_max, int64_t H, const int32_t* inv, const float* gates,
                             int64_t T, int32_t top_k, RowsOut y, cudaStream_t st, int sms);
cudaError_t launch_unpermute_backward(RowsIn dy, RowsIn ys, int64_t R_max, int64_t H, const int32_t* inv,
                                      const float* gates, int64_t T, int32_t top_k, RowsOut dys, float* dgates,
                                      cudaStream_t st, int sms);

cudaError_t launch_glu(const e4b_glu_args& a, bool backward, cudaStream_t st, int sms);

// Largest adapter rank of the kernels.
constexpr int kLoraMaxRank = 64;
size_t lora_workspace_bytes(int64_t G, int r, int64_t N, int64_t K, int64_t R_max, bool backward, int sms);
cudaError_t launch_lora(const e4b_lora_args& a, void* ws, uint32_t flags, cudaStream_t st, int sms, int* launches);
cudaError_t launch_lora_backward(const e4b_lora_args& a, void* ws, uint32_t flags, cudaStream_t st, int sms,
                                 int* launches);

}  // namespace e4b
