// The contraction pass over one row buffer of the adapters (csrc/lora_tc.cu),
// as the adapters' host code (csrc/lora.cu) sees it.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace e4b {

// Z: bf16 rows of C values, by groups of positions as in e4b_lora. The pass
// reads every row once and computes either or both of
//   out[p] = w_g W_g z_i         (W: [G, r, C], or [G, C, r] transposed; w 1 without scale_out)
//   grad_g = sum_p w_g v[p] z_i^T  ([G, r, C], or [G, C, r] transposed; w 1 without scale_v)
struct ContractArgs {
  int G, r;
  int64_t C, R_max;
  const int64_t* offsets;
  const int32_t* row;  // or null
  int64_t rows;        // rows of z
  const uint16_t* z;
  int64_t ld_z;
  const float* scale;  // or null

  const uint16_t* w;   // or null without out
  bool w_t;            // W is [G, C, r]
  float* out;          // [blocks][R_max][r]: one part per column block (contract_blocks); or null
  bool scale_out;

  const float* v;      // [R_max, r], or null without grad
  bool scale_v;
  float* grad;         // or null
  bool grad_t;         // grad is [G, C, r]
  bool accumulate;     // add to grad
  float* grad_part;    // contract_part_bytes

  bool follows;        // the launch before it on the stream belongs to the same call
  int32_t* status;     // or null
  bool no_wait;        // waits give up at once (tests)
};

// Column blocks of a pass: parts of `out`.
int contract_blocks(int G, int r, int64_t C, int64_t R_max, bool out, bool grad, int sms);
// At least the column blocks of a pass with `out` times its rows, for every
// number of rows up to R_max; never less for more rows.
int64_t contract_out_rows(int G, int r, int64_t C, int64_t R_max, bool grad, int sms);
// Bytes of grad_part, whatever the rows.
size_t contract_part_bytes(int r, int64_t C, bool out, int sms);
cudaError_t launch_contract(const ContractArgs& a, cudaStream_t st, int sms);
// What a pass with `grad` leaves to do: the sums of groups whose rows several
// CTAs took, zeros for groups without rows. After launch_contract, with the
// same arguments, of up to two passes.
cudaError_t launch_contract_finish(const ContractArgs* a, const ContractArgs* b, cudaStream_t st, int sms);

}  // namespace e4b
