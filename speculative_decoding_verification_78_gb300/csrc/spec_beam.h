// spec_beam.h -- arguments and launches of the beam operators.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_verify.h"

namespace specv {

struct BeamArgs {
  const void *logits;      // [B, K, V]
  const float *scores;     // [B, K]
  const int32_t *done;     // [B, K] or null
  int32_t *tokens;         // [B, n]
  int32_t *parents;        // [B, n]
  float *out_scores;       // [B, n]
  int32_t *status;
  uint2 *part;             // [B * K * C] (maximum, sum) of each unit
  float4 *quarters;        // [B * K * C] the maxima of its quarters
  int B, K, V, C, n, pad;
  int units;               // B * K * C
};

struct ReorderArgs {
  const char *in[SPEC_MAX_STATES];
  char *out[SPEC_MAX_STATES];
  long long bytes[SPEC_MAX_STATES];   // of a row
  int grain[SPEC_MAX_STATES];         // 16, 8, 4, 2 or 1: what every address and size is a multiple of
  const int32_t *parents;
  int32_t *status;
  int states, rows_in, rows_out;
};

// units per row: a warp's 32 x 8 vectors of 16 bytes, counted from the row's first element
inline int beam_chunks(int V, int dtype) {
  const int per = (dtype == SPEC_BF16 ? 8 : 4) * 256;
  return (V + per - 1) / per;
}
cudaError_t launch_beam_select(int dtype, const BeamArgs &a, int sms, cudaStream_t stream);
cudaError_t launch_beam_reorder(const ReorderArgs &a, cudaStream_t stream);

}  // namespace specv
