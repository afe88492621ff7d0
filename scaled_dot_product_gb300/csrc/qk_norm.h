// The query/key norm: its problem and launch function.
#pragma once

#include "device_words.h"
#include "internal.h"
#include "norm_split.h"

namespace sdpa {

// RMS norm of query and key heads followed by the rotation, or its gradient.
struct NormSide {
  View x, dy, y;             // input, upstream gradient (backward), output (backward: dx)
  const void* w;             // (D)
  void* dw;                  // backward: (D)
  int N;                     // heads
};
struct NormJob {
  NormSide side[2];          // queries, keys
  int B, S, tokens, D, R;    // tokens = B * S; R = 0: no rotation
  int interleaved;
  const void* cos_c;
  const void* sin_c;
  const int64_t* positions;  // (tokens), or nullptr: one cache row per token
  int64_t max_pos;
  float eps, inv_D;
};
// part == nullptr: forward; else the backward with its partial sums there.
cudaError_t launch_qk_norm(sdpa_dtype dt, const NormJob& j, float* part, cudaStream_t st);
cudaError_t take_norm_status(int* status);
cudaError_t take_bounds_norm(int* site);

}  // namespace sdpa
