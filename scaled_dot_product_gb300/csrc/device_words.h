// The words that the kernels of one translation unit report in.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>

namespace sdpa {

// Reads a translation unit's words with one copy, and clears them if any is set.
template <int N>
cudaError_t take_words(const int (&words)[N], int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, words, sizeof words);
  if (e == cudaSuccess && std::any_of(out, out + N, [](int v) { return v != 0; })) {
    const int zero[N] = {};
    e = cudaMemcpyToSymbol(words, zero, sizeof words);
  }
  return e;
}

}  // namespace sdpa
