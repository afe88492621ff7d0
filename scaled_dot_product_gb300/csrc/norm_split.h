// How many blocks of the query/key norm's gradient walk the query rows and how many the key rows.
// Host arithmetic alone, so that it can be checked without a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace sdpa {

// Most blocks of the backward: each leaves D partial sums of dw in the workspace.
constexpr int kNormBwdMaxBlocks = 152 * 2;

struct NormBwdBlocks {
  int q, k;
};

// The blocks are dealt by rows, at least one a side and no more than a side has work for (want_q,
// want_k): q + k <= kNormBwdMaxBlocks, however unequal the head counts are (the key side's rounded
// share leaves the query side its one).
inline NormBwdBlocks norm_bwd_blocks(int Nq, int Nkv, int want_q, int want_k) {
  const int total = (int)std::min<int64_t>((int64_t)want_q + want_k, kNormBwdMaxBlocks);
  const double share = (double)Nkv / ((double)Nq + Nkv);
  NormBwdBlocks b;
  b.k = std::max(1, std::min({want_k, total - 1, (int)(share * total + 0.5)}));
  b.q = std::max(1, std::min(want_q, total - b.k));
  return b;
}

}  // namespace sdpa
