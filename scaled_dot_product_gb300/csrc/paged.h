// Paged caches: the problem as the kernels see it, and their launch functions.
#pragma once

#include "device_words.h"
#include "internal.h"

namespace sdpa {

// A ragged batch over a paged cache.  Sequence b brings the new tokens [cu[b], cu[b+1]) of the
// packed rows; kv_lens[b] counts its keys with them, so new token i sits at key position
// kv_lens[b] - n_b + i.  Key j of sequence b lies in page table[b][j / page_size], slot
// j % page_size.
struct Paged {
  int B, tokens, Nq, Nkv, H, Hv, group;
  int num_pages, page_size, max_pages;
  int cap;                        // max_pages * page_size: keys the table can address
  uint32_t page_mul, page_shift;  // j / page_size = (j * page_mul) >> page_shift for 0 <= j < 2^31
  uint32_t group_mul, group_shift;          // r / group likewise
  View kp, vp;                    // (num_pages, Nkv, page_size, H / Hv)
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* cu;              // nullptr: every sequence brings tokens / B rows
  int uniform;
};

struct PagedAttn {
  Paged g;
  View q, y;                      // packed rows: sh per head, ss per token
  float scale, softcap;
  int causal;                     // 0: every key of the sequence
  int window;                     // 0: unlimited
  const void* head_sink;
  int max_new;                    // hint: most new tokens of one sequence
};

struct PagedRot {                 // rotation of appended keys; R = 0: none
  const void* cos_c;
  const void* sin_c;
  int64_t max_pos;
  int R, interleaved;
};

cudaError_t launch_paged_append(sdpa_dtype dt, const Paged& g, const View& k, const View& v, const PagedRot& rot,
                                cudaStream_t st);

enum PagedKernel { kPagedSimt = 0, kPagedMma = 1, kPagedTc = 2 };
PagedKernel paged_kernel(const PagedAttn& a, sdpa_dtype dt);
// Workspace of the attention: enough for every kernel and tile that the type and the head sizes
// admit, so that it changes with nothing else (rows, lengths, hints, pages, strides) and a caller
// can keep one for all its calls.
size_t paged_workspace(int H, int Hv, sdpa_dtype dt);
cudaError_t launch_paged_attn(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name);
bool paged_mma_supported(int H, int Hv, sdpa_dtype dt);
size_t paged_mma_workspace(int Hv);      // of its widest tile
cudaError_t launch_paged_mma(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name);

cudaError_t take_bounds_append(int* site);
cudaError_t take_bounds_paged_simt(int* site);
cudaError_t take_bounds_paged_mma(int* site);
cudaError_t take_bounds_paged_tc(int* site);
cudaError_t take_paged_append_status(int* status);
// Whether TMA boxes of at least eight rows tile the pages.
bool paged_boxes(const PagedAttn& a);
bool paged_tc_supported(const PagedAttn& a, sdpa_dtype dt);
size_t paged_tc_workspace(int Hv);
cudaError_t launch_paged_tc(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name);
cudaError_t take_paged_simt_status(int* status);
cudaError_t take_paged_mma_status(int* status, int* timeout);
cudaError_t take_paged_tc_status(int* status, int* timeout);

#ifdef __CUDACC__
// Status bits of the device words: reported by sdpa_query_status as SDPA_ERR_INVALID.
enum { kPagedBadPage = 1, kPagedBadLength = 2, kPagedBadPosition = 4 };

__device__ __forceinline__ int page_div(const Paged& g, int j) {
  return (int)(((uint64_t)(uint32_t)j * g.page_mul) >> g.page_shift);
}

__device__ __forceinline__ int group_div(const Paged& g, int r) {
  return (int)(((uint64_t)(uint32_t)r * g.group_mul) >> g.group_shift);
}

// New-token rows [t0, t0 + n) and keys T of sequence b, clamped to what the arrays can hold
// (bad is set when something had to be clamped).
struct SeqInfo { int t0, n, T; };
__device__ __forceinline__ SeqInfo seq_info(const Paged& g, int b, bool& bad) {
  SeqInfo s;
  int T = g.lens[b];
  if (g.cu) {
    const int c0 = g.cu[b], c1 = g.cu[b + 1];
    s.t0 = min(max(c0, 0), g.tokens);
    const int e = min(max(c1, s.t0), g.tokens);
    s.n = e - s.t0;
    bad = bad || c0 != s.t0 || c1 != e;
  } else {
    s.t0 = b * g.uniform;
    s.n = g.uniform;
  }
  s.T = min(max(T, 0), g.cap);
  bad = bad || s.T != T;
  return s;
}
#endif

}  // namespace sdpa
