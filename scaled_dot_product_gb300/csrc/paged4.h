// Paged caches of 4 bits a value, and the step's page tables: the problems as the kernels see them,
// and their launch functions.
//
// A cached head row of D channels is a record of D / 2 bytes of codes (channel 2j in the low half of
// byte j, channel 2j + 1 in the high half) and then, for each 32 channels, a minimum and a scale in
// the model's type T.  A value is minimum + scale * code.
#pragma once

#include "paged.h"

namespace sdpa {

constexpr int kQ4Group = 32;
__host__ __device__ constexpr int q4_row_bytes(int D, int esize) { return D / 2 + D / kQ4Group * 2 * esize; }

struct Paged4Append {
  int tokens, Nkv, H, Hv;
  int num_pages, page_size;
  View k, v, k_held, v_held;      // packed rows; held.p == nullptr: not wanted
  View kp, vp;                    // strides in bytes
  const int64_t* slots;
  const int64_t* positions;
  const void* cos_c;
  const void* sin_c;
  int64_t max_pos;
  int R, interleaved;
  int vec_rot;                    // pairs and caches in whole 16-byte vectors
  uint32_t tok_mul, tok_shift, k_mul, k_shift, v_mul, v_shift, page_mul, page_shift;      // divisions (paged_magic)
};
cudaError_t launch_paged4_append(sdpa_dtype dt, const Paged4Append& a, cudaStream_t st);
cudaError_t take_paged4_append_status(int* status);
cudaError_t take_bounds_paged4_append(int* site);

// Attention over such a cache: PagedAttn with kp and vp in bytes.
cudaError_t launch_paged4_attn(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name);
PagedKernel paged4_kernel(const PagedAttn& a, sdpa_dtype dt);
size_t paged4_workspace(int H, int Hv, sdpa_dtype dt);
bool paged4_mma_supported(int H, int Hv, sdpa_dtype dt);
size_t paged4_mma_workspace(int Hv);     // of its widest tile
int paged4_mma_rows(int H);              // its rows
cudaError_t launch_paged4_mma(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name);
bool paged4_tc_supported(const PagedAttn& a, sdpa_dtype dt);
size_t paged4_tc_workspace(int Hv);
cudaError_t launch_paged4_tc(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name);
cudaError_t take_paged4_tc_status(int* status, int* timeout);
cudaError_t take_bounds_paged4_tc(int* site);
cudaError_t take_paged4_simt_status(int* status);
cudaError_t take_paged4_mma_status(int* status, int* timeout);
cudaError_t take_bounds_paged4_mma(int* site);
cudaError_t take_bounds_paged4_simt(int* site);

struct PagedTables {
  int B, tokens, page_size, max_pages, num_pages, cap;
  uint32_t page_mul, page_shift;
  int32_t* table;
  int64_t table_stride;
  const int32_t* past;
  const int32_t* fresh;           // new tokens of each sequence; negative: it has ended
  int32_t* free_pages;            // (num_pages): a stack, free_count[0] entries deep
  const int32_t* free_count;
  int32_t* kv_lens;
  int32_t* cu;
  int64_t* positions;
  int64_t* slots;
  int32_t* free_count_out;
};
constexpr int kTablesMaxB = 8192;
cudaError_t launch_paged_tables(const PagedTables& a, cudaStream_t st);
cudaError_t take_paged_tables_status(int* status);
cudaError_t take_bounds_paged_tables(int* site);

// Status bits beside those of paged.h.
enum { kPagedNoPages = 8, kPagedBadSlot = 16, kPagedFullList = 32 };

}  // namespace sdpa
