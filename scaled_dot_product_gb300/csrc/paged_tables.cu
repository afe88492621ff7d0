// The page tables of a step, made on the device from past and new lengths: pages of ended sequences
// go back to the list of free pages, grown sequences take theirs from it, and every new token gets its
// row offset, position and cache slot.
//
// One launch of one cluster.  Every CTA scans all sequences for itself (a running sum of the rows,
// of the pages given back and of the pages taken, kept in shared memory), so nothing but the list of
// free pages passes between CTAs; tokens and pages are then dealt to the threads of the whole
// cluster, each finding its sequence by bisection in shared memory.  A thread per sequence would
// leave a long prompt's tokens to one thread.  A page taken is the list's entry from the top down, in
// the order of sequences, whatever the number of threads: results do not vary.  The cluster's barrier
// orders the entries given back before those taken, and the inputs' reads before the outputs that may
// be the inputs themselves.  Bound by latency (a chain of lengths, scans, barrier, list or table,
// slot): 64 sequences of a token, one ended, 7.5 us, 2000 sequences with 15,000 tokens 16.4, 48 prompts of 184,000 tokens 7.7.
#include <algorithm>

#include "paged4.h"
#include "paged_sched.cuh"

namespace sdpa {

static __device__ int g_tables_status[1];

namespace {

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_size() {
  int r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Last i in [0, n) with at[i] <= x, for at[0] <= x, at not decreasing.
__device__ __forceinline__ int last_not_above(const int* at, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

constexpr int kAhead = 4;        // loads of a lane in flight

// Ids of a row's first h entries that are in range, counted by the warp; 32 U of them are on their way together.
template <int U>
__device__ __forceinline__ int count_ids(const int32_t* row, int h, int num_pages, int lane) {
  int c = 0;
#pragma unroll 1
  for (int j0 = 0; j0 < h; j0 += 32 * U) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = j0 + u * 32 + lane < h ? row[j0 + u * 32 + lane] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) c += (unsigned)id[u] < (unsigned)num_pages;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  return c;
}
// The same ids onto the list, in order, from entry `at` on.
template <int U>
__device__ __forceinline__ void give_back(const int32_t* row, int h, int32_t* list, int64_t at, int num_pages, int lane) {
#pragma unroll 1
  for (int j0 = 0; j0 < h; j0 += 32 * U) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = j0 + u * 32 + lane < h ? row[j0 + u * 32 + lane] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool ok = (unsigned)id[u] < (unsigned)num_pages;
      const unsigned m = __ballot_sync(0xffffffffu, ok);
      const int64_t to = at + __popc(m & ((1u << lane) - 1));
      if (ok && to < num_pages) list[to] = id[u];
      at += __popc(m);
    }
  }
}
// Rows of more entries than this take 16 loads a lane at a time, shorter ones four.  16 of 64 sequences ended, of 125 / 256 /
// 400 / 1259 pages: 12.9 / 12.9 / 13.9 / 29.0 us with 16 loads, 8.9 / 11.8 / 17.6 / 35.7 with four; 200 of 2000: 16.5 / 16.6 /
// 17.1 / 30.6 and 12.6 / 15.1 / 19.8 / 34.5.
constexpr int kLongRow = 256;
// Most tokens that one cluster takes.  25,000 / 40,000 / 60,000 tokens of 256 sequences: 7.7 / 9.1 / 11.5 us in one, 8.6 / 8.3 /
// 8.7 in two kernels; of 1000: 8.5 / 10.2 / 12.8 and 10.7 / 10.1 / 9.5.
constexpr int kClusterTokens = 40000;

// kRows: positions and slots too; else paged_slots_kernel writes them.
template <int NT, bool kRows>
__global__ void __launch_bounds__(NT) paged_tables_kernel(const PagedTables a) {
  constexpr int kW = NT / 32;
  extern __shared__ int smem[];
  int* cu = smem;                        // [B + 1]: rows before a sequence
  int* taken = cu + a.B + 1;             // [B + 1]: pages taken before it
  int* given = taken + a.B + 1;          // [B]: pages given back before it
  int* past = given + a.B;               // [B]: keys before the step; -1 - keys where the sequence has ended
  __shared__ long long sum_n[kW], sum_g[kW];
  __shared__ int sum_t[kW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_rank(), ctas = cluster_size();
  if constexpr (!kRows) pdl_launch_dependents();
  int bad = 0;
  auto div = [&](int j) { return (int)(((uint64_t)(uint32_t)j * a.page_mul) >> a.page_shift); };
  auto pages_of = [&](int keys) { return div(keys + a.page_size - 1); };
  const int count0 = a.free_count[0];
  const int c0 = min(max(count0, 0), a.num_pages);
  if (count0 > a.num_pages) bad |= kPagedFullList;

  // running sum over the block of x, before this thread's own; total: of all
  auto scan = [&](auto x, auto* sums, auto& total) {
    auto v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const auto u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    // every warp sums the warps' sums for itself
    auto w = lane < kW ? sums[lane] : decltype(x)(0);
#pragma unroll
    for (int o = 1; o < kW; o <<= 1) {
      const auto u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    total = __shfl_sync(0xffffffffu, w, kW - 1);
    const auto upto = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    return (warp ? upto : decltype(x)(0)) + v - x;
  };

  long long rows = 0, back = 0;
  int pages = 0;
  for (int base = 0; base < a.B; base += NT) {
    const int b = base + tid;
    const bool in = b < a.B;
    const int p_in = in ? a.past[b] : 0, n_in = in ? a.fresh[b] : 0;
    const int p = min(max(p_in, 0), a.cap);
    const bool ended = n_in < 0;
    const int have = pages_of(p);
    const int n1 = ended ? 0 : min(n_in, a.cap - p);
    if (p != p_in || (!ended && n1 != n_in)) bad |= kPagedBadLength;
    // pages that this thread's sequence gives back: entries in range, counted by the warp
    int g = 0;
    unsigned who = __ballot_sync(0xffffffffu, ended && have > 0);
    while (who) {
      const int src = __ffs(who) - 1;
      who &= who - 1;
      const int32_t* row = a.table + (int64_t)(base + warp * 32 + src) * a.table_stride;
      const int h = __shfl_sync(0xffffffffu, have, src);
      const int c = h > kLongRow ? count_ids<16>(row, h, a.num_pages, lane) : count_ids<kAhead>(row, h, a.num_pages, lane);
      if (lane == src) {
        g = c;
        if (c != h) bad |= kPagedBadPage;
      }
    }
    long long all_n, all_g = 0;
    const long long e = rows + scan((long long)n1, sum_n, all_n);
    long long eg = 0;
    if (__syncthreads_or(ended)) eg = scan((long long)g, sum_g, all_g);
    const int n = (int)max(0ll, min((long long)n1, a.tokens - e));
    if (n != n1) bad |= kPagedBadLength;
    const int need = ended ? 0 : pages_of(p + n) - have;
    // pages taken: no more than tokens
    int all_t;
    const int before = pages + scan(need, sum_t, all_t);
    if (in) {
      cu[b] = (int)min(e, (long long)a.tokens);
      taken[b] = before;
      given[b] = (int)min(back + eg, 1ll << 30);
      past[b] = ended ? -1 - p : p;
    }
    rows += all_n;
    back += all_g;
    pages += all_t;
    __syncthreads();                     // the sums are used again
  }
  if (tid == 0) {
    cu[a.B] = (int)min(rows, (long long)a.tokens);
    taken[a.B] = pages;
  }
  __syncthreads();
  const int64_t top = min((long long)c0 + back, (long long)a.num_pages);
  if ((int64_t)c0 + back > a.num_pages) bad |= kPagedFullList;

  // ---- pages given back, in the order of sequences and entries: a warp a sequence
  if (back > 0) {
    for (int b = rank * kW + warp; b < a.B; b += ctas * kW) {
      if (past[b] >= 0) continue;
      const int h = pages_of(-1 - past[b]);
      const int32_t* row = a.table + (int64_t)b * a.table_stride;
      const int64_t at = (int64_t)c0 + given[b];
      if (h > kLongRow) give_back<16>(row, h, a.free_pages, at, a.num_pages, lane);
      else give_back<kAhead>(row, h, a.free_pages, at, a.num_pages, lane);
    }
  }
  cluster_sync();

  // the i-th page taken
  auto take = [&](int i) -> int {
    const int64_t at = top - 1 - i;
    if (at < 0) {
      bad |= kPagedNoPages;
      return -1;
    }
    const int id = SDPA_IN_BOUNDS(at < a.num_pages, 561) ? __ldcg(a.free_pages + at) : -1;
    if ((unsigned)id >= (unsigned)a.num_pages) {
      bad |= kPagedBadPage;
      return -1;
    }
    return id;
  };
  const int step = ctas * NT, first = rank * NT + tid;
  for (int i = first; i < pages; i += step) {
    const int b = last_not_above(taken, a.B, i);
    const int pg = pages_of(past[b]) + i - taken[b];
    if (SDPA_IN_BOUNDS(b < a.B && past[b] >= 0 && pg < a.max_pages, 562)) a.table[(int64_t)b * a.table_stride + pg] = take(i);
  }
  if constexpr (kRows) {
    const int live = cu[a.B];
    // four tokens at a time: their table entries or pages are on their way together
    for (int t0 = first; t0 < a.tokens; t0 += step * kAhead) {
      int pos[kAhead], id[kAhead];
      const int32_t* src[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int t = t0 + u * step;
        src[u] = nullptr;
        pos[u] = 0;
        if (t >= live) continue;
        const int b = last_not_above(cu, a.B, t);
        pos[u] = past[b] + t - cu[b];
        const int pg = div(pos[u]), have = pages_of(past[b]);
        const int64_t at = top - 1 - (taken[b] + pg - have);
        if (pg < have) src[u] = a.table + (int64_t)b * a.table_stride + pg;
        else if (at >= 0) src[u] = a.free_pages + at;
        else bad |= kPagedNoPages;
        if (!SDPA_IN_BOUNDS(b < a.B && pg >= 0 && pg < a.max_pages && at < a.num_pages, 563)) src[u] = nullptr;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) id[u] = src[u] ? __ldcg(src[u]) : -1;
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (src[u] && (unsigned)id[u] >= (unsigned)a.num_pages) {
          bad |= kPagedBadPage;
          id[u] = -1;
        }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int t = t0 + u * step;
        if (t >= a.tokens) break;
        a.positions[t] = pos[u];
        a.slots[t] = id[u] < 0 ? -1 : (int64_t)id[u] * a.page_size + (pos[u] - div(pos[u]) * a.page_size);
      }
    }
  }
  for (int b = first; b <= a.B; b += step) {
    a.cu[b] = cu[b];
    if (b < a.B) a.kv_lens[b] = past[b] < 0 ? 0 : past[b] + cu[b + 1] - cu[b];
  }
  if (first == 0) a.free_count_out[0] = (int)(top - pages);
  if (bad) atomicOr(g_tables_status, bad);
}

// Positions and slots of many tokens, from the offsets, lengths and table entries of the first kernel: a
// cluster's threads would take them in many turns (184,000 tokens 26.6 us, 7.7 this way).
constexpr int kSlotThreads = 256, kSlotTokens = 4;      // per thread
__global__ void __launch_bounds__(kSlotThreads) paged_slots_kernel(const PagedTables a) {
  pdl_wait();
  int bad = 0;                           // missing pages are reported by the first kernel
  auto div = [&](int j) { return (int)(((uint64_t)(uint32_t)j * a.page_mul) >> a.page_shift); };
  const int live = a.B > 0 ? a.cu[a.B] : 0;
  const int t0 = (int)blockIdx.x * kSlotThreads * kSlotTokens + (int)threadIdx.x;
  int pos[kSlotTokens], id[kSlotTokens];
  bool begun[kSlotTokens];               // a page of the keys before the step
#pragma unroll
  for (int u = 0; u < kSlotTokens; ++u) {
    const int t = t0 + u * kSlotThreads;
    pos[u] = 0;
    id[u] = -1;
    begun[u] = false;
    if (t >= live) continue;
    const int b = last_not_above(a.cu, a.B, t);
    const int past = a.kv_lens[b] - a.cu[b + 1] + a.cu[b];
    pos[u] = past + t - a.cu[b];
    const int pg = div(pos[u]);
    begun[u] = pg < div(past + a.page_size - 1);
    if (SDPA_IN_BOUNDS(b < a.B && pg >= 0 && pg < a.max_pages, 564)) id[u] = a.table[(int64_t)b * a.table_stride + pg];
  }
#pragma unroll
  for (int u = 0; u < kSlotTokens; ++u) {
    const int t = t0 + u * kSlotThreads;
    if (t >= a.tokens) break;
    const bool ok = (unsigned)id[u] < (unsigned)a.num_pages;
    if (!ok && begun[u]) bad |= kPagedBadPage;
    a.positions[t] = pos[u];
    a.slots[t] = ok ? (int64_t)id[u] * a.page_size + (pos[u] - div(pos[u]) * a.page_size) : -1;
  }
  if (bad) atomicOr(g_tables_status, bad);
}

template <int NT, bool kRows>
cudaError_t launch_nt(const PagedTables& a, int ctas, cudaStream_t st) {
  const size_t smem = ((size_t)4 * a.B + 2) * sizeof(int);
  auto* kernel = paged_tables_kernel<NT, kRows>;
  // per device: set at every call that needs it (the attribute belongs to the current context)
  if (smem > 48 * 1024 - 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return e;
  count_launch(1);
  if (kRows) return cudaSuccess;
  const int per = kSlotThreads * kSlotTokens;
  cfg.gridDim = dim3((unsigned)((a.tokens + per - 1) / per));
  cfg.blockDim = dim3(kSlotThreads);
  cfg.dynamicSmemBytes = 0;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  e = cudaLaunchKernelEx(&cfg, paged_slots_kernel, a);
  if (e == cudaSuccess) count_launch(1);
  return e;
}

}  // namespace

// One CTA for few tokens.  256 sequences, 256 / 1024 / 2048 / 4096 tokens: 3.7 / 5.2 / 7.5 / 13.5 us with 256 threads, 4.4 / 4.8 /
// 5.5 / 7.9 with 1024, 4.4 / 4.8 / 4.7 / 5.4 with eight CTAs.
cudaError_t launch_paged_tables(const PagedTables& a, cudaStream_t st) {
  if (a.B <= 256 && a.tokens <= 1024) return launch_nt<256, true>(a, 1, st);
  if (a.tokens <= kClusterTokens) return launch_nt<1024, true>(a, a.tokens <= 4096 ? 1 : 8, st);
  return launch_nt<1024, false>(a, 8, st);
}

cudaError_t take_paged_tables_status(int* status) { return take_words(g_tables_status, status); }

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_paged_tables)

}  // namespace sdpa
