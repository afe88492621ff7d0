// How the attention over a paged cache is cut up, shared by its three kernels.
//
// A unit is TM consecutive packed rows (row r = token * group + head of the group) of one
// (sequence, kv head); its cost is the number of TN-key tiles that some of its rows admits (at
// least one, so that rows with no key are written too) and OV more for its query rows and its
// results, in tiles' time.  All units, laid end to end (sequence, row block, kv head, tile), are
// dealt to the CTAs in equal contiguous shares of that cost (in units of 256 rows, a tile of more
// than 128 rows counts 4, one of fewer 3, and OV is in these), so ragged lengths, few rows over many
// keys and many rows over few keys all fill the GPU alike, and a CTA meets at most two units that
// it does not hold whole.  (4 chunks beside 24 single tokens: 81 us with tiles at 4 and 3, 88 at 4 and
// 4, 103 at 4 and 2; without a window 255, 280 and 283.  Without OV, the CTA that gets the first, shortest row blocks of a
// causal prompt had 40 units of one or two tiles and took twice as long as the others.)  Those leave partial results
// (m, l, unnormalised o) in two slots per CTA, which a second kernel joins.  The lengths stay on
// the device: every CTA finds its share by summing the costs of all sequences.
#pragma once

#include "paged.h"
#include "tc_ptx.cuh"

namespace sdpa {

// Where a CTA's share starts; tile > 0: inside a unit begun by an earlier CTA.
struct ShareStart { int b, rb, kvh, tile; };

struct PagedWs {
  ShareStart* start;   // [ctas + 1]: the last entry counts the CTAs that have a share (in .b)
  float* ml;           // [2 * ctas][TM][2]: running maximum (log2 units) and sum
  float* o;            // [2 * ctas][TM][Hv]
};
__host__ __device__ inline size_t paged_ws_ml_off(int ctas) {
  return (((size_t)ctas + 1) * sizeof(ShareStart) + 255) & ~(size_t)255;
}
__host__ __device__ inline size_t paged_ws_o_off(int ctas, int tm) {
  return paged_ws_ml_off(ctas) + (((size_t)2 * ctas * tm * 2 * sizeof(float) + 255) & ~(size_t)255);
}
inline size_t paged_ws_bytes(int ctas, int tm, int Hv) {
  return paged_ws_o_off(ctas, tm) + (((size_t)2 * ctas * tm * Hv * sizeof(float) + 255) & ~(size_t)255);
}
inline PagedWs paged_ws(void* p, int ctas, int tm) {
  char* c = reinterpret_cast<char*>(p);
  return PagedWs{reinterpret_cast<ShareStart*>(c), reinterpret_cast<float*>(c + paged_ws_ml_off(ctas)),
                 reinterpret_cast<float*>(c + paged_ws_o_off(ctas, tm))};
}

// CTAs per SM x most SMs a workspace is sized for.
constexpr int kPagedMaxSms = 160;

cudaError_t launch_paged_merge(const PagedAttn& a, sdpa_dtype dt, const PagedWs& ws, int ctas, int tm, cudaStream_t st);
int paged_sms();
// Tensor map over a page pool for boxes of box_rows slots.
bool paged_map(CUtensorMap* map, const Paged& g, const View& v, int D, sdpa_dtype dt, int box_rows, int* ds, int* dn, int* db);
// Fast division: the multiplier and shift of j / d for 0 <= j < 2^31.
inline void paged_magic(int d, uint32_t* mul, uint32_t* shift) {
  int l = 0;
  while (((int64_t)1 << l) < d) ++l;
  *shift = 31 + l;
  *mul = (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d);
}

#ifdef __CUDACC__
// One row block of a sequence: rows, the keys some row admits, its tiles.
struct RowBlock {
  int row0, rows;      // packed rows of the sequence
  int lo, hi;          // admitted keys [lo, hi] (hi < lo: none)
  int tile0, tiles;    // first key tile, tiles (>= 1)
  int weight;          // cost of a tile
};
template <int TM, int TN>
__device__ __forceinline__ RowBlock row_block(const PagedAttn& a, const SeqInfo& s, int rb) {
  RowBlock r;
  const int all = s.n * a.g.group;
  r.row0 = rb * TM;
  r.rows = min(TM, all - r.row0);
  const int i0 = group_div(a.g, r.row0), i1 = group_div(a.g, r.row0 + r.rows - 1);
  r.hi = a.causal ? s.T - s.n + i1 : s.T - 1;
  r.lo = a.window > 0 ? max(0, s.T - s.n + i0 - a.window + 1) : 0;
  r.tile0 = r.lo / TN;
  r.tiles = r.hi >= r.lo ? r.hi / TN - r.tile0 + 1 : 1;
  r.weight = TM > 128 ? (r.rows > 128 ? 4 : 3) : 1;
  return r;
}
__device__ __forceinline__ int row_blocks(const PagedAttn& a, const SeqInfo& s, int TM) {
  return (s.n * a.g.group + TM - 1) / TM;
}

// Admitted keys [lo, hi] of packed row r of a sequence (hi < lo: none).
__device__ __forceinline__ void row_keys(const PagedAttn& a, const SeqInfo& s, int r, int& lo, int& hi) {
  const int pos = s.T - s.n + group_div(a.g, r);
  hi = a.causal ? pos : s.T - 1;
  lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
}

__device__ __forceinline__ int unit_cost(const RowBlock& r, int OV) { return r.tiles * r.weight + OV; }

struct Share {
  int64_t count;           // the CTA's part of the whole cost
  int pos;                 // where it starts in its first unit's cost
  ShareStart at;
  SeqInfo s;               // of sequence at.b
  int active;              // CTAs that have a share
};

// Finds the share of CTA `cta` among `ctas`; called by all NT threads of the block.  min_share:
// least cost worth a CTA.
template <int TM, int TN, int OV, int NT>
__device__ __forceinline__ Share find_share(const PagedAttn& a, int cta, int ctas, int min_share, int* status) {
  constexpr int kW = NT / 32, kChunks = 32;
  __shared__ long long sh_sum[kW + 1];
  __shared__ long long sh_chunk[kChunks];      // costs of NT sequences each, the last of all that follow
  __shared__ ShareStart sh_at;
  __shared__ SeqInfo sh_s;
  __shared__ int sh_pos;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;

  auto info_of = [&](int b) { return b < a.g.B ? seq_info(a.g, b, bad) : SeqInfo{0, 0, 0}; };
  // cost of this thread's sequence; sequences of several row blocks are summed by the warp
  auto cost_of = [&](const SeqInfo& s) -> long long {
    long long c = 0;
    const int nrb = row_blocks(a, s, TM);
    if (nrb == 1) c = unit_cost(row_block<TM, TN>(a, s, 0), OV);
    unsigned many = __ballot_sync(0xffffffffu, nrb > 1);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      SeqInfo t;
      t.t0 = 0;
      t.n = __shfl_sync(0xffffffffu, s.n, src);
      t.T = __shfl_sync(0xffffffffu, s.T, src);
      const int n = row_blocks(a, t, TM);
      long long part = 0;
      for (int rb = lane; rb < n; rb += 32) part += unit_cost(row_block<TM, TN>(a, t, rb), OV);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if (lane == src) c = part;
    }
    return c * a.g.Nkv;
  };

  // running sum of x over the warp; the warps' sums go to sh_sum
  auto scan = [&](long long x) -> long long {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += u;
    }
    if (lane == 31) sh_sum[warp] = x;
    return x;
  };

  const bool one = a.g.B <= NT;      // a sequence per thread: one pass, whose running sums also find the share
  const int chunks = min(kChunks, (a.g.B + NT - 1) / NT);
  long long mine = 0, v = 0, total = 0;
  SeqInfo s = info_of(threadIdx.x);
  if (one) {
    mine = cost_of(s);
    v = scan(mine);
    __syncthreads();
    for (int i = 0; i < kW; ++i) total += sh_sum[i];
  } else {
    if (threadIdx.x < kChunks) sh_chunk[threadIdx.x] = 0;
    __syncthreads();
    for (int base = 0, chunk = 0; base < a.g.B; base += NT, ++chunk) {
      const SeqInfo next = base + NT < a.g.B ? info_of(base + NT + (int)threadIdx.x) : SeqInfo{0, 0, 0};
      long long c = cost_of(s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
      // integers: the order of the additions does not matter
      auto* sum = reinterpret_cast<unsigned long long*>(&sh_chunk[min(chunk, kChunks - 1)]);
      if (lane == 0 && c) atomicAdd(sum, (unsigned long long)c);
      if (base + NT < a.g.B) s = next;
    }
    __syncthreads();
    for (int c = 0; c < chunks; ++c) total += sh_chunk[c];
  }
  if (bad && cta == 0) atomicOr(status, kPagedBadLength);

  Share r;
  r.active = total >= (long long)ctas * min_share ? ctas : max(1, (int)total / min_share);
  if (total == 0) r.active = 0;
  r.at = ShareStart{a.g.B, 0, 0, 0};
  r.s = SeqInfo{0, 0, 0};
  r.count = 0;
  r.pos = 0;
  if (cta >= r.active) return r;
  // total / active tiles each, the first total % active CTAs one more (32-bit divisions where
  // they do: a 64-bit one takes a microsecond's fraction that short calls feel)
  long long each, more;
  if (total < (1ll << 32)) {
    each = (unsigned)total / (unsigned)r.active;
    more = (unsigned)total - (unsigned)each * (unsigned)r.active;
  } else {
    each = total / r.active;
    more = total - each * r.active;
  }
  const long long begin_at = cta * each + min((long long)cta, more);
  r.count = each + (cta < more ? 1 : 0);

  // the sequence that holds begin_at, from its chunk on
  long long before = 0;
  int from = 0;
  while (from + 1 < chunks && before + sh_chunk[from] <= begin_at) before += sh_chunk[from++];
  for (int base = from * NT; base < a.g.B; base += NT) {
    if (!one) {
      s = info_of(base + (int)threadIdx.x);
      mine = cost_of(s);
      v = scan(mine);
      __syncthreads();
    }
    long long off = before, all = 0;
#pragma unroll 1
    for (int w = 0; w < kW; ++w) {
      if (w < warp) off += sh_sum[w];
      all += sh_sum[w];
    }
    const long long end = off + v, begin = end - mine;
    // exactly one warp holds it; its lanes find the row block
    const bool here = begin_at >= begin && begin_at < end;
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
      const int src = __ffs(who) - 1;
      SeqInfo t;
      t.t0 = __shfl_sync(0xffffffffu, s.t0, src);
      t.n = __shfl_sync(0xffffffffu, s.n, src);
      t.T = __shfl_sync(0xffffffffu, s.T, src);
      const int n = row_blocks(a, t, TM);
      long long o = begin_at - __shfl_sync(0xffffffffu, begin, src);
      for (int rb0 = 0; rb0 < n; rb0 += 32) {
        const RowBlock block = row_block<TM, TN>(a, t, min(rb0 + lane, n - 1));
        const int cost = rb0 + lane < n ? unit_cost(block, OV) : 0;
        long long c = (long long)cost * a.g.Nkv;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long u = __shfl_up_sync(0xffffffffu, c, d);
          if (lane >= d) c += u;
        }
        const long long lo = c - (long long)cost * a.g.Nkv;
        if (o >= lo && o < c) {
          // within one row block: fewer than Nkv * cost, which fits 32 bits with room
          const unsigned in = (unsigned)(o - lo), k = in / (unsigned)cost;
          const int off = (int)(in - k * (unsigned)cost);
          sh_at = ShareStart{base + warp * 32 + src, rb0 + lane, (int)k, max(0, off - OV) / block.weight};
          sh_pos = off;
          sh_s = t;
        }
        const long long sum = __shfl_sync(0xffffffffu, c, 31);
        if (o < sum) break;
        o -= sum;
      }
    }
    __syncthreads();
    before += all;
    if (before > begin_at) break;
  }
  r.at = sh_at;
  r.s = sh_s;
  r.pos = sh_pos;
  return r;
}

// Walks a share unit by unit.  The CTA takes the tiles [tile, tile + take()) of the present unit: those
// whose cost, behind the unit's OV, ends in the share.  (A share of at least two tiles' weight that
// starts inside a unit has a tile of it; one that ends in a unit's OV leaves it to the next CTA.)
template <int TM, int TN, int OV>
struct Walk {
  int64_t left;            // cost left, from pos on
  int pos;                 // of the present unit's cost
  int b, rb, kvh, tile, upto;
  SeqInfo s;
  RowBlock r;
  __device__ __forceinline__ Walk(const PagedAttn& a, const Share& sh)
      : left(sh.count), pos(sh.pos), b(sh.at.b), rb(sh.at.rb), kvh(sh.at.kvh), tile(sh.at.tile), upto(0), s(sh.s) {
    if (left > 0) {
      r = row_block<TM, TN>(a, s, rb);
      bound();
    }
  }
  __device__ __forceinline__ void bound() {
    upto = (int)min((int64_t)r.tiles, max((int64_t)0, pos + left - OV) / r.weight);
    if (upto <= tile) left = 0;
  }
  __device__ __forceinline__ bool done() const { return left <= 0; }
  __device__ __forceinline__ int take() const { return upto - tile; }
  __device__ __forceinline__ bool begins() const { return tile == 0; }
  __device__ __forceinline__ bool whole() const { return tile == 0 && upto == r.tiles; }
  __device__ __forceinline__ void next(const PagedAttn& a) {
    left -= unit_cost(r, OV) - pos;
    pos = tile = 0;
    if (left <= 0) return;
    if (++kvh == a.g.Nkv) {
      kvh = 0;
      if (++rb >= row_blocks(a, s, TM)) {
        rb = 0;
        bool bad = false;
        while (++b < a.g.B) {
          s = seq_info(a.g, b, bad);
          if (s.n > 0) break;
        }
        if (b >= a.g.B) { left = 0; return; }
      }
      r = row_block<TM, TN>(a, s, rb);
    }
    bound();
  }
};

// Whether a row, or a part of one, has no weight so far: no admitted key.  Scores that are not
// numbers leave the maximum at -inf too (a maximum drops them), but not the sum.
__device__ __forceinline__ bool no_key(float m, float l) { return m == -INFINITY && l == 0.f; }

// Final scale of row (head h): 1 / (l + sink term), 0 for a row with no key; m, l in log2 units.
template <typename T>
__device__ __forceinline__ float row_scale(const PagedAttn& a, int h, float m, float l) {
  if (no_key(m, l)) return 0.f;
  if (a.head_sink) l += exp2f(Elem<T>::to_f32(reinterpret_cast<const T*>(a.head_sink)[h]) * kLog2e - m);
  return 1.f / l;                        // about 1 or more where m is finite; NaN, also of a sink, stays NaN
}

// Lets the joining kernel be scheduled; it waits for this one's results itself.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

}  // namespace sdpa
