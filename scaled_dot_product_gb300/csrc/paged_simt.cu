// Attention over a paged cache in fp32 arithmetic, for every type and head size, and the kernel
// that joins the partial results of all three attention kernels.
//
// LPK lanes read one key or value row as 16-byte vectors; the 128 / LPK lane groups of a block
// take different keys and keep their own running maximum, sum and accumulator of TM query rows,
// joined in shared memory at the end of a unit.  Bound by latency: eight float32 sequences of 500 to 4000
// keys, 16/4 heads of 64, take 20 to 21 us (38.8 MB); 30.5 us with 64 full reductions a step instead of 15
// exchanges and one thread an item of the join, 34.6 with four CTAs an SM.  It serves fp32 (whose sums the 16-bit tensor
// products cannot carry) and head sizes that the tensor-core kernels do not tile, for single tokens and a
// few: 16 sequences of 2000 to 16000 keys, 32/8 heads, float32 of 128 334 us (4.5 TB/s), bfloat16 of 96 428 us
// (1.3 TB/s), of 256 830 us (1.8 TB/s).  Chunks read their keys again for every four rows: 200 tokens
// over 4000 keys, 16/4 float32 heads of 64, 296 us; 512 over 4000, 32/8 heads of 96, 2.96 ms (9 TFLOP/s).
#include <algorithm>

#include "paged_sched.cuh"

namespace sdpa {

static __device__ int g_paged_status[1];

namespace {

constexpr int kThreads = 128;
constexpr int kTN = 64;          // keys per tile of the schedule

constexpr int log2i(int x) { return x <= 1 ? 0 : 1 + log2i(x / 2); }
constexpr int kCtasPerSm = 3;
constexpr int kOV = 1;                // a unit's cost beside its tiles, in tiles
constexpr int kMinShare = 2;

template <typename T, int LPK, int NV, int TM>
__global__ void __launch_bounds__(kThreads, NV == 1 ? kCtasPerSm : 2) paged_simt_kernel(const PagedAttn a, const PagedWs ws) {
  constexpr int V = Elem<T>::kVec;
  constexpr int KPI = kThreads / LPK;
  constexpr int HM = LPK * NV * V;       // widest head
  constexpr int kUnroll = NV == 1 ? 4 : 2;
  extern __shared__ float smem[];        // [KPI][TM][HM]
  __shared__ float sm_m[KPI][TM], sm_l[KPI][TM];
  const Paged& g = a.g;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const Share sh = find_share<TM, kTN, kOV, kThreads>(a, cta, ctas, kMinShare, g_paged_status);
  if (threadIdx.x == 0) {
    if (cta == 0) ws.start[ctas].b = sh.active;
    if (cta < sh.active) ws.start[cta] = sh.at;
  }
  pdl_launch_dependents();
  const int grp = threadIdx.x / LPK, t = threadIdx.x % LPK;
  const float cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  // Scores of a step: score r * kUnroll + u of row r and key u.  After SC exchanges a lane holds the sums
  // of R of them, of one row, from key my_u on; UB exchanges span the lanes of a row.
  constexpr int NS = TM * kUnroll, SC = log2i(NS) < log2i(LPK) ? log2i(NS) : log2i(LPK), R = NS >> SC;
  constexpr int UB = log2i(kUnroll) - log2i(R);
  static_assert(R <= kUnroll, "a lane's scores belong to one row");
  const int first = (t >> (log2i(LPK) - SC)) << (log2i(NS) - SC);
  const int my_row = first / kUnroll, my_u = first % kUnroll;
  auto lane_of = [](int score) { return (score >> (log2i(NS) - SC)) << (log2i(LPK) - SC); };

  for (Walk<TM, kTN, kOV> w(a, sh); !w.done(); w.next(a)) {
    const int nr = w.r.rows;
    float q[TM][NV * V], acc[TM][NV * V];
#pragma unroll
    for (int r = 0; r < TM; ++r) {
      const int pr = w.r.row0 + min(r, nr - 1);
      const T* row = reinterpret_cast<const T*>(a.q.p) +
                     a.q.off(0, w.kvh * g.group + pr - group_div(g, pr) * g.group, w.s.t0 + group_div(g, pr));
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int c = (n * LPK + t) * V;
        const uint4 u = c < g.H ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
        unpack16<T>(u, q[r] + n * V);
      }
#pragma unroll
      for (int e = 0; e < NV * V; ++e) acc[r][e] = 0.f;
    }
    // this lane's row of the scores: its keys, running maximum and part of the sum
    int lo, hi;
    row_keys(a, w.s, w.r.row0 + min(my_row, nr - 1), lo, hi);
    float m = -INFINITY, l = 0.f;
    const int64_t j_tile = (int64_t)(w.r.tile0 + w.tile) * kTN;
    const int64_t j_begin = max(j_tile, (int64_t)w.r.lo);      // pages below a window are not read
    const int64_t j_end = min((int64_t)w.r.hi + 1, j_tile + (int64_t)w.take() * kTN);
    const int32_t* table = g.table + (int64_t)w.b * g.table_stride;

    // keys of one step: those at base + grp + u * KPI.  Their rows are loaded one step ahead, the ids of
    // their pages two.
    constexpr int kStep = KPI * kUnroll;
    auto load_ids = [&](int64_t base, int* id) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t j = base + grp + u * KPI;
        id[u] = j < j_end ? table[page_div(g, (int)j)] : -1;
      }
    };
    auto load_rows = [&](int64_t base, const int* id, uint4 (&kv)[kUnroll][NV], uint4 (&vv)[kUnroll][NV]) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t j = base + grp + u * KPI;
        const int key = (int)min(j, (int64_t)g.cap), slot = key - page_div(g, key) * g.page_size;
        bool take = j < j_end;
        if (take && (unsigned)id[u] >= (unsigned)g.num_pages) {
          atomicOr(g_paged_status, kPagedBadPage);
          take = false;                    // read as zeros
        }
        take = take && SDPA_IN_BOUNDS(key < g.cap && slot < g.page_size, 521);
        const T* kr = reinterpret_cast<const T*>(g.kp.p) + g.kp.off(id[u], w.kvh, slot);
        const T* vr = reinterpret_cast<const T*>(g.vp.p) + g.vp.off(id[u], w.kvh, slot);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int c = (n * LPK + t) * V;
          kv[u][n] = take && c < g.H ? __ldg(reinterpret_cast<const uint4*>(kr + c)) : make_uint4(0u, 0u, 0u, 0u);
          vv[u][n] = take && c < g.Hv ? __ldg(reinterpret_cast<const uint4*>(vr + c)) : make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    int id[kUnroll];
    load_ids(j_begin, id);
#pragma unroll 1
    for (int64_t base = j_begin; base < j_end; base += kStep) {
      uint4 kv[kUnroll][NV], vv[kUnroll][NV];
      load_rows(base, id, kv, vv);
      load_ids(base + kStep, id);
      // every lane's part of the step's TM x kUnroll scores, then their sums dealt to the lanes: at each
      // exchange a lane keeps the half of the scores that its lane bit names
      float s[NS];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float kf[NV * V];
#pragma unroll
        for (int n = 0; n < NV; ++n) unpack16<T>(kv[u][n], kf + n * V);
#pragma unroll
        for (int r = 0; r < TM; ++r) {
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < NV * V; ++e) dot = fmaf(q[r][e], kf[e], dot);
          s[r * kUnroll + u] = dot;
        }
      }
#pragma unroll
      for (int k = 0; k < SC; ++k) {
        const int o = LPK >> (k + 1), half = NS >> (k + 1);
        const bool up = t & o;
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const float give = up ? s[i] : s[i + half];
          s[i] = (up ? s[i + half] : s[i]) + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
#pragma unroll
      for (int o = LPK >> (SC + 1); o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int64_t j = base + grp + (my_u + i) * KPI;
        float v = a.softcap > 0.f ? a.softcap * tanhf(s[i] * cap_in) : s[i] * a.scale;
        v = (j < j_end && j >= lo && j <= hi) ? v * kLog2e : -INFINITY;
        s[i] = v;
        mx = fmaxf(mx, v);
      }
#pragma unroll
      for (int o = 0; o < UB; ++o) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1 << (log2i(LPK) - SC + o)));
      float corr = 1.f;
      const bool need = mx > m;
      if (need) {
        corr = exp2f(m - mx);
        m = mx;
        l *= corr;
      }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int r = 0; r < TM; ++r) {
          const float c = __shfl_sync(0xffffffffu, corr, lane_of(r * kUnroll), LPK);
#pragma unroll
          for (int e = 0; e < NV * V; ++e) acc[r][e] *= c;
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        s[i] = s[i] == -INFINITY ? 0.f : exp2f(s[i] - m);
        l += s[i];
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float vf[NV * V];
#pragma unroll
        for (int n = 0; n < NV; ++n) unpack16<T>(vv[u][n], vf + n * V);
#pragma unroll
        for (int r = 0; r < TM; ++r) {
          const float p = __shfl_sync(0xffffffffu, s[(r * kUnroll + u) & (R - 1)], lane_of(r * kUnroll + u), LPK);
#pragma unroll
          for (int e = 0; e < NV * V; ++e) acc[r][e] = fmaf(p, vf[e], acc[r][e]);
        }
      }
    }
#pragma unroll
    for (int o = 0; o < UB; ++o) l += __shfl_xor_sync(0xffffffffu, l, 1 << (log2i(LPK) - SC + o));

    // join the lane groups
    __syncthreads();
    if (t == lane_of(my_row * kUnroll)) {
      sm_m[grp][my_row] = m;
      sm_l[grp][my_row] = l;
    }
#pragma unroll
    for (int r = 0; r < TM; ++r) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < V; ++e) smem[(grp * TM + r) * HM + (n * LPK + t) * V + e] = acc[r][n * V + e];
    }
    __syncthreads();
    const bool whole = w.whole();
    const int64_t slot = 2 * (int64_t)cta + (w.begins() ? 1 : 0);
    for (int x = threadIdx.x; x < nr * g.Hv; x += kThreads) {
      const int r = x / g.Hv, d = x - r * g.Hv;
      float M = -INFINITY;
      for (int k = 0; k < KPI; ++k) M = fmaxf(M, sm_m[k][r]);
      float O = 0.f, L = 0.f;
      for (int k = 0; k < KPI; ++k) {
        if (no_key(sm_m[k][r], sm_l[k][r])) continue;
        const float f = exp2f(sm_m[k][r] - M);
        O = fmaf(f, smem[(k * TM + r) * HM + d], O);
        L = fmaf(f, sm_l[k][r], L);
      }
      if (whole) {
        const int pr = w.r.row0 + r, h = w.kvh * g.group + pr - group_div(g, pr) * g.group;
        T* y = reinterpret_cast<T*>(const_cast<void*>(a.y.p)) + a.y.off(0, h, w.s.t0 + group_div(g, pr));
        if (SDPA_IN_BOUNDS(w.s.t0 + group_div(g, pr) < g.tokens && h < g.Nq, 522))
          y[d] = Elem<T>::from_f32(O * row_scale<T>(a, h, M, L));
      } else if (SDPA_IN_BOUNDS(slot < 2 * ctas, 523)) {
        ws.o[(slot * TM + r) * g.Hv + d] = O;
        if (d == 0) {
          ws.ml[(slot * TM + r) * 2] = M;
          ws.ml[(slot * TM + r) * 2 + 1] = L;
        }
      }
    }
  }
}

// ---------------------------------------------------------------- joining the partial results

constexpr int kMergeThreads = 256;

// How a joined unit is cut: a block takes `rows` rows (a power of two up to 32) and `cols` groups of four
// columns; with fewer than 256 of these items, 256 / (rows * cols) threads share one, each taking
// a part of the partial results.
struct MergeCut { int rows, cols; };

// The blocks (c, .) join the unit that CTA c's share starts inside of, if c is the first such CTA of
// the unit.  The partials are those of CTA c - 1 (which began the unit) and of the CTAs from c on
// whose shares start inside it, taken in that order.  Bound by latency: a chain of five dependent
// loads, so rows and columns are spread over threads rather than taken in turn (a warp per row,
// eight rows in turn, took 25 us where two partials of every unit of 256 rows were joined).
template <typename T, int TM, int TN>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedAttn a, const PagedWs ws, const int ctas,
                                                                    const MergeCut cut) {
  __shared__ float sm_m[32], sm_inv[32];
  __shared__ long long sm_y[32];
  __shared__ float4 part[kMergeThreads];
  pdl_wait();
  const Paged& g = a.g;
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31;
  // one look at the starts of CTAs c - 1 .. c + 30 (and of c - 1 alone: entries behind the active ones
  // are not used)
  const int active = ws.start[ctas].b;
  const ShareStart mine = ws.start[min(c - 1 + lane, ctas - 1)];
  if (c >= active) return;
  ShareStart at;
  at.b = __shfl_sync(0xffffffffu, mine.b, 1);
  at.rb = __shfl_sync(0xffffffffu, mine.rb, 1);
  at.kvh = __shfl_sync(0xffffffffu, mine.kvh, 1);
  at.tile = __shfl_sync(0xffffffffu, mine.tile, 1);
  if (at.tile == 0) return;
  auto inside = [&](const ShareStart& s) { return s.tile > 0 && s.b == at.b && s.rb == at.rb && s.kvh == at.kvh; };
  unsigned in = __ballot_sync(0xffffffffu, c - 1 + lane < active && inside(mine));
  if (in & 1u) return;                         // an earlier CTA joins this unit
  int n = 1 + __ffs(~(in >> 1)) - 1;           // partials: CTA c - 1's second slot, then first slots
  for (int k = c + 31; n == 32 + (k - c - 31);) {
    in = __ballot_sync(0xffffffffu, k + lane < active && inside(ws.start[min(k + lane, active - 1)]));
    const int more = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
    n += more;
    k += 32;
    if (more < 32) break;
  }
  bool bad = false;
  const SeqInfo s = seq_info(g, at.b, bad);
  const int cols_all = g.Hv / 4;
  const int row0 = (int)blockIdx.y * cut.rows, col0 = (int)blockIdx.z * cut.cols;
  auto slot_of = [&](int i) -> int64_t { return (i == 0 ? 2 * (int64_t)(c - 1) + 1 : 2 * (int64_t)(c + i - 1)) * TM; };

  const int items = cut.rows * cut.cols, share = max(1, kMergeThreads / items);      // threads of one item
  if (n <= 4) {
    // Few partials: a thread reads all of an item's at once, beside the lengths, and finds the row's
    // maximum and sum by itself.  (Every slot of a joined unit holds TM rows; those past the unit's
    // rows are not used.)
    for (int x = threadIdx.x; x < items; x += kMergeThreads) {
      const int r = row0 + x / cut.cols, d = (col0 + x % cut.cols) * 4;
      if (r >= TM || d >= cols_all * 4) continue;
      float2 ml[4];
      float4 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) {
          ml[i] = *reinterpret_cast<const float2*>(ws.ml + (slot_of(i) + r) * 2);
          o[i] = *reinterpret_cast<const float4*>(ws.o + (slot_of(i) + r) * g.Hv + d);
        } else {
          ml[i] = make_float2(-INFINITY, 0.f);
          o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      const RowBlock rbk = row_block<TM, TN>(a, s, at.rb);
      if (r >= rbk.rows) continue;
      const int pr = rbk.row0 + r, tok = s.t0 + group_div(g, pr), h = at.kvh * g.group + pr - group_div(g, pr) * g.group;
      const float M = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
      float L = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (no_key(ml[i].x, ml[i].y)) continue;
        const float f = exp2f(ml[i].x - M);
        L = fmaf(f, ml[i].y, L);
        v.x = fmaf(f, o[i].x, v.x);
        v.y = fmaf(f, o[i].y, v.y);
        v.z = fmaf(f, o[i].z, v.z);
        v.w = fmaf(f, o[i].w, v.w);
      }
      const float inv = row_scale<T>(a, h, M, L);
      T out[4] = {Elem<T>::from_f32(v.x * inv), Elem<T>::from_f32(v.y * inv), Elem<T>::from_f32(v.z * inv),
                  Elem<T>::from_f32(v.w * inv)};
      T* y = reinterpret_cast<T*>(const_cast<void*>(a.y.p)) + a.y.off(0, h, tok) + d;
      if (!SDPA_IN_BOUNDS(tok < g.tokens && h < g.Nq, 525)) continue;
      if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(out);
      else *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(out);
    }
    return;
  }
  const RowBlock rbk = row_block<TM, TN>(a, s, at.rb);
  if (row0 >= rbk.rows) return;

  // maximum and sum of each row, 256 / rows threads (8, 16 or 32 at most) a row
  {
    const int tpr = min(32, kMergeThreads / cut.rows), r = threadIdx.x / tpr, sub = threadIdx.x % tpr;
    const bool live = r < cut.rows && row0 + r < rbk.rows;
    float M = -INFINITY, L = 0.f;
    for (int i = sub; i < n && live; i += tpr) {
      const float2 v = *reinterpret_cast<const float2*>(ws.ml + (slot_of(i) + row0 + r) * 2);
      const float mn = fmaxf(M, v.x);
      L = mn == -INFINITY ? L + v.y : L * exp2f(M - mn) + v.y * exp2f(v.x - mn);
      M = mn;
    }
    for (int o = tpr / 2; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, M, o), l2 = __shfl_xor_sync(0xffffffffu, L, o);
      const float mn = fmaxf(M, m2);
      L = mn == -INFINITY ? L + l2 : L * exp2f(M - mn) + l2 * exp2f(m2 - mn);
      M = mn;
    }
    if (sub == 0 && live) {
      const int pr = rbk.row0 + row0 + r, h = at.kvh * g.group + pr - group_div(g, pr) * g.group;
      sm_m[r] = M;
      sm_inv[r] = row_scale<T>(a, h, M, L);
      sm_y[r] = a.y.off(0, h, s.t0 + group_div(g, pr));
    }
  }
  __syncthreads();

  const int per = kMergeThreads / share, g0 = threadIdx.x / per;
  // the sum of item x over partials g0, g0 + share, ...
  auto sum_of = [&](int x) {
    const int r = x / cut.cols, d = (col0 + x % cut.cols) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + r >= rbk.rows || d >= cols_all * 4) return v;
    const float M = sm_m[r];
#pragma unroll 4
    for (int i = g0; i < n; i += share) {
      const int64_t at_row = slot_of(i) + row0 + r;
      const float2 ml = *reinterpret_cast<const float2*>(ws.ml + at_row * 2);
      const float4 o = *reinterpret_cast<const float4*>(ws.o + at_row * g.Hv + d);
      if (no_key(ml.x, ml.y)) continue;
      const float f = exp2f(ml.x - M);
      v.x = fmaf(f, o.x, v.x);
      v.y = fmaf(f, o.y, v.y);
      v.z = fmaf(f, o.z, v.z);
      v.w = fmaf(f, o.w, v.w);
    }
    return v;
  };
  auto store = [&](int x, const float4& v) {
    const int r = x / cut.cols, d = (col0 + x % cut.cols) * 4;
    if (row0 + r >= rbk.rows || d >= cols_all * 4) return;
    if (!SDPA_IN_BOUNDS(s.t0 + group_div(g, rbk.row0 + row0 + r) < g.tokens, 524)) return;
    const float inv = sm_inv[r];
    T out[4] = {Elem<T>::from_f32(v.x * inv), Elem<T>::from_f32(v.y * inv), Elem<T>::from_f32(v.z * inv),
                Elem<T>::from_f32(v.w * inv)};
    T* y = reinterpret_cast<T*>(const_cast<void*>(a.y.p)) + sm_y[r] + d;
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(out);
    else *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(out);
  };
  if (share == 1) {
    for (int x = threadIdx.x; x < items; x += kMergeThreads) store(x, sum_of(x));
    return;
  }
  const int x = threadIdx.x % per;               // fewer items than threads: one each, every thread at the barrier
  if (x < items) part[threadIdx.x] = sum_of(x);
  __syncthreads();
  if (g0 > 0 || x >= items) return;
  float4 v = part[x];
  for (int k = 1; k < share; ++k) {
    const float4 w = part[x + k * per];
    v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
  }
  store(x, v);
}

template <typename T, int TM, int TN>
cudaError_t merge_tn(const PagedAttn& a, const PagedWs& ws, int ctas, cudaStream_t st) {
  // Few units are cut into many partials each (16 and more): then 8 rows and 32 columns a block, four threads an
  // item.  Otherwise whole rows, at most 16 (or 32 of a 256-row unit) a block.  Both sides, 16000 keys a
  // sequence, units of 16 / 32 / 64 rows (304 CTAs): 1 unit 29 / 29 / 49 us in whole rows, 15 / 15 / 24 cut; 8
  // units 25 / 26 / 49 and 19 / 20 / 38; 16 units 35 / 26 / 56 and 32 / 24 / 56; 24 units 43 / 30 / 67 and 42 / 30 / 70;
  // 64 units 89 / 61 / 133 and 90 / 63 / 144.  Of 4 rows (456 CTAs): 1 unit 17.9 and 16.3, 24 units 54.0 and
  // 54.6.  At 2000 keys they are within 2 us of each other up to 16 units.
  const int cols = a.g.Hv / 4;
  const bool few = TM <= 64 && (int64_t)a.g.B * a.g.Nkv < ctas / 16;
  const MergeCut cut = few ? MergeCut{std::min(TM, 8), 8} : MergeCut{TM == 256 ? 32 : std::min(TM, 16), cols};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::max(1, ctas - 1), (unsigned)((TM + cut.rows - 1) / cut.rows),
                     (unsigned)((cols + cut.cols - 1) / cut.cols));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, TM, TN>, a, ws, ctas, cut);
  if (e == cudaSuccess) count_launch(1);
  return e;
}

template <typename T>
cudaError_t merge_t(const PagedAttn& a, const PagedWs& ws, int ctas, int tm, cudaStream_t st) {
  switch (tm) {
    case 1: return merge_tn<T, 1, kTN>(a, ws, ctas, st);
    case 4: return merge_tn<T, 4, kTN>(a, ws, ctas, st);
    case 16: return merge_tn<T, 16, kTN>(a, ws, ctas, st);
    case 32: return merge_tn<T, 32, kTN>(a, ws, ctas, st);
    case 64: return merge_tn<T, 64, kTN>(a, ws, ctas, st);
    default: return merge_tn<T, 256, 128>(a, ws, ctas, st);
  }
}

// Rows per unit: the tokens of a uniform single-row batch need no more than one.
constexpr int kMaxTM = 4;
int simt_tm(const PagedAttn& a) { return a.g.group == 1 && a.g.uniform == 1 ? 1 : kMaxTM; }

template <typename T, int LPK, int NV, int TM>
cudaError_t launch_simt(const PagedAttn& a, sdpa_dtype dt, void* wsp, int ctas, cudaStream_t st) {
  const PagedWs ws = paged_ws(wsp, ctas, TM);
  const size_t smem = sizeof(float) * (kThreads / LPK) * TM * LPK * NV * Elem<T>::kVec;
  paged_simt_kernel<T, LPK, NV, TM><<<(unsigned)ctas, kThreads, smem, st>>>(a, ws);
  count_launch(1);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_merge(a, dt, ws, ctas, TM, st) : e;
}

template <typename T, int TM>
cudaError_t launch_width(const PagedAttn& a, sdpa_dtype dt, void* ws, int ctas, cudaStream_t st) {
  constexpr int V = Elem<T>::kVec;
  const int vecs = (std::max(a.g.H, a.g.Hv) + V - 1) / V;
  if (vecs <= 8) return launch_simt<T, 8, 1, TM>(a, dt, ws, ctas, st);
  if (vecs <= 16) return launch_simt<T, 16, 1, TM>(a, dt, ws, ctas, st);
  if (vecs <= 32) return launch_simt<T, 32, 1, TM>(a, dt, ws, ctas, st);
  return launch_simt<T, 32, 2, TM>(a, dt, ws, ctas, st);
}

template <typename T>
cudaError_t launch_t(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st) {
  const int ctas = paged_sms() * kCtasPerSm;
  if (ctas <= 0) return cudaErrorInvalidDevice;
  return simt_tm(a) == 1 ? launch_width<T, 1>(a, dt, ws, ctas, st) : launch_width<T, 4>(a, dt, ws, ctas, st);
}

}  // namespace

int paged_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return std::min(n, kPagedMaxSms);
}

cudaError_t launch_paged_merge(const PagedAttn& a, sdpa_dtype dt, const PagedWs& ws, int ctas, int tm, cudaStream_t st) {
  switch (dt) {
    case SDPA_F32: return merge_t<float>(a, ws, ctas, tm, st);
    case SDPA_F16: return merge_t<__half>(a, ws, ctas, tm, st);
    default: return merge_t<__nv_bfloat16>(a, ws, ctas, tm, st);
  }
}

PagedKernel paged_kernel(const PagedAttn& a, sdpa_dtype dt) {
  if (paged_tc_supported(a, dt)) return kPagedTc;
  return paged_mma_supported(a.g.H, a.g.Hv, dt) ? kPagedMma : kPagedSimt;
}

size_t paged_workspace(int H, int Hv, sdpa_dtype dt) {
  if (paged_mma_supported(H, Hv, dt)) return std::max(paged_mma_workspace(Hv), paged_tc_workspace(Hv));
  return paged_ws_bytes(kPagedMaxSms * kCtasPerSm, kMaxTM, Hv);
}

cudaError_t launch_paged_attn(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name) {
  switch (paged_kernel(a, dt)) {
    case kPagedTc: return launch_paged_tc(a, dt, ws, st, name);
    case kPagedMma: return launch_paged_mma(a, dt, ws, st, name);
    default: break;
  }
  *name = dt == SDPA_F32 ? "paged_simt_f32" : dt == SDPA_F16 ? "paged_simt_f16" : "paged_simt_bf16";
  switch (dt) {
    case SDPA_F32: return launch_t<float>(a, dt, ws, st);
    case SDPA_F16: return launch_t<__half>(a, dt, ws, st);
    default: return launch_t<__nv_bfloat16>(a, dt, ws, st);
  }
}

cudaError_t take_paged_simt_status(int* status) { return take_words(g_paged_status, status); }

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_paged_simt)

}  // namespace sdpa
