// Attention over a paged cache of 4 bits a value in fp32 arithmetic, for every type and head size.
//
// A lane has 16 channels of a key: two words of codes and the minimum and scale of their group, so
// that a score's part is scale * sum(q * code) + minimum * sum(q).  LPK lanes hold a key; the 128 / LPK
// lane groups of a block take different keys and keep their own running maximum, sum and
// accumulator of TM query rows, joined in shared memory at the end of a unit (and between CTAs by
// the joining kernel of the caches in the model's type).  It serves fp32, since the tensor-core
// kernels take a query and a weight as one 16-bit operand each, and head sizes that those do not tile.
// Eight float32 sequences of 500 to 4000 keys, 16/4 heads of 64, 21.3 us (latency); 16 of 500 to 16000 keys, 64/8 heads
// of 128, 296 us (0.75 TB/s: arithmetic, four rows a unit).  Registers leave two CTAs an SM at four rows.
#include <algorithm>

#include "paged4.h"
#include "paged_sched.cuh"

namespace sdpa {

static __device__ int g_paged4_status[1];

namespace {

constexpr int kThreads = 128;
constexpr int kTN = 64;          // keys per tile of the schedule
// CTAs per SM: what the registers of TM rows leave.
constexpr int ctas_per_sm(int tm) { return tm == 1 ? 3 : 2; }
constexpr int kOV = 1;           // a unit's cost beside its tiles, in tiles
constexpr int kMinShare = 2;
constexpr int kCh = 16;          // channels per lane
constexpr int kMaxTM = 4;
constexpr int kUnroll = 4;       // keys per lane group and step

constexpr int log2i(int x) { return x <= 1 ? 0 : 1 + log2i(x / 2); }

// A lane's part of a record.
template <typename T> struct Part { uint2 code; uint32_t side; };
template <> struct Part<float> { uint2 code; float2 side; };

template <typename T>
__device__ __forceinline__ Part<T> load_part(const unsigned char* rec, int D, int c0) {
  Part<T> p;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(rec + c0 / 2);
  p.code = make_uint2(__ldg(w), __ldg(w + 1));
  const unsigned char* s = rec + D / 2 + c0 / kQ4Group * 2 * (int)sizeof(T);
  if constexpr (sizeof(T) == 4) p.side = __ldg(reinterpret_cast<const float2*>(s));
  else p.side = __ldg(reinterpret_cast<const uint32_t*>(s));
  return p;
}
template <typename T>
__device__ __forceinline__ Part<T> zero_part() {
  Part<T> p;
  p.code = make_uint2(0u, 0u);
  if constexpr (sizeof(T) == 4) p.side = make_float2(0.f, 0.f);
  else p.side = 0u;
  return p;
}
// minimum and scale
template <typename T>
__device__ __forceinline__ float2 side_of(const Part<T>& p) {
  if constexpr (sizeof(T) == 4) return p.side;
  else {
    const T* e = reinterpret_cast<const T*>(&p.side);
    return make_float2(Elem<T>::to_f32(e[0]), Elem<T>::to_f32(e[1]));
  }
}
// The sixteen codes as floats: 2^23 + code has the code in its last bits.
__device__ __forceinline__ void codes_of(const uint2& w, float* f) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f[e] = __uint_as_float(0x4b000000u | ((w.x >> (4 * e)) & 15u)) - 8388608.f;
    f[8 + e] = __uint_as_float(0x4b000000u | ((w.y >> (4 * e)) & 15u)) - 8388608.f;
  }
}

template <typename T, int LPK, int TM>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(TM)) paged4_simt_kernel(const PagedAttn a, const PagedWs ws) {
  constexpr int KPI = kThreads / LPK;
  constexpr int HM = LPK * kCh;          // widest head
  extern __shared__ float smem[];        // [KPI][TM][HM]
  __shared__ float sm_m[KPI][TM], sm_l[KPI][TM];
  const Paged& g = a.g;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const Share sh = find_share<TM, kTN, kOV, kThreads>(a, cta, ctas, kMinShare, g_paged4_status);
  if (threadIdx.x == 0) {
    if (cta == 0) ws.start[ctas].b = sh.active;
    if (cta < sh.active) ws.start[cta] = sh.at;
  }
  pdl_launch_dependents();
  const int grp = threadIdx.x / LPK, t = threadIdx.x % LPK, c0 = t * kCh;
  const float cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  // Scores of a step: score r * kUnroll + u of row r and key u.  After SC exchanges a lane holds the sums
  // of R of them, of one row, from key my_u on; UB exchanges span the lanes of a row.
  constexpr int NS = TM * kUnroll, SC = log2i(NS) < log2i(LPK) ? log2i(NS) : log2i(LPK), R = NS >> SC;
  constexpr int UB = log2i(kUnroll) > log2i(R) ? log2i(kUnroll) - log2i(R) : 0;
  static_assert(R <= kUnroll, "a lane's scores belong to one row");
  const int first = (t >> (log2i(LPK) - SC)) << (log2i(NS) - SC);
  const int my_row = first / kUnroll, my_u = first % kUnroll;
  auto lane_of = [](int score) { return (score >> (log2i(NS) - SC)) << (log2i(LPK) - SC); };

  for (Walk<TM, kTN, kOV> w(a, sh); !w.done(); w.next(a)) {
    const int nr = w.r.rows;
    float q[TM][kCh], qs[TM], acc[TM][kCh];
#pragma unroll
    for (int r = 0; r < TM; ++r) {
      const int pr = w.r.row0 + min(r, nr - 1);
      const T* row = reinterpret_cast<const T*>(a.q.p) +
                     a.q.off(0, w.kvh * g.group + pr - group_div(g, pr) * g.group, w.s.t0 + group_div(g, pr));
      qs[r] = 0.f;
      constexpr int V = Elem<T>::kVec;
#pragma unroll
      for (int n = 0; n < kCh / V; ++n)
        unpack16<T>(c0 < g.H ? *reinterpret_cast<const uint4*>(row + c0 + n * V) : make_uint4(0u, 0u, 0u, 0u), q[r] + n * V);
#pragma unroll
      for (int e = 0; e < kCh; ++e) {
        qs[r] += q[r][e];
        acc[r][e] = 0.f;
      }
    }
    // this lane's row of the scores: its keys, running maximum and part of the sum
    int lo, hi;
    row_keys(a, w.s, w.r.row0 + min(my_row, nr - 1), lo, hi);
    float m = -INFINITY, l = 0.f;
    const int64_t j_tile = (int64_t)(w.r.tile0 + w.tile) * kTN;
    const int64_t j_begin = max(j_tile, (int64_t)w.r.lo);      // pages below a window are not read
    const int64_t j_end = min((int64_t)w.r.hi + 1, j_tile + (int64_t)w.take() * kTN);
    const int32_t* table = g.table + (int64_t)w.b * g.table_stride;

    // keys of one step: those at base + grp + u * KPI.  Their records are loaded one step ahead, the ids
    // of their pages two.
    constexpr int kStep = KPI * kUnroll;
    auto load_ids = [&](int64_t base, int* id) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t j = base + grp + u * KPI;
        id[u] = j < j_end ? table[page_div(g, (int)j)] : -1;
      }
    };
    auto load_rows = [&](int64_t base, const int* id, Part<T> (&kv)[kUnroll], Part<T> (&vv)[kUnroll]) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t j = base + grp + u * KPI;
        const int key = (int)min(j, (int64_t)g.cap), slot = key - page_div(g, key) * g.page_size;
        bool take = j < j_end;
        if (take && (unsigned)id[u] >= (unsigned)g.num_pages) {
          atomicOr(g_paged4_status, kPagedBadPage);
          take = false;                    // read as zeros
        }
        take = take && SDPA_IN_BOUNDS(key < g.cap && slot < g.page_size, 581);
        const unsigned char* kr = reinterpret_cast<const unsigned char*>(g.kp.p) + g.kp.off(id[u], w.kvh, slot);
        const unsigned char* vr = reinterpret_cast<const unsigned char*>(g.vp.p) + g.vp.off(id[u], w.kvh, slot);
        kv[u] = take && c0 < g.H ? load_part<T>(kr, g.H, c0) : zero_part<T>();
        vv[u] = take && c0 < g.Hv ? load_part<T>(vr, g.Hv, c0) : zero_part<T>();
      }
    };
    int id[kUnroll];
    load_ids(j_begin, id);
#pragma unroll 1
    for (int64_t base = j_begin; base < j_end; base += kStep) {
      Part<T> kv[kUnroll], vv[kUnroll];
      load_rows(base, id, kv, vv);
      load_ids(base + kStep, id);
      // every lane's part of the step's TM x kUnroll scores, then their sums dealt to the lanes: at each
      // exchange a lane keeps the half of the scores that its lane bit names
      float s[NS];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float kf[kCh];
        codes_of(kv[u].code, kf);
        const float2 side = side_of<T>(kv[u]);
#pragma unroll
        for (int r = 0; r < TM; ++r) {
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < kCh; ++e) dot = fmaf(q[r][e], kf[e], dot);
          s[r * kUnroll + u] = fmaf(side.y, dot, side.x * qs[r]);
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
          for (int e = 0; e < kCh; ++e) acc[r][e] *= c;
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        s[i] = s[i] == -INFINITY ? 0.f : exp2f(s[i] - m);
        l += s[i];
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float vf[kCh];
        codes_of(vv[u].code, vf);
        const float2 side = side_of<T>(vv[u]);
#pragma unroll
        for (int e = 0; e < kCh; ++e) vf[e] = fmaf(vf[e], side.y, side.x);
#pragma unroll
        for (int r = 0; r < TM; ++r) {
          const float p = __shfl_sync(0xffffffffu, s[(r * kUnroll + u) & (R - 1)], lane_of(r * kUnroll + u), LPK);
#pragma unroll
          for (int e = 0; e < kCh; ++e) acc[r][e] = fmaf(p, vf[e], acc[r][e]);
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
    for (int r = 0; r < TM; ++r)
#pragma unroll
      for (int e = 0; e < kCh; ++e) smem[(grp * TM + r) * HM + c0 + e] = acc[r][e];
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
        if (SDPA_IN_BOUNDS(w.s.t0 + group_div(g, pr) < g.tokens && h < g.Nq, 582))
          y[d] = Elem<T>::from_f32(O * row_scale<T>(a, h, M, L));
      } else if (SDPA_IN_BOUNDS(slot < 2 * ctas, 583)) {
        ws.o[(slot * TM + r) * g.Hv + d] = O;
        if (d == 0) {
          ws.ml[(slot * TM + r) * 2] = M;
          ws.ml[(slot * TM + r) * 2 + 1] = L;
        }
      }
    }
  }
}

// Rows per unit: the tokens of a uniform single-row batch need no more than one.
int simt_tm(const PagedAttn& a) { return a.g.group == 1 && a.g.uniform == 1 ? 1 : kMaxTM; }

template <typename T, int LPK, int TM>
cudaError_t launch_simt(const PagedAttn& a, sdpa_dtype dt, void* wsp, int ctas, cudaStream_t st) {
  const PagedWs ws = paged_ws(wsp, ctas, TM);
  paged4_simt_kernel<T, LPK, TM><<<(unsigned)ctas, kThreads, sizeof(float) * kThreads * TM * kCh, st>>>(a, ws);
  count_launch(1);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_merge(a, dt, ws, ctas, TM, st) : e;
}

template <typename T, int TM>
cudaError_t launch_width(const PagedAttn& a, sdpa_dtype dt, void* ws, int ctas, cudaStream_t st) {
  const int D = std::max(a.g.H, a.g.Hv);
  if (D <= 64) return launch_simt<T, 4, TM>(a, dt, ws, ctas, st);
  if (D <= 128) return launch_simt<T, 8, TM>(a, dt, ws, ctas, st);
  return launch_simt<T, 16, TM>(a, dt, ws, ctas, st);
}

template <typename T>
cudaError_t launch_t(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st) {
  const int sms = paged_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  return simt_tm(a) == 1 ? launch_width<T, 1>(a, dt, ws, sms * ctas_per_sm(1), st)
                         : launch_width<T, kMaxTM>(a, dt, ws, sms * ctas_per_sm(kMaxTM), st);
}

}  // namespace

PagedKernel paged4_kernel(const PagedAttn& a, sdpa_dtype dt) {
  if (paged4_tc_supported(a, dt)) return kPagedTc;
  return paged4_mma_supported(a.g.H, a.g.Hv, dt) ? kPagedMma : kPagedSimt;
}

size_t paged4_workspace(int H, int Hv, sdpa_dtype dt) {
  if (paged4_mma_supported(H, Hv, dt)) return std::max(paged4_mma_workspace(Hv), paged4_tc_workspace(Hv));
  return paged_ws_bytes(kPagedMaxSms * ctas_per_sm(1), kMaxTM, Hv);
}

cudaError_t launch_paged4_attn(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name) {
  switch (paged4_kernel(a, dt)) {
    case kPagedTc: return launch_paged4_tc(a, dt, ws, st, name);
    case kPagedMma: return launch_paged4_mma(a, dt, ws, st, name);
    default: break;
  }
  *name = dt == SDPA_F32 ? "paged4_simt_f32" : dt == SDPA_F16 ? "paged4_simt_f16" : "paged4_simt_bf16";
  switch (dt) {
    case SDPA_F32: return launch_t<float>(a, dt, ws, st);
    case SDPA_F16: return launch_t<__half>(a, dt, ws, st);
    default: return launch_t<__nv_bfloat16>(a, dt, ws, st);
  }
}

cudaError_t take_paged4_simt_status(int* status) { return take_words(g_paged4_status, status); }

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_paged4_simt)

}  // namespace sdpa
