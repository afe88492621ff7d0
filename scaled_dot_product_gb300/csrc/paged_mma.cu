// Attention over a paged cache for few rows per key (single tokens, drafted tokens) and for pages
// of any size: fp16 / bf16, H == Hv in {64, 128}.
//
// Bound by the cache's bytes: every key and value row is read once per (sequence, kv head, row
// block) whatever the number of grouped heads.  The packed rows of a unit (token x group head)
// fill the 16 rows of warp-level matrix products (m16n8k16, fp32 accumulators), which need a
// tenth of the time the bytes take; tcgen05 tiles of 128 rows would be mostly empty here and
// their scores would pass through tensor memory.  A CTA is four warps: WM of them hold 16 rows
// each, the other factor WK = 4 / WM splits the 64 keys of a tile, each warp with its own
// running maximum, sum and accumulator, joined through shared memory at the end of a unit.  Tiles arrive by 16-byte
// asynchronous copies, whose addresses go through the page table row by row, so a tile may span
// pages of any size; page ids are fetched 64 at a time, a tile before they are needed.  Rows
// past a sequence's keys are filled with zeros.  Copies run ahead of the products across unit
// boundaries.
#include <algorithm>
#include <mutex>

#include "paged_sched.cuh"

namespace sdpa {

static __device__ int g_paged_status;

namespace {

using namespace ptx;

constexpr int kThreads = 128;
constexpr int kTN = 64;
constexpr int kCtasPerSm = 2;
constexpr int kMinShare = 2;
constexpr float kRescale = 8.f;      // log2 units a maximum may grow before o is rescaled

template <int H, int WM>
struct Cfg {
  static constexpr int WK = 4 / WM, TM = 16 * WM, KW = kTN / WK;
  static constexpr int kRow = H * 2;                       // bytes of a row
  static constexpr int kTile = kTN * kRow;
  static constexpr int kStages = 3 * 128 / H;
  static constexpr int kSmem = kStages * 2 * kTile;
  static_assert(2 * kTile == 4 * 16 * H * 4, "a stage holds the four warps' accumulators");
  static constexpr int CPR = kRow / 16;                    // 16-byte chunks of a row
  static constexpr int kPass = kThreads / CPR;             // rows copied per pass
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma(float* d, const uint32_t* a, const uint32_t* b) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return BF ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi); }

// cap * tanh(x / cap) in log2 units for x given as u = x / cap: 1 - 2 / (e^2u + 1), whose absolute
// error (about 2^-23) the cap multiplies.
__device__ __forceinline__ float softcap_log2(float u, float cap_log2) {
  return cap_log2 * (1.f - __fdividef(2.f, ex2_approx(2.f * kLog2e * u) + 1.f));
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// 16-byte copy, or 16 zero bytes.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool BF, int H, int WM>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_mma_kernel(const PagedAttn a, const PagedWs ws) {
  using C = Cfg<H, WM>;
  using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
  constexpr int WK = C::WK, TM = C::TM, KW = C::KW, NT = KW / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sm_m[WK][TM], sm_l[WK][TM], sm_f[WK][TM];
  const Paged& g = a.g;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const Share sh = find_share<TM, kTN, kThreads>(a, cta, ctas, kMinShare, &g_paged_status);
  if (threadIdx.x == 0) {
    if (cta == 0) ws.start[ctas].b = sh.active;
    if (cta < sh.active) ws.start[cta] = sh.at;
  }
  pdl_launch_dependents();
  if (sh.count == 0) return;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp / WK, wk = warp % WK;
  const uint32_t sb = smem_u32(smem);

  // ---- query fragments of a unit, straight from memory: rows lane / 4 and 8 further of 16
  uint32_t qf[H / 16][4];
  auto load_q = [&](const Walk<TM, kTN>& w) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int pr = w.r.row0 + min(wm * 16 + (lane >> 2) + 8 * x, w.r.rows - 1);
      const int tok = pr / g.group;
      const uint32_t* qr = reinterpret_cast<const uint32_t*>(
          reinterpret_cast<const T*>(a.q.p) + a.q.off(0, w.kvh * g.group + pr - tok * g.group, w.s.t0 + tok));
#pragma unroll
      for (int kk = 0; kk < H / 16; ++kk) {
        qf[kk][x] = qr[kk * 8 + (lane & 3)];
        qf[kk][2 + x] = qr[kk * 8 + 4 + (lane & 3)];
      }
    }
  };
  Walk<TM, kTN> w(a, sh);

  // ---- the copying side: its own walk over the share, kStages - 1 tiles ahead.  The ids of 64
  // pages are at hand, one or two per lane; when the next tile reaches beyond them the following
  // 64 are fetched, one tile before they are needed.
  Walk<TM, kTN> wl = w;
  int lt = 0;                         // tile of wl's unit
  int wbase = 0, id0 = -1, id1 = -1;  // pages wbase + lane and wbase + 32 + lane of wl's sequence
  bool fresh = true;                  // wl entered another unit
  const T *kbase = nullptr, *vbase = nullptr;
  const int chunk = threadIdx.x % C::CPR, row_in = threadIdx.x / C::CPR;
  const bool same = g.kp.sb == g.vp.sb && g.kp.ss == g.vp.ss;
  auto fetch_ids = [&]() {
    const int k0 = (wl.r.tile0 + wl.tile + lt) * kTN;
    const int last = page_div(g, max(0, min(k0 + kTN - 1, wl.r.hi)));
    if (!fresh && last < wbase + 64) return;
    wbase = page_div(g, max(k0, wl.r.lo));
    const int32_t* table = g.table + (int64_t)wl.b * g.table_stride + wbase;
    const int end = wl.r.hi >= wl.r.lo ? page_div(g, wl.r.hi) - wbase : -1;     // last page some row admits
    id0 = lane <= end ? table[lane] : -1;
    id1 = lane + 32 <= end ? table[lane + 32] : -1;
    if (fresh) {
      kbase = reinterpret_cast<const T*>(g.kp.p) + g.kp.sh * wl.kvh + chunk * 8;
      vbase = reinterpret_cast<const T*>(g.vp.p) + g.vp.sh * wl.kvh + chunk * 8;
      fresh = false;
    }
  };
  auto copy_tile = [&](int st) {
    if (!wl.done()) {
      const int k0 = (wl.r.tile0 + wl.tile + lt) * kTN;
      const uint32_t sk = sb + st * 2 * C::kTile;
#pragma unroll
      for (int p = 0; p < kTN / C::kPass; ++p) {
        const int r = p * C::kPass + row_in;
        const int key = k0 + r, pg = page_div(g, key), i = pg - wbase;
        const int a0 = __shfl_sync(0xffffffffu, id0, i & 31), a1 = __shfl_sync(0xffffffffu, id1, i & 31);
        const int id = i < 32 ? a0 : a1;
        bool take = key >= wl.r.lo && key <= wl.r.hi;      // other keys: zeros, their pages are not read
        if (take && (unsigned)id >= (unsigned)g.num_pages) {
          atomicOr(&g_paged_status, kPagedBadPage);
          take = false;
        }
        take = take && SDPA_IN_BOUNDS(i >= 0 && i < 64 && key < g.cap, 531);
        const int slot = key - pg * g.page_size;
        const int64_t ko = take ? id * g.kp.sb + slot * g.kp.ss : 0;
        const int64_t vo = same ? ko : take ? id * g.vp.sb + slot * g.vp.ss : 0;
        const uint32_t d = sk + r * C::kRow + ((chunk ^ (r & 7)) << 4);
        cp_async16_or_zero(d, kbase + ko, take);
        cp_async16_or_zero(d + C::kTile, vbase + vo, take);
      }
      if (++lt == wl.take()) {
        lt = 0;
        wl.next(a);
        fresh = true;
      }
      if (!wl.done()) fetch_ids();
    }
    cp_async_commit();
  };
  fetch_ids();
  load_q(w);

  const float cap_log2 = a.softcap * kLog2e, cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  const float kfac = a.softcap > 0.f ? 1.f : a.scale * kLog2e;
  // fragment addresses: lane -> row and 16-byte chunk of the four 8x8 matrices of one load
  const int kr = wk * KW + ((lane >> 4) << 3) + (lane & 7), kc = (lane >> 3) & 1;
  const int vr = wk * KW + (((lane >> 3) & 1) << 3) + (lane & 7), vc = lane >> 4;
  const int prow = wm * 16 + (lane >> 2);      // this thread's rows of the unit: prow and prow + 8

  int lo[2], hi[2], full_lo = 0, full_hi = 0;  // admitted keys of the two rows, of every row
  float o[H / 8][4], m[2], l[2];
  int t = 0;                                   // tile of w's unit
  // One loop for filling the ring, the products and the units' ends: straight-line code runs once
  // per call from a cold instruction cache, which short calls feel (3 us a section, measured).
  int put = 0;                                 // stage the next copy goes to
#pragma unroll 1
  for (int ahead = C::kStages - 1;;) {
    if (ahead == 0) {
      cp_async_wait<C::kStages - 2>();
      __syncthreads();               // the tile is there, and the previous one has been read
    }
    copy_tile(put);
    put = put + 1 == C::kStages ? 0 : put + 1;
    if (ahead > 0) {
      --ahead;
      continue;
    }
    const uint32_t sk = sb + put * 2 * C::kTile, sv = sk + C::kTile;   // the oldest tile's stage
    if (t == 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        row_keys(a, w.s, w.r.row0 + min(prow + 8 * x, w.r.rows - 1), lo[x], hi[x]);
        m[x] = -INFINITY;
        l[x] = 0.f;
      }
      int tmp;
      row_keys(a, w.s, w.r.row0, tmp, full_hi);
      row_keys(a, w.s, w.r.row0 + w.r.rows - 1, full_lo, tmp);
#pragma unroll
      for (int n = 0; n < H / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    }
    {
      const int key0 = (w.r.tile0 + w.tile + t) * kTN + wk * KW;

      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < H / 16; ++kk) {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t b[4];
          const int r = kr + n * 8, c = kk * 2 + kc;
          ldsm_x4(sk + r * C::kRow + ((c ^ (r & 7)) << 4), b);
          mma<BF>(s[n], qf[kk], b);
          mma<BF>(s[n + 1], qf[kk], b + 2);
        }
      }
      if (a.softcap > 0.f) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = softcap_log2(s[n][e] * cap_in, cap_log2);
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= kfac;
      }
      if (key0 < full_lo || key0 + KW - 1 > full_hi) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + n * 8 + 2 * (lane & 3) + (e & 1), x = e >> 1;
            if (key < lo[x] || key > hi[x]) s[n][e] = -INFINITY;
          }
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      bool need = false;
      float corr[2] = {1.f, 1.f};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mx[x] = quad_max(mx[x]);
        if (mx[x] > m[x] + kRescale || (m[x] == -INFINITY && mx[x] != -INFINITY)) {
          corr[x] = ex2_approx(m[x] - mx[x]);
          m[x] = mx[x];
          need = true;
        }
      }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int n = 0; n < H / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= corr[e >> 1];
        l[0] *= corr[0];
        l[1] *= corr[1];
      }
      // rows with nothing admitted so far: exponent -inf, weight 0
      const float nm[2] = {m[0] == -INFINITY ? -INFINITY : -m[0], m[1] == -INFINITY ? -INFINITY : -m[1]};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = ex2_approx(s[n][e] + nm[e >> 1]);
          l[e >> 1] += s[n][e];
        }
#pragma unroll
      for (int kt = 0; kt < KW / 16; ++kt) {
        const uint32_t p[4] = {pack2<BF>(s[2 * kt][0], s[2 * kt][1]), pack2<BF>(s[2 * kt][2], s[2 * kt][3]),
                               pack2<BF>(s[2 * kt + 1][0], s[2 * kt + 1][1]), pack2<BF>(s[2 * kt + 1][2], s[2 * kt + 1][3])};
#pragma unroll
        for (int n = 0; n < H / 8; n += 2) {
          uint32_t b[4];
          const int r = vr + kt * 16, c = n + vc;
          ldsm_x4_t(sv + r * C::kRow + ((c ^ (r & 7)) << 4), b);
          mma<BF>(o[n], p, b);
          mma<BF>(o[n + 1], p, b + 2);
        }
      }
    }

    if (++t < w.take()) continue;

    // ---- end of the unit's tiles in this share; the next unit's query rows are on their way
    // while its results are joined and written.  The warps' accumulators, as they lie in registers
    // (float4 n of lane i at [warp][n][i]), go to the stage of the tile just read, which the next
    // copy fills only after the barrier above.
    const bool whole = w.whole();
    const int64_t slot = 2 * (int64_t)cta + (w.begins() ? 1 : 0);
    const int rows = w.r.rows, row0 = w.r.row0, t0 = w.s.t0, head0 = w.kvh * g.group;
    w.next(a);
    t = 0;
    if (!w.done()) load_q(w);
    __syncthreads();                 // every warp has read the tile
    float4* acc = reinterpret_cast<float4*>(smem + (sk - sb));
#pragma unroll
    for (int n = 0; n < H / 8; ++n) acc[(warp * (H / 8) + n) * 32 + lane] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] = quad_sum(l[x]);
      if ((lane & 3) == 0) {
        sm_m[wk][prow + 8 * x] = m[x];
        sm_l[wk][prow + 8 * x] = l[x];
      }
    }
    __syncthreads();
    if ((int)threadIdx.x < rows) {
      const int r = threadIdx.x;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int k = 0; k < WK; ++k) M = fmaxf(M, sm_m[k][r]);
      float f[WK];
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        f[k] = sm_m[k][r] == -INFINITY ? 0.f : ex2_approx(sm_m[k][r] - M);
        L = fmaf(f[k], sm_l[k][r], L);
      }
      float sc = 1.f;
      if (whole) {
        sc = row_scale<T>(a, head0 + (row0 + r) % g.group, M, L);
      } else if (SDPA_IN_BOUNDS(slot < 2 * ctas, 533)) {
        *reinterpret_cast<float2*>(ws.ml + (slot * TM + r) * 2) = make_float2(M, L);
      }
#pragma unroll
      for (int k = 0; k < WK; ++k) sm_f[k][r] = f[k] * sc;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (H / 4); i += kThreads) {
      // row r, columns c .. c + 3: two lanes' halves of one fragment per warp
      const int r = i / (H / 4), c = (i % (H / 4)) * 4;
      const float2* src = reinterpret_cast<const float2*>(acc) +
                          ((((r >> 4) * WK) * (H / 8) + (c >> 3)) * 32 + (r & 7) * 4 + ((c & 4) >> 1)) * 2 + ((r >> 3) & 1);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const float f = sm_f[k][r];
        const float2 p = src[k * (H / 8) * 64], q = src[k * (H / 8) * 64 + 2];
        v.x = fmaf(f, p.x, v.x);
        v.y = fmaf(f, p.y, v.y);
        v.z = fmaf(f, q.x, v.z);
        v.w = fmaf(f, q.y, v.w);
      }
      if (whole) {
        const int pr = row0 + r, tok = pr / g.group, h = head0 + pr - tok * g.group;
        T* y = reinterpret_cast<T*>(const_cast<void*>(a.y.p)) + a.y.off(0, h, t0 + tok);
        if (SDPA_IN_BOUNDS(t0 + tok < g.tokens && h < g.Nq, 532))
          *reinterpret_cast<uint2*>(y + c) = make_uint2(pack2<BF>(v.x, v.y), pack2<BF>(v.z, v.w));
      } else if (SDPA_IN_BOUNDS(slot < 2 * ctas, 534)) {
        *reinterpret_cast<float4*>(ws.o + (slot * TM + r) * H + c) = v;
      }
    }
    if (w.done()) break;
  }
  cp_async_wait<0>();
}

// Rows per unit: the smallest of 16, 32 and 64 that holds all rows of a sequence with max_new
// tokens, at most 64.
int mma_tm(const PagedAttn& a) {
  const int64_t rows = (int64_t)a.max_new * a.g.group;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

template <bool BF, int H, int WM>
cudaError_t launch_wm(const PagedAttn& a, sdpa_dtype dt, void* wsp, cudaStream_t st) {
  using C = Cfg<H, WM>;
  // 228 KB per SM, of which each CTA takes 1 KB for itself
  static_assert(C::kSmem + 3 * C::WK * C::TM * 4 + 128 + 1024 <= 233472 / kCtasPerSm, "shared memory");
  const int ctas = paged_sms() * kCtasPerSm;
  if (ctas <= 0) return cudaErrorInvalidDevice;
  // per device: set at every call (the attribute belongs to the current context)
  cudaError_t e = cudaFuncSetAttribute(paged_mma_kernel<BF, H, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const PagedWs ws = paged_ws(wsp, ctas, C::TM);
  paged_mma_kernel<BF, H, WM><<<(unsigned)ctas, kThreads, C::kSmem, st>>>(a, ws);
  count_launch(1);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_merge(a, dt, ws, ctas, C::TM, st) : e;
}

template <bool BF, int H>
cudaError_t launch_h(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st) {
  switch (mma_tm(a)) {
    case 16: return launch_wm<BF, H, 1>(a, dt, ws, st);
    case 32: return launch_wm<BF, H, 2>(a, dt, ws, st);
    default: return launch_wm<BF, H, 4>(a, dt, ws, st);
  }
}

}  // namespace

bool paged_mma_supported(const PagedAttn& a, sdpa_dtype dt) {
  return dt != SDPA_F32 && a.g.H == a.g.Hv && (a.g.H == 64 || a.g.H == 128);
}

size_t paged_mma_workspace(const PagedAttn& a) {
  return paged_ws_bytes(kPagedMaxSms * kCtasPerSm, mma_tm(a), a.g.Hv);
}

cudaError_t launch_paged_mma(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name) {
  const bool bf = dt == SDPA_BF16;
  if (a.g.H == 128) {
    *name = bf ? "paged_mma_bf16_h128" : "paged_mma_f16_h128";
    return bf ? launch_h<true, 128>(a, dt, ws, st) : launch_h<false, 128>(a, dt, ws, st);
  }
  *name = bf ? "paged_mma_bf16_h64" : "paged_mma_f16_h64";
  return bf ? launch_h<true, 64>(a, dt, ws, st) : launch_h<false, 64>(a, dt, ws, st);
}

cudaError_t take_paged_mma_status(int* status) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_paged_status, sizeof v);
  if (e != cudaSuccess) return e;
  *status = v;
  if (v) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_paged_status, &zero, sizeof zero);
  }
  return e;
}

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_paged_mma)

}  // namespace sdpa
