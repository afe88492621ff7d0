// Attention over a paged cache of 4 bits a value for few rows per key (single tokens, drafted tokens):
// fp16 / bf16, H == Hv in {64, 128}.
//
// The cache's bytes bound it, with the instructions that make operands of its codes close behind, so
// as few of those as possible are spent on a code.  The products are warp-level ones (m16n8k16, fp16 with fp32
// accumulators), with keys on the long side, S^T = K Q^T and O^T = V^T P^T: the eight rows of the short side are what
// a token's group of heads fills.
//  - A code c in the last bits of a 16-bit word is the subnormal fp16 number c 2^-24, which the products take
//    exactly; the next four bits are 16 times that.  One AND makes two operands, one shift four more.  No
//    code is converted, scaled or rounded.  The queries that meet the 16-fold codes are divided by 16.
//  - Keys: a score is sum over groups of scale_g (q . code)_g + minimum_g sum(q)_g, in fp32 after the products.
//    Any order of channels serves, so a lane takes eight neighbouring codes as they lie.  Queries enter as fp16,
//    their row times the power of two that brings its largest to 2^13: bf16 values keep their eight bits down
//    to 2^-27 of that.
//  - Values: a weight times its key's scale, rounded to fp16, is the second operand, one for each group;
//    the minima are summed in fp32.  In fp16 caches 8 is taken off every code by a further product with the same
//    rounded operand (and 8 scales added to the minimum), so that the rounding touches a value's distance from the
//    middle of its range and not from the minimum; in bf16 the output's rounding is far larger.
//  - fp16's range: a power of two for each row and group of channels, the factor, brings the largest product of weight and
//    scale that the warp has seen there to [1/2, 1) whenever it is set.  That is anew where a score passes the running
//    maximum by 2^4, or a scale times some row's factor 2^11: operands stay within 2^15, and one far below the largest
//    of its row and group is off by 2^-24 of that at most.  It has to follow the products themselves: with one factor a
//    warp, of the largest weight and the largest scale, a large value of no weight took the others' bits away.  Packed
//    products keep its cost small (single tokens 535 us, 531 with one factor; 16 rows 132, 121); a sequence whose weight lies
//    on values 2^-11 and less of all others takes up to 1.3 times as long, as every block asks for new factors.
// A unit's rows are dealt to WM warps (8 NT each), the keys of a tile to WK; each warp keeps its own m, factors, sum and
// accumulator, joined through shared memory at the end of a unit.
//
// One producer warp keeps a ring of tiles of keys full across unit boundaries. A page's records of a head lie
// one after another, so whatever part of a page falls into a tile is one bulk copy. Rows of 80 (40) bytes put
// the words that a warp reads at a time into different banks. About 380 instructions a block of 16 keys of 128
// channels, half of them on the half-rate integer pipe, in chains that 14 warps an SM do not cover: 55 % of the issue
// slots and 50 % of that pipe are taken (32 single tokens), and a fixed latency is what a warp waits for most. 128 single
// tokens, 1000 to 32000 keys, 64/8 heads of 128: 535 us, 4.9 TB/s of records (floor 383); fp16 586; 64 channels 296 (floor
// 191); four short sequences 11.7 us. Keys that no row of the unit admits take a scale and a minimum of zero, since 0 x NaN is
// not 0. Every wait is bounded: on expiry the kernel raises an abort flag, goes through its loops without
// waiting, lets its own copies finish and records SDPA_ERR_TIMEOUT.
#include <algorithm>
#include <cstdlib>
#include <type_traits>

#include "paged4.h"
#include "paged_sched.cuh"

namespace sdpa {

static __device__ int g_paged4_words[2];     // status bits, SDPA_ERR_TIMEOUT after an expired wait

namespace {

using namespace ptx;

constexpr int kCtasPerSm = 2;
constexpr int kOV = 1;                // a unit's cost beside its tiles, in tiles
constexpr int kMinShare = 2;
constexpr float kRescale = 4.f;       // log2 units a maximum may grow before the state is rescaled
// An operand is at most 2^(kRescale + kScaleRoom) = 2^15: a scale times its row's factor stays within 2^kScaleRoom.
constexpr int kScaleRoom = 11;
constexpr int kMostF = 120;           // log2 of the largest factor, where a row has no product yet
constexpr float kNone = -1e30f;       // the maximum of a row that has admitted no key: finite, so that differences are numbers

template <int H, int NT, int WM>
struct Cfg {
  // Product warps.  With the producer eight warps leave 128 registers a thread at two CTAs an SM, which
  // eight rows take; five leave 168 for 16 rows.
  static constexpr int NW = NT == 1 ? 7 : 4;
  static constexpr int kProducts = NW * 32, kThreads = kProducts + 32;
  // Keys of a tile: 32 a warp, 64 where records are half as long (with 16 a warp's waits and loops took 585 us
  // where these take 535, and with 64 channels 469 where these take 299).
  static constexpr int WK = NW / WM, TN = NT == 1 ? (H == 64 ? 64 : 32) * NW : 128, KW = TN / WK, TM = 8 * NT * WM, G = H / kQ4Group;
  static constexpr int kRow = q4_row_bytes(H, 2);
  static constexpr int kTile = TN * kRow;
  static constexpr int kPitch = H + 4;                     // floats of a row of the joining buffer
  static constexpr int kAcc = NW * 8 * NT * kPitch * 4;
  static constexpr int kStages = H == 64 ? (NT == 1 ? 2 : 8) : NT == 1 ? 2 : 3;
  static constexpr bool kSharedFac = NT == 2 && H == 128;
  static constexpr int kSmem = kStages * 2 * kTile + kAcc + 128;
  static_assert(KW % 16 == 0, "a warp takes whole blocks of 16 keys");
};

struct Mma4Args {
  PagedAttn a;
  PagedWs ws;
  uint64_t wait_ns;
};

__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with accumulators that start at zero.
__device__ __forceinline__ void mma_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Minima times sums of queries: the first operand holds numbers of the cache's type.
template <typename T>
__device__ __forceinline__ void mma_minima(float* d, uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%4,%5}, {%6,%7}, {%8,%8,%8,%8};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%4,%5}, {%6,%7}, {%8,%8,%8,%8};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0), "r"(b1), "f"(0.f));
}
// 8 x 8 matrix of 16-bit values, a row in four lanes, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar) : "memory");
}
// cap * tanh(x / cap) in log2 units for x given as u = x / cap: 1 - 2 / (e^2u + 1), whose absolute
// error (about 2^-23) the cap multiplies.
__device__ __forceinline__ float softcap_log2(float u, float cap_log2) {
  return cap_log2 * (1.f - __fdividef(2.f, ex2_approx(2.f * kLog2e * u) + 1.f));
}
// Over the eight lanes that hold the same rows.
__device__ __forceinline__ float rows_max(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float rows_sum(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// The minimum (low half) and scale (high half) of a group.
template <typename T>
__device__ __forceinline__ float low_half(uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(w << 16);
  else return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
}
template <typename T>
__device__ __forceinline__ float high_half(uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(w & 0xffff0000u);
  else return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// floor(log2 x), for x normal; -127 for less.
__device__ __forceinline__ int log2_floor(float x) { return ((__float_as_int(x) >> 23) & 255) - 127; }

// The sides of a record: G words.
template <int G>
__device__ __forceinline__ void load_sides(const unsigned char* p, uint32_t* w) {
  if constexpr (G == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  }
}

template <typename T, int H, int NT, int WM>
__global__ void __launch_bounds__(Cfg<H, NT, WM>::kThreads, kCtasPerSm) paged4_mma_kernel(const __grid_constant__ Mma4Args args) {
  using C = Cfg<H, NT, WM>;
  using Wk = Walk<C::TM, C::TN, kOV>;
  constexpr int kTN = C::TN, WK = C::WK, TM = C::TM, KW = C::KW, G = C::G, kRow = C::kRow;
  constexpr bool kCentre = std::is_same<T, __half>::value;
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bar_full[C::kStages], bar_empty[C::kStages];
  __shared__ float sm_m[WK][TM], sm_l[WK][TM], sm_f[WK][TM];
  __shared__ __align__(8) float sm_fac[C::kSharedFac ? C::NW : 1][NT][G][8];
  __shared__ int abort_flag;
  const PagedAttn& a = args.a;
  const PagedWs& ws = args.ws;
  const Paged& g = a.g;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto b_full = [&](int s) { return smem_u32(&bar_full[s]); };
  auto b_empty = [&](int s) { return smem_u32(&bar_empty[s]); };
  volatile int* abortp = &abort_flag;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full(s), 32);
      mbar_init(b_empty(s), C::NW);
    }
    fence_mbar_init();
  }
  const Share sh = find_share<TM, kTN, kOV, C::kThreads>(a, cta, ctas, kMinShare, &g_paged4_words[0]);
  if (threadIdx.x == 0) {
    if (cta == 0) ws.start[ctas].b = sh.active;
    if (cta < sh.active) ws.start[cta] = sh.at;
  }
  pdl_launch_dependents();
  if (sh.count == 0) return;
  __syncthreads();
  Wk w(a, sh);
  if (w.done()) return;

  if (warp == C::NW) {
    // ================================================================ producer
    // A tile's admitted keys, widened to even ones (records of 40 bytes are copied in pairs: pages
    // have an even number of them), are cut at page ends; a lane has the parts lane, lane + 32, ...
    const uint32_t sb = smem_u32(smem);
    int st = 0, it = 0;               // stage, turns of the ring
    bool ok = true;
    auto wait_free = [&]() {
      if (it > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(b_empty(st), (it - 1) & 1, abortp, args.wait_ns));
      return ok;
    };
    auto keys_of = [&](int t, int& k0, int& first, int& last) {
      k0 = (w.r.tile0 + w.tile + t) * kTN;
      first = max(k0, w.r.lo) & ~1;
      last = min(k0 + kTN, (w.r.hi + 2) & ~1);
      if (kRow % 16 == 0) {           // a page may end behind an odd slot
        first = max(k0, w.r.lo);
        last = min(k0 + kTN, w.r.hi + 1);
      }
    };
    // The ids of 64 pages are at hand, two in a lane; the further 32 are on their way while the nearer
    // ones are used.
    int wbase = 0, near_id = -1, far_id = -1;
    const int32_t* table = nullptr;
    int end = -1;                     // last page that some row of the unit admits
    auto fetch = [&](int page) { return page <= end ? table[page] : -1; };
    auto start_unit = [&]() {
      if (w.done()) return;
      int k0, first, last;
      table = g.table + (int64_t)w.b * g.table_stride;
      keys_of(0, k0, first, last);
      wbase = page_div(g, max(first, 0));
      keys_of(w.take() - 1, k0, first, last);
      end = first < last ? page_div(g, last - 1) : -1;
      near_id = fetch(wbase + lane);
      far_id = fetch(wbase + 32 + lane);
    };
    start_unit();
    while (!w.done() && wait_free()) {
      const int n = w.take();
      for (int t = 0; t < n && wait_free(); ++t) {
        int k0, first, last;
        keys_of(t, k0, first, last);
        const int p0 = page_div(g, max(first, 0)), parts = first < last ? page_div(g, last - 1) - p0 + 1 : 0;
        const uint32_t at = sb + st * 2 * C::kTile;
        while (p0 >= wbase + 32) {
          wbase += 32;
          near_id = far_id;
          far_id = fetch(wbase + 32 + lane);
        }
        // page of this lane's first part
        const int x = p0 - wbase + lane;
        const int from_near = __shfl_sync(0xffffffffu, near_id, x & 31), from_far = __shfl_sync(0xffffffffu, far_id, x & 31);
        const int id = x < 32 ? from_near : from_far;
        // this lane's parts are announced before any of them is copied
        uint32_t bytes = 0;
        auto span = [&](int part, int& from, int& to) {
          from = max(first, (p0 + part) * g.page_size);
          to = min(last, (p0 + part + 1) * g.page_size);
        };
        int pid = id;
        for (int part = lane; part < parts; part += 32) {
          if (part >= 32) pid = table[p0 + part];
          int from, to;
          span(part, from, to);
          if ((unsigned)pid < (unsigned)g.num_pages) {
            bytes += 2 * (to - from) * kRow;
            continue;
          }
          atomicOr(&g_paged4_words[0], kPagedBadPage);
          // its keys and values read as zeros
          for (int i = 0; i < (to - from) * kRow; i += 16) {
            st_shared_v4(at + (from - k0) * kRow + i, 0u, 0u, 0u, 0u);
            st_shared_v4(at + C::kTile + (from - k0) * kRow + i, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();      // before a later copy is written there
        }
        mbar_arrive_expect_tx(b_full(st), bytes);
        pid = id;
        for (int part = lane; part < parts; part += 32) {
          if (part >= 32) pid = table[p0 + part];
          int from, to;
          span(part, from, to);
          if ((unsigned)pid < (unsigned)g.num_pages &&
              SDPA_IN_BOUNDS(st < C::kStages && from >= k0 && to <= k0 + kTN && from < to && w.kvh < g.Nkv, 591)) {
            const int slot = from - (p0 + part) * g.page_size;
            const uint32_t d = at + (from - k0) * kRow;
            const unsigned char* ks = reinterpret_cast<const unsigned char*>(g.kp.p) + g.kp.off(pid, w.kvh, 0) + slot * kRow;
            const unsigned char* vs = reinterpret_cast<const unsigned char*>(g.vp.p) + g.vp.off(pid, w.kvh, 0) + slot * kRow;
            bulk_load(d, ks, (to - from) * kRow, b_full(st));
            bulk_load(d + C::kTile, vs, (to - from) * kRow, b_full(st));
          }
        }
        __syncwarp();
        if (++st == C::kStages) { st = 0; ++it; }
      }
      if (!ok) break;
      w.next(a);
      start_unit();
    }
    // Copies may still be on their way when a wait has expired, whichever role's it was and however
    // early the last copy was issued: the CTA, whose shared memory they write, ends behind them.
    named_bar_sync(2, C::kThreads);
    if (*abortp) {
      constexpr uint64_t kDrainNs = 2000000000ull;
      for (int s = 0; s < C::kStages; ++s) {
        const int turns = it + (s < st ? 1 : 0);
        if (turns > 0) mbar_wait_bounded(b_full(s), (turns - 1) & 1, nullptr, kDrainNs);
      }
      if (lane == 0) atomicExch(&g_paged4_words[1], (int)SDPA_ERR_TIMEOUT);
    }
    return;
  }

  // ================================================================ products
  const int wm = warp / WK, wk = warp % WK;
  const int r8 = lane >> 2, j4 = lane & 3;
  const int prow = wm * 8 * NT;                // first row of this warp in the unit
  // Queries: rows r8 of each eight, channels 8 j4 .. + 7 of each group, as the codes of a word come:
  // (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16.  For rows 2 j4 and + 1 of each eight: sums of each group and
  // the factor of the scores.
  uint32_t qf[NT][G][4];
  // qm: the sum of group j4 of row r8 in three parts of the type (in fp16 times 2^-6), for the minima
  uint32_t qm[NT][2];
  float kf[NT][2];
  auto load_q = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int pr = w.r.row0 + min(prow + n * 8 + r8, w.r.rows - 1);
      const int tok = group_div(g, pr);
      const T* row = reinterpret_cast<const T*>(a.q.p) + a.q.off(0, w.kvh * g.group + pr - tok * g.group, w.s.t0 + tok) + 8 * j4;
      uint4 raw[G];
      float top = 0.f;
#pragma unroll
      for (int x = 0; x < G; ++x) {
        raw[x] = *reinterpret_cast<const uint4*>(row + 32 * x);
        float f[8];
        unpack16<T>(raw[x], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int shift = max(-103, min(13 - log2_floor(top), 100));
      const float up = pow2(shift);
      float sum[G];
#pragma unroll
      for (int x = 0; x < G; ++x) {
        float f[8];
        unpack16<T>(raw[x], f);
        sum[x] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] *= up;
          sum[x] += f[e];
        }
        qf[n][x][0] = pack_f16x2(f[0], f[4]);
        qf[n][x][1] = pack_f16x2(f[1] * 0.0625f, f[5] * 0.0625f);
        qf[n][x][2] = pack_f16x2(f[2], f[6]);
        qf[n][x][3] = pack_f16x2(f[3] * 0.0625f, f[7] * 0.0625f);
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
      }
      {
        float part = sum[0];
#pragma unroll
        for (int y = 1; y < G; ++y) part = j4 == y ? sum[y] : part;
        part = j4 < G ? part * pow2(std::is_same<T, __half>::value ? -6 : -24) : 0.f;
        const float hi = Elem<T>::to_f32(Elem<T>::from_f32(part));
        const float mid = Elem<T>::to_f32(Elem<T>::from_f32(part - hi));
        const float lo = part - hi - mid;
        if constexpr (std::is_same<T, __half>::value) {
          qm[n][0] = pack_f16x2(hi, mid);
          qm[n][1] = pack_f16x2(lo, 0.f);
        } else {
          qm[n][0] = pack_bf16x2(hi, mid);
          qm[n][1] = pack_bf16x2(lo, 0.f);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int from = (2 * j4 + x) * 4;
        const int sf = __shfl_sync(0xffffffffu, shift, from);
        // 24 - sf lies in -76 .. 127
        kf[n][x] = (a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e) * pow2(24) * pow2(-sf);
      }
    }
  };
  load_q();
  const float cap_log2 = a.softcap * kLog2e;
  // addresses in a tile: words of this lane's two keys, of its four values
  const int koff = r8 * kRow + 4 * j4, voff = 2 * j4 * kRow + 4 * (r8 >> 1), soff = r8 * kRow + H / 2;
  const uint32_t vsel = r8 & 1 ? 0x7632u : 0x5410u;

  int full_lo = 0, full_hi = 0;                // keys that every row admits
  float o[NT][G][2][4], mt[NT][2][G], m[NT][2], l[NT][2];
  // Factors of a row's products of weight and scale, powers of two, which o holds too; in shared memory where registers are full
  // (16 rows of 128 channels: 132 us, in registers 162).
  float fac[C::kSharedFac ? 1 : NT][2][G];
  float* my_fac = &sm_fac[C::kSharedFac ? warp : 0][0][0][2 * j4];
  auto factors = [&](int n, int y) -> float2 {
    if constexpr (C::kSharedFac) return *reinterpret_cast<const float2*>(my_fac + (n * G + y) * 8);
    else return make_float2(fac[n][0][y], fac[n][1][y]);
  };
  auto set_factor = [&](int n, int x, int y, float f) {
    if constexpr (C::kSharedFac) my_fac[(n * G + y) * 8 + x] = f;      // the same in the eight lanes of a row
    else fac[n][x][y] = f;
  };
  uint32_t s_most = 0;                         // largest scale (its bits) of group j4 that every row's factor has room for
  int t = 0, st = 0, phase = 0;                // tile of w's unit, stage and its phase
  bool ok = true;
  // One loop for the products and the units' ends: straight-line code runs once per call from a
  // cold instruction cache, which short calls feel.
#pragma unroll 1
  while (true) {
    if (t == 0) {
      int tmp;
      row_keys(a, w.s, w.r.row0, tmp, full_hi);
      row_keys(a, w.s, w.r.row0 + w.r.rows - 1, full_lo, tmp);
      s_most = 0;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          m[n][x] = kNone;
          l[n][x] = 0.f;
#pragma unroll
          for (int y = 0; y < G; ++y) {
            mt[n][x][y] = 0.f;
            set_factor(n, x, y, pow2(kMostF));
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][y][x][e] = 0.f;
          }
        }
    }
    const unsigned char* tile_k = smem + st * 2 * C::kTile;
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(b_full(st), phase, abortp, args.wait_ns));
    const int tile_key = (w.r.tile0 + w.tile + t) * kTN;
#pragma unroll(NT == 1 ? 4 : 2)
    for (int kb = 0; kb < KW / 16; ++kb) {
      const int blk = wk * KW + kb * 16, key0 = tile_key + blk;
      const unsigned char* kp = tile_k + blk * kRow;
      const unsigned char* vp = kp + C::kTile;
      const bool edge = key0 < full_lo || key0 + 15 > full_hi;
      // ---- scores
      float s[NT][4];
      {
        uint32_t sd[2][G];
        load_sides<G>(kp + soff, sd[0]);
        load_sides<G>(kp + soff + 8 * kRow, sd[1]);
        const unsigned char* own = kp + soff + 4 * (j4 & (G - 1));
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(own), w1 = *reinterpret_cast<const uint32_t*>(own + 8 * kRow);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_minima<T>(s[n], __byte_perm(w0, w0, 0x1010), __byte_perm(w1, w1, 0x1010), qm[n][0], qm[n][1]);
          if (kCentre) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] *= pow2(-18);
          }
        }
#pragma unroll
        for (int y = 0; y < G; ++y) {
          const uint32_t k0 = *reinterpret_cast<const uint32_t*>(kp + koff + 16 * y);
          const uint32_t k1 = *reinterpret_cast<const uint32_t*>(kp + koff + 8 * kRow + 16 * y);
          const float c0 = high_half<T>(sd[0][y]), c1 = high_half<T>(sd[1][y]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float d[4];
            mma_first(d, k0 & kLow, k1 & kLow, k0 & kHigh, k1 & kHigh, qf[n][y][0], qf[n][y][1]);
            mma(d, (k0 >> 8) & kLow, (k1 >> 8) & kLow, (k0 >> 8) & kHigh, (k1 >> 8) & kHigh, qf[n][y][2], qf[n][y][3]);
            s[n][0] = fmaf(c0, d[0], s[n][0]);
            s[n][1] = fmaf(c0, d[1], s[n][1]);
            s[n][2] = fmaf(c1, d[2], s[n][2]);
            s[n][3] = fmaf(c1, d[3], s[n][3]);
          }
        }
      }
      uint32_t vd[2][G];
      load_sides<G>(vp + soff, vd[0]);
      load_sides<G>(vp + soff + 8 * kRow, vd[1]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] *= kf[n][e & 1];
          if (a.softcap > 0.f) s[n][e] = softcap_log2(s[n][e], cap_log2);
        }
      if (edge) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            int lo, hi;
            row_keys(a, w.s, w.r.row0 + min(prow + n * 8 + 2 * j4 + x, w.r.rows - 1), lo, hi);
            if (key0 + r8 < lo || key0 + r8 > hi) s[n][x] = -INFINITY;
            if (key0 + r8 + 8 < lo || key0 + r8 + 8 > hi) s[n][2 + x] = -INFINITY;
          }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int key = key0 + r8 + 8 * x;
          if (key < w.r.lo || key > w.r.hi) {
#pragma unroll
            for (int y = 0; y < G; ++y) vd[x][y] = 0u;
          }
        }
      }
      // ---- running maximum and factors
      // (a lane looks at one group of its two keys, the four lanes of a key at all of them)
      const unsigned char* own = vp + soff + 4 * (j4 & (G - 1));
      uint32_t own0 = *reinterpret_cast<const uint32_t*>(own), own1 = *reinterpret_cast<const uint32_t*>(own + 8 * kRow);
      if (edge) {
        if (key0 + r8 < w.r.lo || key0 + r8 > w.r.hi) own0 = 0u;
        if (key0 + r8 + 8 < w.r.lo || key0 + r8 + 8 > w.r.hi) own1 = 0u;
      }
      bool need = (max(own0, own1) >> 16) > s_most;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) need = need || fmaxf(s[n][x], s[n][2 + x]) > m[n][x] + kRescale;
      if (__any_sync(0xffffffffu, need)) {
        int most_f[G];                         // largest exponents of the factors, of rows with a key
#pragma unroll
        for (int y = 0; y < G; ++y) most_f[y] = -126;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float mx = rows_max(fmaxf(s[n][x], s[n][2 + x]));
            const float was = m[n][x];
            if (mx > was + kRescale) m[n][x] = mx;
            const float corr = ex2_approx(was - m[n][x]);
            const float p0 = ex2_approx(s[n][x] - m[n][x]), p1 = ex2_approx(s[n][2 + x] - m[n][x]);
            l[n][x] *= corr;
#pragma unroll
            for (int y = 0; y < G; ++y) {
              mt[n][x][y] *= corr;
              // The factor brings the largest product so far to [1/2, 1).  Of those before this block the old factor tells
              // a lower bound, half its reciprocal.
              const float c0 = fabsf(high_half<T>(vd[0][y])), c1 = fabsf(high_half<T>(vd[1][y]));
              const float old = x ? factors(n, y).y : factors(n, y).x, had = corr * pow2(-log2_floor(old));
              const float top = rows_max(fmaxf(c0 < INFINITY ? p0 * c0 : 0.f, c1 < INFINITY ? p1 * c1 : 0.f));
              const int e = max(-126, min(-1 - log2_floor(fmaxf(0.5f * had, top)), kMostF));
              const float f = had * pow2(e);
              if (C::kSharedFac) __syncwarp();
              set_factor(n, x, y, pow2(e));
              if (m[n][x] > kNone) most_f[y] = max(most_f[y], e);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                o[n][y][q][x] *= f;
                o[n][y][q][2 + x] *= f;
              }
            }
          }
        int e = most_f[0];
#pragma unroll
        for (int y = 0; y < G; ++y) {
          most_f[y] = max(most_f[y], __shfl_xor_sync(0xffffffffu, most_f[y], 1));
          most_f[y] = max(most_f[y], __shfl_xor_sync(0xffffffffu, most_f[y], 2));
          if (y == 0 || (j4 & (G - 1)) == y) e = most_f[y];
        }
        if (C::kSharedFac) __syncwarp();
        e = kScaleRoom - e;                    // a scale beyond 2^e asks again
        if constexpr (std::is_same<T, __nv_bfloat16>::value) s_most = e < -126 ? 0u : (uint32_t)(min(e, 127) + 127) << 7;
        else s_most = e > 15 ? 0x7bffu : e < -126 ? 0u : (uint32_t)__half_as_ushort(__float2half_rn(pow2(e)));
      }
      // ---- weights
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = ex2_approx(s[n][e] - m[n][e & 1]);
          l[n][e & 1] += s[n][e];
        }
      // ---- values
#pragma unroll
      for (int y = 0; y < G; ++y) {
        const unsigned char* v = vp + voff + 16 * y;
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(v), w1 = *reinterpret_cast<const uint32_t*>(v + kRow);
        const uint32_t w8 = *reinterpret_cast<const uint32_t*>(v + 8 * kRow), w9 = *reinterpret_cast<const uint32_t*>(v + 9 * kRow);
        const uint32_t xa = __byte_perm(w0, w1, vsel), xb = __byte_perm(w8, w9, vsel);
        const float c0 = high_half<T>(vd[0][y]), c1 = high_half<T>(vd[1][y]);
        float m0 = low_half<T>(vd[0][y]), m1 = low_half<T>(vd[1][y]);
        if (kCentre) {
          m0 = fmaf(8.f, c0, m0);
          m1 = fmaf(8.f, c1, m1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 fr = factors(n, y);
          const f2_t f = f2_pack(fr.x, fr.y);
          float v0, v1, v2, v3;
          f2_unpack(f2_mul(f2_mul(f2_pack(s[n][0], s[n][1]), f), f2_pack(c0, c0)), v0, v1);
          f2_unpack(f2_mul(f2_mul(f2_pack(s[n][2], s[n][3]), f), f2_pack(c1, c1)), v2, v3);
          const uint32_t b0 = transposed(pack_f16x2(v0, v1)), b1 = transposed(pack_f16x2(v2, v3));
          mt[n][0][y] = fmaf(s[n][0], m0, fmaf(s[n][2], m1, mt[n][0][y]));
          mt[n][1][y] = fmaf(s[n][1], m0, fmaf(s[n][3], m1, mt[n][1][y]));
          mma(o[n][y][0], xa & kLow, xa & kHigh, xb & kLow, xb & kHigh, b0, b1);
          mma(o[n][y][1], (xa >> 8) & kLow, (xa >> 8) & kHigh, (xb >> 8) & kLow, (xb >> 8) & kHigh, b0, b1);
          if (kCentre) {
            // -8 and -128 times 2^-24
            mma(o[n][y][0], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, b0, b1);
            mma(o[n][y][1], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, b0, b1);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(b_empty(st));
    if (++st == C::kStages) { st = 0; phase ^= 1; }
    if (++t < w.take()) continue;

    // ---- end of the unit's tiles in this share; the next unit's query rows are on their way while its
    // results are joined and written
    const bool whole = w.whole();
    const int64_t slot = 2 * (int64_t)cta + (w.begins() ? 1 : 0);
    const int rows = w.r.rows, row0 = w.r.row0, t0 = w.s.t0, head0 = w.kvh * g.group;
    float* acc = reinterpret_cast<float*>(smem + C::kStages * 2 * C::kTile);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float* dst = acc + (warp * 8 * NT + n * 8 + 2 * j4 + x) * C::kPitch + 4 * r8;
#pragma unroll
        for (int y = 0; y < G; ++y) {
          const float base = rows_sum(mt[n][x][y]);
          // 2^24 (16-fold codes: 2^20) over the factor, in two steps that stay within fp32
          const int e = 24 - log2_floor(x ? factors(n, y).y : factors(n, y).x);
          const float h0 = pow2(e / 2), h1 = pow2(e - e / 2), h2 = pow2(e - e / 2 - 4);
          *reinterpret_cast<float4*>(dst + 32 * y) =
              make_float4(fmaf(o[n][y][0][x] * h0, h1, base), fmaf(o[n][y][0][2 + x] * h0, h2, base),
                          fmaf(o[n][y][1][x] * h0, h1, base), fmaf(o[n][y][1][2 + x] * h0, h2, base));
        }
        const float sum = rows_sum(l[n][x]);
        if (r8 == 0) {
          sm_m[wk][prow + n * 8 + 2 * j4 + x] = m[n][x] <= 0.5f * kNone ? -INFINITY : m[n][x];
          sm_l[wk][prow + n * 8 + 2 * j4 + x] = sum;
        }
      }
    w.next(a);
    t = 0;
    if (!w.done()) load_q();
    named_bar_sync(1, C::kProducts);
    if ((int)threadIdx.x < rows) {
      const int r = threadIdx.x;
      float M = -INFINITY, Ls = 0.f;
#pragma unroll
      for (int k = 0; k < WK; ++k) M = fmaxf(M, sm_m[k][r]);
      float f[WK];
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        // a part whose scores are no numbers has no maximum, but a sum
        f[k] = no_key(sm_m[k][r], sm_l[k][r]) ? 0.f : sm_m[k][r] == -INFINITY ? 1.f : ex2_approx(sm_m[k][r] - M);
        Ls = fmaf(f[k], sm_l[k][r], Ls);
      }
      float sc = 1.f;
      if (whole) {
        sc = row_scale<T>(a, head0 + row0 + r - group_div(g, row0 + r) * g.group, M, Ls);
      } else if (SDPA_IN_BOUNDS(slot < 2 * ctas, 593)) {
        *reinterpret_cast<float2*>(ws.ml + (slot * TM + r) * 2) = make_float2(M, Ls);
      }
#pragma unroll
      for (int k = 0; k < WK; ++k) sm_f[k][r] = f[k] * sc;
    }
    named_bar_sync(1, C::kProducts);
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (H / 4); i += C::kProducts) {
      const int r = i / (H / 4), c = (i % (H / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      // row r of the unit lies in the warps of its part
      const int part = r / (8 * NT), in = r % (8 * NT);
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const float f = sm_f[k][r];
        const float4 p = *reinterpret_cast<const float4*>(acc + ((part * WK + k) * 8 * NT + in) * C::kPitch + c);
        v.x = fmaf(f, p.x, v.x);
        v.y = fmaf(f, p.y, v.y);
        v.z = fmaf(f, p.z, v.z);
        v.w = fmaf(f, p.w, v.w);
      }
      if (whole) {
        const int pr = row0 + r, tok = group_div(g, pr), h = head0 + pr - tok * g.group;
        T* y = reinterpret_cast<T*>(const_cast<void*>(a.y.p)) + a.y.off(0, h, t0 + tok);
        T out[4] = {Elem<T>::from_f32(v.x), Elem<T>::from_f32(v.y), Elem<T>::from_f32(v.z), Elem<T>::from_f32(v.w)};
        if (SDPA_IN_BOUNDS(t0 + tok < g.tokens && h < g.Nq, 595))
          *reinterpret_cast<uint2*>(y + c) = *reinterpret_cast<const uint2*>(out);
      } else if (SDPA_IN_BOUNDS(slot < 2 * ctas, 594)) {
        *reinterpret_cast<float4*>(ws.o + (slot * TM + r) * H + c) = v;
      }
    }
    if (w.done()) break;
    named_bar_sync(1, C::kProducts);     // the buffer is written again at the next unit's end
  }
  asm volatile("bar.arrive 2, %0;" ::"n"(C::kThreads) : "memory");
}

// Rows per unit: the smallest of 8, 16 and, of 64 channels, 32 that holds all rows of a sequence with max_new
// tokens, at most the widest.  16 sequences of 2000 to 30000 keys, 8 key heads, bf16: 8 / 16 rows of 128 channels
// 79 / 132 us (400 bytes of spills at 16; two warps of eight rows each, without spills, took 188 where that took 166), 8 /
// 16 / 32 rows of 64 50 / 75 / 130.
int mma4_tm(const PagedAttn& a) {
  const int64_t rows = (int64_t)a.max_new * a.g.group;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : paged4_mma_rows(a.g.H);
}

uint64_t wait_limit_ns() {
  static const uint64_t v = [] {
    const char* e = std::getenv("SDPA_WAIT_LIMIT_NS");
    return e ? std::strtoull(e, nullptr, 10) : 4000000000ull;
  }();
  return v;
}

template <typename T, int H, int NT, int WM>
cudaError_t launch_wm(const PagedAttn& a, sdpa_dtype dt, void* wsp, cudaStream_t st) {
  using C = Cfg<H, NT, WM>;
  // 228 KB per SM, of which each CTA takes 1 KB for itself
  static_assert(C::kSmem + 3 * C::WK * C::TM * 4 + C::NW * NT * C::G * 32 + 2048 + 1024 <= 233472 / kCtasPerSm, "shared memory");
  const int ctas = paged_sms() * kCtasPerSm;
  if (ctas <= 0) return cudaErrorInvalidDevice;
  // per device: set at every call (the attribute belongs to the current context)
  cudaError_t e = cudaFuncSetAttribute(paged4_mma_kernel<T, H, NT, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  Mma4Args t{};
  t.a = a;
  t.ws = paged_ws(wsp, ctas, C::TM);
  t.wait_ns = wait_limit_ns();
  paged4_mma_kernel<T, H, NT, WM><<<(unsigned)ctas, C::kThreads, C::kSmem, st>>>(t);
  count_launch(1);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_merge(a, dt, t.ws, ctas, C::TM, st) : e;
}

template <typename T, int H>
cudaError_t launch_h(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st) {
  switch (mma4_tm(a)) {
    case 8: return launch_wm<T, H, 1, 1>(a, dt, ws, st);
    case 16: return launch_wm<T, H, 2, 1>(a, dt, ws, st);
    default: break;
  }
  if constexpr (H == 64) return launch_wm<T, H, 2, 2>(a, dt, ws, st);
  return cudaErrorInvalidValue;
}

}  // namespace

bool paged4_mma_supported(int H, int Hv, sdpa_dtype dt) { return dt != SDPA_F32 && H == Hv && (H == 64 || H == 128); }

size_t paged4_mma_workspace(int Hv) { return paged_ws_bytes(kPagedMaxSms * kCtasPerSm, 32, Hv); }

int paged4_mma_rows(int H) { return H == 128 ? 16 : 32; }

cudaError_t launch_paged4_mma(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name) {
  const bool bf = dt == SDPA_BF16;
  if (a.g.H == 128) {
    *name = bf ? "paged4_mma_bf16_h128" : "paged4_mma_f16_h128";
    return bf ? launch_h<__nv_bfloat16, 128>(a, dt, ws, st) : launch_h<__half, 128>(a, dt, ws, st);
  }
  *name = bf ? "paged4_mma_bf16_h64" : "paged4_mma_f16_h64";
  return bf ? launch_h<__nv_bfloat16, 64>(a, dt, ws, st) : launch_h<__half, 64>(a, dt, ws, st);
}

cudaError_t take_paged4_mma_status(int* status, int* timeout) {
  int v[2] = {0, 0};
  const cudaError_t e = take_words(g_paged4_words, v);
  *status = v[0];
  *timeout = v[1];
  return e;
}

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_paged4_mma)

}  // namespace sdpa
