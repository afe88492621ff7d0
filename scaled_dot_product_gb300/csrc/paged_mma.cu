// Attention over a paged cache for few rows per key (single tokens, drafted tokens) and for pages
// of any size: fp16 / bf16, H == Hv in {64, 128}.
//
// Bound by the cache's bytes: every key and value row is read once per (sequence, kv head, row
// block) whatever the number of grouped heads.  The packed rows of a unit (token x group head)
// fill the 16 rows of warp-level matrix products (m16n8k16, fp32 accumulators), which need a
// tenth of the time the bytes take; tcgen05 tiles of 128 rows would be mostly empty here and
// their scores would pass through tensor memory.  Two CTAs share an SM.  A CTA is one producer
// warp and four product warps: WM of these hold 16 rows each, the other factor WK = 4 / WM splits
// the 64 keys of a tile, each warp with its own running maximum, sum and accumulator, joined
// through shared memory at the end of a unit.
//
// The producer keeps a ring of 96 KB per CTA full across unit boundaries.  Pages of a multiple of
// 8 slots come by TMA, in boxes of gcd(page_size, 64) rows, each lane issuing one box of one
// 64-column region of K or V; other pages by 16-byte asynchronous copies, row by row through the
// page table.  (When the product warps issued the copies themselves, a third of their
// instructions went into addresses, and a single-token batch of 4.48 GB took 851 us.)  Rows of V that
// no row of the unit admits (past its keys, below every window) are set to zero before they are
// multiplied, since 0 x NaN is not 0.  Single tokens of 64 sequences, 1000 to 32000 keys, 64/8 heads of
// 128: 650 to 682 us, 6.6 to 6.9 TB/s (97 % of the measured copy rate and more); five drafted tokens of 16
// sequences 95 us, 5.4 TB/s; four short sequences 11.3 us.  The weights enter the second product rounded
// to the element type (half a step each; their sum takes them unrounded), since that product's
// operands are 16-bit (the dense decode's one row a step keeps them in fp32).  With H = 128 the tiles of
// 32 and 64 rows spill 12 and 78 bytes a thread (168 registers at two CTAs an SM).  Every wait is
// bounded: on expiry the kernel raises an abort flag, goes through its loops without waiting, lets its
// own copies finish and records SDPA_ERR_TIMEOUT.
#include <algorithm>
#include <cstdlib>
#include <type_traits>

#include "paged_sched.cuh"

namespace sdpa {

static __device__ int g_paged_words[2];      // status bits, SDPA_ERR_TIMEOUT after an expired wait

namespace {

using namespace ptx;

constexpr int kProducts = 128;       // threads of the product warps
constexpr int kThreads = kProducts + 32;
constexpr int kTN = 64;
constexpr int kCtasPerSm = 2;
constexpr int kOV = 1;                // a unit's cost beside its tiles, in tiles
constexpr int kMinShare = 3;
constexpr float kRescale = 8.f;      // log2 units a maximum may grow before o is rescaled

template <int H, int WM>
struct Cfg {
  static constexpr int WK = 4 / WM, TM = 16 * WM, KW = kTN / WK;
  static constexpr int kRegions = H / 64;                  // 64-column regions: rows of 128 bytes
  static constexpr int kRegion = kTN * 128;
  static constexpr int kTile = kRegions * kRegion;
  static constexpr int kStages = 3 * 128 / H;
  static constexpr int kSmem = kStages * 2 * kTile + 1024; // + alignment slack
  static_assert(2 * kTile == 4 * 16 * H * 4, "a stage holds the four warps' accumulators");
};

struct MmaArgs {
  PagedAttn a;
  PagedWs ws;
  int box;                           // rows per TMA box; 0: row by row
  int k_ds, k_dn, k_db, v_ds, v_dn, v_db;   // tensor-map dimension of slot / head / page
  uint64_t wait_ns;
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
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// The product warps say that they are done; the producer waits until all of them have.
__device__ __forceinline__ void ended_arrive() { asm volatile("bar.arrive 2, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void ended_sync() { named_bar_sync(2, kThreads); }

template <bool BF, int H, int WM>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    paged_mma_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                     const __grid_constant__ MmaArgs args) {
  using C = Cfg<H, WM>;
  using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
  using Wk = Walk<C::TM, kTN, kOV>;
  constexpr int WK = C::WK, TM = C::TM, KW = C::KW, NT = KW / 8;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[C::kStages], bar_empty[C::kStages];
  __shared__ float sm_m[WK][TM], sm_l[WK][TM], sm_f[WK][TM];
  __shared__ int abort_flag;
  const PagedAttn& a = args.a;
  const PagedWs& ws = args.ws;
  const Paged& g = a.g;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sb = (smem_u32(smem_raw) + 1023) & ~1023u;
  auto b_full = [&](int s) { return smem_u32(&bar_full[s]); };
  auto b_empty = [&](int s) { return smem_u32(&bar_empty[s]); };
  volatile int* abortp = &abort_flag;
  if (threadIdx.x == 0) {
    if (args.box) {
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
    }
    abort_flag = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full(s), args.box ? 1 : 32);
      mbar_init(b_empty(s), kProducts / 32);
    }
    fence_mbar_init();
  }
  const Share sh = find_share<TM, kTN, kOV, kThreads>(a, cta, ctas, kMinShare, &g_paged_words[0]);
  if (threadIdx.x == 0) {
    if (cta == 0) ws.start[ctas].b = sh.active;
    if (cta < sh.active) ws.start[cta] = sh.at;
  }
  pdl_launch_dependents();
  if (sh.count == 0) return;
  __syncthreads();
  Wk w(a, sh);
  if (w.done()) return;

  if (warp == kProducts / 32) {
    // ================================================================ producer
    int st = 0, it = 0;               // stage, turns of the ring
    bool ok = true;
    // the stage is free, or the call is being given up
    auto wait_free = [&]() {
      if (it > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(b_empty(st), (it - 1) & 1, abortp, args.wait_ns));
      return ok;
    };
    auto advance = [&]() {
      if (++st == C::kStages) { st = 0; ++it; }
    };
    if (args.box) {
      // lane: box (lane & 7), K or V (bit 3), region (bit 4)
      const bool is_v = lane & 8;
      const int row = (lane & 7) * args.box, region = lane >> 4;
      const bool mine = row < kTN && region < C::kRegions;
      const CUtensorMap* map = is_v ? &tv : &tk;
      // page of this lane's box of the t-th tile of w's unit (-1: the box is not brought)
      auto page_of = [&](int t) -> int {
        if (!mine || w.done() || t >= w.take()) return -1;
        const int key = (w.r.tile0 + w.tile + t) * kTN + row;
        if (key >= w.s.T || key + args.box <= w.r.lo) return -1;
        return g.table[(int64_t)w.b * g.table_stride + page_div(g, key)];
      };
      auto brought = [&](int t) {
        const int key = (w.r.tile0 + w.tile + t) * kTN + row;
        return mine && key < w.s.T && key + args.box > w.r.lo;
      };
      int id = page_of(0);
      while (!w.done() && wait_free()) {
        const int n = w.take();
        for (int t = 0; t < n && wait_free(); ++t) {
          const bool take = brought(t);
          const int key = (w.r.tile0 + w.tile + t) * kTN + row;
          if (take && (unsigned)id >= (unsigned)g.num_pages) {
            atomicOr(&g_paged_words[0], kPagedBadPage);
            id = g.num_pages;          // outside the map: the box is filled with zeros
          }
          const unsigned all = __ballot_sync(0xffffffffu, take);
          if (lane == 0) mbar_arrive_expect_tx(b_full(st), __popc(all) * args.box * 128);
          __syncwarp();
          if (take && SDPA_IN_BOUNDS(st < C::kStages && row + args.box <= kTN && w.kvh < g.Nkv, 531)) {
            const int slot = key - page_div(g, key) * g.page_size;
            const int ds = is_v ? args.v_ds : args.k_ds, dn = is_v ? args.v_dn : args.k_dn;
            const int c1 = ds == 1 ? slot : dn == 1 ? w.kvh : id, c2 = ds == 2 ? slot : dn == 2 ? w.kvh : id,
                      c3 = ds == 3 ? slot : dn == 3 ? w.kvh : id;
            tma_load_4d(sb + st * 2 * C::kTile + (is_v ? C::kTile : 0) + region * C::kRegion + row * 128, map, b_full(st),
                        64 * region, c1, c2, c3);
          }
          __syncwarp();
          advance();
          if (t + 1 < n) id = page_of(t + 1);      // arrives while the ring is waited for
        }
        if (!ok) break;
        w.next(a);
        id = page_of(0);
      }
    } else {
      // rows lane / 8 and on, 16-byte chunk lane % 8 of each region; the ids of 64 pages are at hand,
      // two per lane, and the next ones are fetched when a tile reaches beyond them
      const int chunk = lane & 7, row_in = lane >> 3;
      int wbase = 0, id0 = -1, id1 = -1;
      while (!w.done() && ok) {
        const int n = w.take();
        const int32_t* table = g.table + (int64_t)w.b * g.table_stride;
        const T* kb = reinterpret_cast<const T*>(g.kp.p) + g.kp.sh * w.kvh + chunk * 8;
        const T* vb = reinterpret_cast<const T*>(g.vp.p) + g.vp.sh * w.kvh + chunk * 8;
        const int end = w.r.hi >= w.r.lo ? page_div(g, w.r.hi) : -1;       // last page some row admits
        int have = -1;                 // last page at hand
        for (int t = 0; t < n; ++t) {
          const int k0 = (w.r.tile0 + w.tile + t) * kTN;
          if (end >= 0 && page_div(g, min(k0 + kTN - 1, w.r.hi)) > have) {
            wbase = page_div(g, max(k0, w.r.lo));
            have = wbase + 63;
            id0 = wbase + lane <= end ? table[wbase + lane] : -1;
            id1 = wbase + 32 + lane <= end ? table[wbase + 32 + lane] : -1;
          }
          if (!wait_free()) break;
#pragma unroll 4
          for (int p = 0; p < kTN / 4; ++p) {
            const int r = p * 4 + row_in, key = k0 + r, pg = page_div(g, key), i = pg - wbase;
            const int a0 = __shfl_sync(0xffffffffu, id0, i & 31), a1 = __shfl_sync(0xffffffffu, id1, i & 31);
            const int id = i < 32 ? a0 : a1;
            bool take = key >= w.r.lo && key <= w.r.hi;      // other keys: zeros, their pages are not read
            if (take && (unsigned)id >= (unsigned)g.num_pages) {
              atomicOr(&g_paged_words[0], kPagedBadPage);
              take = false;
            }
            take = take && SDPA_IN_BOUNDS(i >= 0 && i < 64 && key < g.cap, 532);
            const int slot = key - pg * g.page_size;
            const T* ks = kb + (take ? id * g.kp.sb + slot * g.kp.ss : 0);
            const T* vs = vb + (take ? id * g.vp.sb + slot * g.vp.ss : 0);
            const uint32_t d = sb + st * 2 * C::kTile + r * 128 + ((chunk ^ (r & 7)) << 4);
#pragma unroll
            for (int reg = 0; reg < C::kRegions; ++reg) {
              cp_async16_or_zero(d + reg * C::kRegion, ks + reg * 64, take);
              cp_async16_or_zero(d + C::kTile + reg * C::kRegion, vs + reg * 64, take);
            }
          }
          cp_async_arrive(b_full(st));
          advance();
        }
        if (ok) w.next(a);
      }
    }
    // Copies may still be on their way when a wait has expired, whichever role's it was and however
    // early the last copy was issued: the CTA, whose shared memory they write, ends behind them.
    ended_sync();
    if (*abortp) {
      constexpr uint64_t kDrainNs = 2000000000ull;
      cp_async_wait_all();
      for (int s = 0; s < C::kStages; ++s) {
        const int turns = it + (s < st ? 1 : 0);
        if (turns > 0) mbar_wait_bounded(b_full(s), (turns - 1) & 1, nullptr, kDrainNs);
      }
      if (lane == 0) atomicExch(&g_paged_words[1], (int)SDPA_ERR_TIMEOUT);
    }
    return;
  }

  // ================================================================ products
  const int wm = warp / WK, wk = warp % WK;
  uint32_t qf[H / 16][4];
  // query fragments of a unit, straight from memory: rows lane / 4 and 8 further of 16
  auto load_q = [&]() {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int pr = w.r.row0 + min(wm * 16 + (lane >> 2) + 8 * x, w.r.rows - 1);
      const int tok = group_div(g, pr);
      const uint32_t* qr = reinterpret_cast<const uint32_t*>(
          reinterpret_cast<const T*>(a.q.p) + a.q.off(0, w.kvh * g.group + pr - tok * g.group, w.s.t0 + tok));
#pragma unroll
      for (int kk = 0; kk < H / 16; ++kk) {
        qf[kk][x] = qr[kk * 8 + (lane & 3)];
        qf[kk][2 + x] = qr[kk * 8 + 4 + (lane & 3)];
      }
    }
  };
  load_q();
  const float cap_log2 = a.softcap * kLog2e, cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  const float kfac = a.softcap > 0.f ? 1.f : a.scale * kLog2e;
  // fragment addresses in a region: lane -> row and 16-byte chunk of the four 8x8 matrices of a load;
  // the chunk of a later column block is the same address with other bits flipped
  const int kr = wk * KW + ((lane >> 4) << 3) + (lane & 7);
  const uint32_t koff = kr * 128 + ((((lane >> 3) & 1) ^ (kr & 7)) << 4);
  const int vr = wk * KW + (((lane >> 3) & 1) << 3) + (lane & 7);
  const uint32_t voff = vr * 128 + (((lane >> 4) ^ (vr & 7)) << 4);
  const int prow = wm * 16 + (lane >> 2);      // this thread's rows of the unit: prow and prow + 8

  int lo[2], hi[2], full_lo = 0, full_hi = 0;  // admitted keys of the two rows, of every row
  float o[H / 8][4], m[2], l[2];
  int t = 0, st = 0, phase = 0;                // tile of w's unit, stage and its phase
  bool ok = true;
  // One loop for the products and the units' ends: straight-line code runs once per call from a
  // cold instruction cache, which short calls feel (up to 3 us a section, measured).
#pragma unroll 1
  while (true) {
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
    const uint32_t sk = sb + st * 2 * C::kTile, sv = sk + C::kTile;
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(b_full(st), phase, abortp, args.wait_ns));
    {
      const int tile_key = (w.r.tile0 + w.tile + t) * kTN, key0 = tile_key + wk * KW;
      if (args.box && (tile_key + kTN > w.r.hi + 1 || tile_key < w.r.lo)) {
        // this warp's rows of V that no row of the unit admits become zeros, brought or not
        const int first = w.r.lo - tile_key, last = w.r.hi + 1 - tile_key;
        for (int i = lane; i < KW * 8; i += 32) {
          const int r = wk * KW + (i >> 3);
          if (r < first || r >= last) {
#pragma unroll
            for (int reg = 0; reg < C::kRegions; ++reg)
              st_shared_v4(sv + reg * C::kRegion + r * 128 + (i & 7) * 16, 0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();      // before a later box is written here
        __syncwarp();
      }

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
          ldsm_x4(sk + (kk >> 2) * C::kRegion + n * 1024 + (koff ^ ((kk & 3) * 32)), b);
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
          ldsm_x4_t(sv + (n >> 3) * C::kRegion + kt * 2048 + (voff ^ ((n & 7) * 16)), b);
          mma<BF>(o[n], p, b);
          mma<BF>(o[n + 1], p, b + 2);
        }
      }
    }

    const int done_st = st;
    if (++st == C::kStages) { st = 0; phase ^= 1; }
    if (++t < w.take()) {
      __syncwarp();
      if (lane == 0) mbar_arrive(b_empty(done_st));
      continue;
    }

    // ---- end of the unit's tiles in this share; the next unit's query rows are on their way
    // while its results are joined and written.  The warps' accumulators, as they lie in registers
    // (float4 n of lane i at [warp][n][i]), go to the stage of the tile just read, which is handed
    // back to the producer afterwards.
    const bool whole = w.whole();
    const int64_t slot = 2 * (int64_t)cta + (w.begins() ? 1 : 0);
    const int rows = w.r.rows, row0 = w.r.row0, t0 = w.s.t0, head0 = w.kvh * g.group;
    w.next(a);
    t = 0;
    if (!w.done()) load_q();
    named_bar_sync(1, kProducts);    // every warp has read the tile
    float4* acc = reinterpret_cast<float4*>(smem_raw + (sk - smem_u32(smem_raw)));
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
    named_bar_sync(1, kProducts);
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
        sc = row_scale<T>(a, head0 + row0 + r - group_div(g, row0 + r) * g.group, M, L);
      } else if (SDPA_IN_BOUNDS(slot < 2 * ctas, 533)) {
        *reinterpret_cast<float2*>(ws.ml + (slot * TM + r) * 2) = make_float2(M, L);
      }
#pragma unroll
      for (int k = 0; k < WK; ++k) sm_f[k][r] = f[k] * sc;
    }
    named_bar_sync(1, kProducts);
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (H / 4); i += kProducts) {
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
        const int pr = row0 + r, tok = group_div(g, pr), h = head0 + pr - tok * g.group;
        T* y = reinterpret_cast<T*>(const_cast<void*>(a.y.p)) + a.y.off(0, h, t0 + tok);
        if (SDPA_IN_BOUNDS(t0 + tok < g.tokens && h < g.Nq, 535))
          *reinterpret_cast<uint2*>(y + c) = make_uint2(pack2<BF>(v.x, v.y), pack2<BF>(v.z, v.w));
      } else if (SDPA_IN_BOUNDS(slot < 2 * ctas, 534)) {
        *reinterpret_cast<float4*>(ws.o + (slot * TM + r) * H + c) = v;
      }
    }
    if (w.done()) break;
    fence_proxy_async_smem();        // the accumulators, before a box is written there
    __syncwarp();
    if (lane == 0) mbar_arrive(b_empty(done_st));
  }
  ended_arrive();
}

// Rows per unit: the smallest of 16, 32 and 64 that holds all rows of a sequence with max_new
// tokens, at most 64.
int mma_tm(const PagedAttn& a) {
  const int64_t rows = (int64_t)a.max_new * a.g.group;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

uint64_t wait_limit_ns() {
  static const uint64_t v = [] {
    const char* e = std::getenv("SDPA_WAIT_LIMIT_NS");
    return e ? std::strtoull(e, nullptr, 10) : 4000000000ull;
  }();
  return v;
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
  MmaArgs t{};
  t.a = a;
  t.ws = paged_ws(wsp, ctas, C::TM);
  t.wait_ns = wait_limit_ns();
  CUtensorMap tk{}, tv{};
  if (paged_boxes(a)) {
    t.box = kTN;
    while (a.g.page_size % t.box) t.box >>= 1;
    if (!paged_map(&tk, a.g, a.g.kp, H, dt, t.box, &t.k_ds, &t.k_dn, &t.k_db) ||
        !paged_map(&tv, a.g, a.g.vp, H, dt, t.box, &t.v_ds, &t.v_dn, &t.v_db))
      return cudaErrorInvalidValue;
  }
  paged_mma_kernel<BF, H, WM><<<(unsigned)ctas, kThreads, C::kSmem, st>>>(tk, tv, t);
  count_launch(1);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_merge(a, dt, t.ws, ctas, C::TM, st) : e;
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

bool paged_mma_supported(int H, int Hv, sdpa_dtype dt) { return dt != SDPA_F32 && H == Hv && (H == 64 || H == 128); }

size_t paged_mma_workspace(int Hv) { return paged_ws_bytes(kPagedMaxSms * kCtasPerSm, 64, Hv); }

cudaError_t launch_paged_mma(const PagedAttn& a, sdpa_dtype dt, void* ws, cudaStream_t st, const char** name) {
  const bool bf = dt == SDPA_BF16;
  if (a.g.H == 128) {
    *name = bf ? "paged_mma_bf16_h128" : "paged_mma_f16_h128";
    return bf ? launch_h<true, 128>(a, dt, ws, st) : launch_h<false, 128>(a, dt, ws, st);
  }
  *name = bf ? "paged_mma_bf16_h64" : "paged_mma_f16_h64";
  return bf ? launch_h<true, 64>(a, dt, ws, st) : launch_h<false, 64>(a, dt, ws, st);
}

cudaError_t take_paged_mma_status(int* status, int* timeout) {
  int v[2] = {0, 0};
  const cudaError_t e = take_words(g_paged_words, v);
  *status = v[0];
  *timeout = v[1];
  return e;
}

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_paged_mma)

}  // namespace sdpa
