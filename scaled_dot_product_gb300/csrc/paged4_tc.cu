// Attention over a paged cache of 4 bits a value for chunks of new tokens: fp16 / bf16, H == Hv in {64, 128}.
//
// Bound by the tensor cores.  A unit is 256 packed rows (token x group head) of one (sequence,
// kv head): two 128-row tiles that stream the same keys and values.  A unit of at most 128 rows (a
// single token beside chunks) has one tile of rows; there the two softmax warpgroups take turns with
// the keys, even tiles and odd ones with their own maximum, sum and accumulator, joined at its end.
// One CTA per SM walks its share (paged_sched.cuh) of all units' 128-key tiles:
//
//   warp 0        query tiles by TMA where the group divides 128
//   warp 1        tensor products (one elected lane issues): S_X = Q_X K^T, O_X += P_X V with P
//                 read from tensor memory
//   warp 3        query rows by 16-byte asynchronous copies for the other groups
//   warps 4-7     softmax of tile 0, one thread per row; warps 8-11 softmax of tile 1
//   warps 12-15   keys and values: a thread has one record of each tile, loads it a tile ahead and writes
//                 its values, rounded to the type, into the ring in the operands' layout
//
// Issue order, softmax roles, joining, abort path and teardown are those of paged_tc.cu, for a ring that warps fill instead of
// copies: what is mended in a wait or in the abort path of one has to be mended in the other.
//
// Every unit makes its operands anew from the codes, which 256 rows share. A code becomes the last bits of 1024
// (fp16) or 128 (bf16), less that number, times the scale, plus the minimum: exact up to the one rounding to
// the type, as the tensor cores' operands are 16-bit (half a step, like the keys and values of a cache in the
// type). Weights are rounded to the type too; their sum takes them unrounded. Records of keys that no row of
// the unit admits become zeros, since 0 x NaN is not 0. The softmax takes 64 columns of its scores at a time,
// which fits the registers that 16 warps leave: a running maximum is passed by at most 2^8, and where it has to
// move, the weights and products made with it are rescaled by a power of two. A chunk of 2048 tokens over 32000
// keys, 32/8 heads of 128: 870 us, 1223 TFLOP/s (64 % of the measured rate; pages in the type take 721); of 64: 720 us
// (625); softmax and record warps wait for one another (without the softmax 697; tensor pipe 45 %, issue slots
// 46 %). Every wait is bounded: on expiry the kernel raises an abort flag, lets its own copies and products finish,
// frees its tensor memory and records SDPA_ERR_TIMEOUT.
#include <algorithm>
#include <cstdlib>
#include <type_traits>

#include "paged4.h"
#include "paged_sched.cuh"
#include "prefill_tc.h"

namespace sdpa {

static __device__ int g_paged4_words[2];      // status bits, SDPA_ERR_TIMEOUT after an expired wait

namespace {

using namespace ptx;

constexpr int kBM = 128, kTM = 256, kTN = 128;
constexpr int kThreads = 512;
// A unit's cost beside its tiles (a tile costs 4, or 3 in a narrow unit), and the least cost worth a CTA: as for
// caches in the type.
constexpr int kOV = 8, kMinShare = 24;
// Register split: control, softmax and record warps; the sum stays within the launch's kThreads x
// kLaunchRegs, which the host checks.  A chunk of 2048 over 32000 keys, H = 128 / 64: 876 / 750 us; with 96, 160
// and 96 registers 905 / 743, with 120, 152 and 88 880 / 793.
constexpr int kLaunchRegs = 128, kCtlRegs = 104, kSmxRegs = 152, kRecRegs = 104;
static_assert(kCtlRegs * 128 + kSmxRegs * 256 + kRecRegs * 128 <= kLaunchRegs * kThreads, "register split");
constexpr float kRescale = 8.f;      // log2 units
constexpr float kNone = -1e30f;      // the maximum of a row that has admitted no key: finite, so that differences are numbers

template <int H>
struct Cfg {
  static constexpr int kRegions = H / 64;
  static constexpr int kRegionBytes = 128 * 128;
  static constexpr int kTile = 128 * H * 2;
  static constexpr int kKVOff = 2 * kTile;                          // two Q tiles first
  static constexpr int kYWarp = 32 * 128;                           // output staging per softmax warp
  static constexpr int kFit = (232448 - 1024 - kKVOff - 8 * kYWarp) / kTile;
  static constexpr int kStages = kFit < 10 ? kFit : 10;
  static constexpr int kYOff = kKVOff + kStages * kTile;
  static constexpr int kSmem = kYOff + 8 * kYWarp + 1024;
  // 227 KB per block, of which the barriers and the share take less than 2 KB
  static_assert(kSmem + 2048 <= 232448 && kStages >= 4, "shared memory");
  // with H = 128 P_X overwrites S_X's first columns
  static constexpr bool kAlias = H == 128;
  static constexpr int kO0 = 256, kO1 = 256 + H;
  static constexpr int kP0 = kAlias ? 0 : 256 + 2 * H, kP1 = kAlias ? 128 : kP0 + 64;
};

struct TcArgs {
  PagedAttn a;
  PagedWs ws;
  float scale_log2, cap_in, cap_log2;
  int q_tma;                         // query rows by TMA: boxes of one group's heads x 128 / group tokens
  int pre;                           // scale <= 0: scores are scaled before the maximum
  uint64_t wait_ns;
};

// Admitted keys [lo, hi] among the 32 from key on, as bits.
__device__ __forceinline__ uint32_t key_bits(int key, int lo, int hi) {
  const int a = max(lo - key, 0), b = min(hi - key, 31);
  const uint32_t up = 0xffffffffu >> (31 - max(b, 0));
  return a <= b ? up & (0xffffffffu << min(a, 31)) : 0u;
}

// 32 lanes x 8 columns, for the seldom paths: few registers.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}

// Two weights times a power of two, in fp32: in fp16 the factor itself may lie below the type's range while the
// products do not.
template <typename T>
__device__ __forceinline__ uint32_t times2(uint32_t w, float f) {
  const T* e = reinterpret_cast<const T*>(&w);
  const float a = Elem<T>::to_f32(e[0]) * f, b = Elem<T>::to_f32(e[1]) * f;
  return std::is_same<T, __half>::value ? pack_f16x2(a, b) : pack_bf16x2(a, b);
}

// A word's eight codes as four pairs of values, minimum + scale * code rounded once.
template <typename T>
__device__ __forceinline__ void values_of(uint32_t w, uint32_t m2, uint32_t s2, uint32_t* v) {
  using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
  // the type's number whose last bits count ones: 1024, 128
  constexpr uint32_t kBase = std::is_same<T, __half>::value ? 0x64006400u : 0x43004300u;
  const uint32_t base = kBase, high = w >> 4;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t x = (__byte_perm(w, high, (b | b << 4) | (4 + b) << 8 | (4 + b) << 12) & 0x000f000fu) | kBase;
    const T2 code = __hsub2(*reinterpret_cast<const T2*>(&x), *reinterpret_cast<const T2*>(&base));
    const T2 y = __hfma2(code, *reinterpret_cast<const T2*>(&s2), *reinterpret_cast<const T2*>(&m2));
    v[b] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// Ring positions, from the unit's first, of the key and value tiles of a unit of n: in the order of
// their first use.  With P in S's columns PV(j) comes before S(j + 1): K_0 V_0 K_1 V_1 ...; else S runs a
// tile ahead: K_0 K_1 V_0 K_2 V_1 ... V_{n-1}.
template <bool kAlias>
__device__ __forceinline__ int k_at(int j) { return kAlias ? 2 * j : j == 0 ? 0 : 2 * j - 1; }
template <bool kAlias>
__device__ __forceinline__ int v_at(int j, int n) { return kAlias ? 2 * j + 1 : j + 1 < n ? 2 * j + 2 : 2 * n - 1; }

template <int H, bool BF, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    paged4_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ TcArgs t) {
  using C = Cfg<H>;
  using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
  using Wk = Walk<kTM, kTN, kOV>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bar_full[C::kStages], bar_empty[C::kStages];
  __shared__ __align__(8) uint64_t bar_qready, bar_qempty, bar_drain, bar_sfull[2], bar_sfree[2], bar_pfull[2], bar_odone[2];
  __shared__ __align__(8) uint64_t bar_xfull[4], bar_xfree[4];      // joining the halves of a narrow unit
  __shared__ float2 sm_ml[4][32];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_flag;
  __shared__ int issued_q;                   // units whose query tiles came by TMA
  const PagedAttn& a = t.a;
  const Paged& g = a.g;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sQ = smem_u32(smem), sKV = sQ + C::kKVOff;
  auto b_full = [&](int s) { return smem_u32(&bar_full[s]); };
  auto b_empty = [&](int s) { return smem_u32(&bar_empty[s]); };
  auto b_sfull = [&](int x) { return smem_u32(&bar_sfull[x]); };
  auto b_sfree = [&](int x) { return smem_u32(&bar_sfree[x]); };
  auto b_pfull = [&](int x) { return smem_u32(&bar_pfull[x]); };
  auto b_odone = [&](int x) { return smem_u32(&bar_odone[x]); };
  const uint32_t b_qready = smem_u32(&bar_qready), b_qempty = smem_u32(&bar_qempty), b_drain = smem_u32(&bar_drain);
  volatile int* abortp = &abort_flag;
  constexpr uint64_t kDrainNs = 2000000000ull;

  if (threadIdx.x == 0) {
    if (t.q_tma) prefetch_tmap(&tq);
    abort_flag = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full(s), 4);
      mbar_init(b_empty(s), 1);
    }
    issued_q = 0;
    mbar_init(b_qready, 1);
    mbar_init(b_qempty, 1);
    mbar_init(b_drain, 1);
    for (int x = 0; x < 4; ++x) { mbar_init(smem_u32(&bar_xfull[x]), 32); mbar_init(smem_u32(&bar_xfree[x]), 32); }
    for (int x = 0; x < 2; ++x) {
      mbar_init(b_sfull(x), 1);
      mbar_init(b_sfree(x), kBM);
      mbar_init(b_pfull(x), kBM);
      mbar_init(b_odone(x), 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_sh), 512);
    tmem_relinquish();
  }
  const Share sh = find_share<kTM, kTN, kOV, kThreads>(a, cta, ctas, kMinShare, &g_paged4_words[0]);
  if (threadIdx.x == 0) {
    if (cta == 0) t.ws.start[ctas].b = sh.active;
    if (cta < sh.active) t.ws.start[cta] = sh.at;
  }
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abortp, t.wait_ns));
  };
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));

  if (warp == 0) {
    // ================================================================ query tiles by TMA
    int it = 0;
    bool ok = true;
    for (Wk w(a, sh); ok && t.q_tma && !w.done(); w.next(a)) {
      // the previous unit's last S products have read its query tiles; rows of the box behind the
      // unit's belong to other rows and go nowhere
      if (it > 0 && !(ok = wait_all(b_qempty, (it - 1) & 1))) break;
      const int nx = w.r.rows > kBM ? 2 : 1;
      if (lane == 0) {
        mbar_arrive_expect_tx(b_qready, nx * C::kTile);
        for (int x = 0; x < nx; ++x)
          for (int r = 0; r < C::kRegions; ++r)
            tma_load_4d(sQ + x * C::kTile + r * C::kRegionBytes, &tq, b_qready, 64 * r, w.kvh * g.group,
                        w.s.t0 + group_div(g, w.r.row0 + x * kBM), 0);
      }
      ++it;
      if (lane == 0) issued_q = it;
      __syncwarp();
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ================================================================ keys and values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRecRegs));
    constexpr int kRow = q4_row_bytes(H, 2), kVecs = kRow / 8, G = H / kQ4Group;
    const int row = threadIdx.x - 384;               // this thread's key of a tile
    int base = 0;                                    // ring position of the unit's first tile
    bool ok = true;
    for (Wk w(a, sh); ok && !w.done(); w.next(a)) {
      const int n = w.take(), kt0 = w.r.tile0 + w.tile;
      const int32_t* table = g.table + (int64_t)w.b * g.table_stride;
      auto admitted = [&](int j) {
        const int key = (kt0 + j) * kTN + row;
        return j < n && key >= w.r.lo && key <= w.r.hi;
      };
      auto look_up = [&](int j) { return admitted(j) ? table[page_div(g, (kt0 + j) * kTN + row)] : -1; };
      // the record of tile j, or zeros
      auto load = [&](bool is_v, int j, int id, uint32_t (&rec)[2 * kVecs]) {
        bool take = admitted(j);
        if (take && (unsigned)id >= (unsigned)g.num_pages) {
          atomicOr(&g_paged4_words[0], kPagedBadPage);
          take = false;
        }
        const int key = (kt0 + j) * kTN + row;
        if (take && SDPA_IN_BOUNDS(key < g.cap && w.kvh < g.Nkv, 601)) {
          const View& v = is_v ? g.vp : g.kp;
          const unsigned char* p = reinterpret_cast<const unsigned char*>(v.p) + v.off(id, w.kvh, key - page_div(g, key) * g.page_size);
          if constexpr (kRow % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kVecs / 2; ++i) {
              const uint4 x = __ldg(reinterpret_cast<const uint4*>(p) + i);
              rec[4 * i] = x.x;
              rec[4 * i + 1] = x.y;
              rec[4 * i + 2] = x.z;
              rec[4 * i + 3] = x.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
              const uint2 x = __ldg(reinterpret_cast<const uint2*>(p) + i);
              rec[2 * i] = x.x;
              rec[2 * i + 1] = x.y;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2 * kVecs; ++i) rec[i] = 0u;
        }
      };
      auto write = [&](int st, const uint32_t (&word)[2 * kVecs]) {
        const uint32_t dst = sKV + st * C::kTile + row * 128;
#pragma unroll
        for (int y = 0; y < G; ++y) {
          const uint32_t side = word[H / 8 + y];
          const uint32_t m2 = __byte_perm(side, side, 0x1010), s2 = __byte_perm(side, side, 0x3232);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[4];
            values_of<T>(word[y * 4 + c], m2, s2, v);
            const int chunk = y * 4 + c;             // eight channels
            st_shared_v4(dst + (chunk >> 3) * C::kRegionBytes + (((chunk & 7) ^ (row & 7)) << 4), v[0], v[1], v[2], v[3]);
          }
        }
      };
      auto put = [&](int sq, const uint32_t (&rec)[2 * kVecs]) -> bool {
        const int st = sq % C::kStages;
        if (sq >= C::kStages && !wait_all(b_empty(st), ((sq / C::kStages) - 1) & 1)) return false;
        write(st, rec);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_full(st));
        return true;
      };
      // in the ring's order: K_0, then V_j before or behind K_{j+1}; records are loaded one ahead, ids two tiles
      uint32_t rk[2 * kVecs], rv[2 * kVecs];
      int id = look_up(0), next = look_up(1);
      load(false, 0, id, rk);
      load(true, 0, id, rv);
      if (!(ok = put(base + k_at<C::kAlias>(0), rk))) break;
      for (int j = 0; j < n; ++j) {
        id = next;
        if (j + 1 < n) load(false, j + 1, id, rk);
        next = look_up(j + 2);
        if constexpr (C::kAlias) {
          if (!(ok = put(base + v_at<true>(j, n), rv))) break;
          if (j + 1 < n) {
            load(true, j + 1, id, rv);
            if (!(ok = put(base + k_at<true>(j + 1), rk))) break;
          }
        } else {
          if (j + 1 < n && !(ok = put(base + k_at<false>(j + 1), rk))) break;
          if (!(ok = put(base + v_at<false>(j, n), rv))) break;
          if (j + 1 < n) load(true, j + 1, id, rv);
        }
      }
      base += 2 * n;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================================================ tensor products
    const uint32_t leader = elect_one();
    auto commit = [&](uint32_t bar) {
      if (leader) mma_commit(bar);
    };
    constexpr uint32_t kIdQK = idesc_f16(BF, kBM, kTN, false);
    constexpr uint32_t kIdPV = idesc_f16(BF, kBM, H, true);
    const uint32_t tO[2] = {tmem + C::kO0, tmem + C::kO1}, tP[2] = {tmem + C::kP0, tmem + C::kP1};
    const uint64_t dQ0 = desc_sw128(sQ, 16, 1024), dK0 = desc_sw128(sKV, 16, 1024);
    const uint64_t dV0 = desc_sw128(sKV, C::kRegionBytes, 1024);
    int seq = 0, it = 0;
    int ns[2] = {0, 0}, np[2] = {0, 0};      // S issued, P consumed, per tile
    auto wait_full = [&]() -> bool {
      const bool ok = wait_all(b_full(seq % C::kStages), (seq / C::kStages) & 1);
      tc_fence_after();
      return ok;
    };
    // scores x of query tile q
    auto issue_S = [&](int x, int q, int st) {
      const uint64_t dq = dQ0 + (uint64_t)((q * C::kTile) >> 4), dk = dK0 + (uint64_t)((st * C::kTile) >> 4);
#pragma unroll
      for (int kk = 0; kk < H / 16; ++kk) {
        const uint64_t off = (uint64_t)(((kk / 4) * C::kRegionBytes + (kk % 4) * 32) >> 4);
        if (leader) mma_f16_ss(tmem + 128 * x, dq + off, dk + off, kIdQK, kk > 0);
      }
    };
    auto issue_PV = [&](int x, int st, bool acc) {
      const uint64_t dv = dV0 + (uint64_t)((st * C::kTile) >> 4);
#pragma unroll
      for (int kk = 0; kk < kTN / 16; ++kk)
        if (leader) mma_f16_ts(tO[x], tP[x] + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), kIdPV, (acc || kk > 0) ? 1u : 0u);
    };
    auto wait_sfree = [&](int x) -> bool {
      if (C::kAlias || ns[x] == 0) return true;
      const bool ok = wait_all(b_sfree(x), (ns[x] - 1) & 1);
      tc_fence_after();
      return ok;
    };
    bool ok = true;
    for (Wk w(a, sh); ok && !w.done(); w.next(a)) {
      const int n = w.take(), nx = w.r.rows > kBM ? 2 : 1;
      if (!(ok = wait_all(b_qready, it & 1))) break;
      tc_fence_after();
      ++it;
      if (nx == 1) {
        // key tile j belongs to softmax group j & 1; S of the next tile runs before PV of this one
        const int base = seq;
        auto wait_at = [&](int sq) -> bool {
          const bool ready = wait_all(b_full(sq % C::kStages), (sq / C::kStages) & 1);
          tc_fence_after();
          return ready;
        };
        auto scores = [&](int j) -> bool {
          const int y = j & 1, st = (base + k_at<C::kAlias>(j)) % C::kStages;
          if (!wait_at(base + k_at<C::kAlias>(j)) || !wait_sfree(y)) return false;
          issue_S(y, 0, st);
          commit(b_sfull(y));
          ++ns[y];
          if (j + 1 == n) commit(b_qempty);
          commit(b_empty(st));
          return true;
        };
        ok = scores(0);
        for (int j = 0; j < n && ok; ++j) {
          const int x = j & 1, vst = (base + v_at<C::kAlias>(j, n)) % C::kStages;
          if (j + 1 < n && !(ok = scores(j + 1))) break;
          if (!(ok = wait_at(base + v_at<C::kAlias>(j, n)))) break;
          if (!(ok = wait_all(b_pfull(x), np[x] & 1))) break;
          tc_fence_after();
          ++np[x];
          issue_PV(x, vst, j > 1);
          if (!C::kAlias || j + 2 >= n) commit(b_odone(x));
          commit(b_empty(vst));
        }
        seq = base + 2 * n;
        continue;
      }
      if (!(ok = wait_full())) break;
      {
        const int st = seq % C::kStages;
        for (int x = 0; x < nx && ok; ++x) {
          if (!(ok = wait_sfree(x))) break;
          issue_S(x, x, st);
          commit(b_sfull(x));
          ++ns[x];
        }
        if (!ok) break;
        if (n == 1) commit(b_qempty);
        commit(b_empty(st));
        ++seq;
      }
      for (int j = 0; j < n && ok; ++j) {
        const bool more = j + 1 < n;
        if constexpr (C::kAlias) {
          // P_X(j) lives in S_X's columns: PV_X(j) first, then S_X(j+1), whose sfull also says
          // that PV_X(j) is done; the unit's last PV_X completes on odone_X
          const int vst = seq % C::kStages;
          if (!(ok = wait_full())) break;
          ++seq;
          const int kst = seq % C::kStages;
          for (int x = 0; x < nx && ok; ++x) {
            if (!(ok = wait_all(b_pfull(x), np[x] & 1))) break;
            tc_fence_after();
            ++np[x];
            issue_PV(x, vst, j > 0);
            if (more) {
              if (x == 0 && !(ok = wait_full())) break;
              issue_S(x, x, kst);
              commit(b_sfull(x));
              ++ns[x];
            } else {
              commit(b_odone(x));
            }
          }
          if (!ok) break;
          if (more && j + 2 == n) commit(b_qempty);
          commit(b_empty(vst));
          if (more) {
            commit(b_empty(kst));
            ++seq;
          }
        } else {
          if (more) {
            const int kst = seq % C::kStages;
            if (!(ok = wait_full())) break;
            ++seq;
            for (int x = 0; x < nx && ok; ++x) {
              if (!(ok = wait_sfree(x))) break;
              issue_S(x, x, kst);
              commit(b_sfull(x));
              ++ns[x];
            }
            if (!ok) break;
            if (j + 2 == n) commit(b_qempty);
            commit(b_empty(kst));
          }
          const int vst = seq % C::kStages;
          if (!(ok = wait_full())) break;
          ++seq;
          for (int x = 0; x < nx && ok; ++x) {
            if (!(ok = wait_all(b_pfull(x), np[x] & 1))) break;
            tc_fence_after();
            ++np[x];
            issue_PV(x, vst, j > 0);
            commit(b_odone(x));
          }
          if (!ok) break;
          commit(b_empty(vst));
        }
      }
    }
    // every product this thread issued completes before the CTA frees its tensor memory
    commit(b_drain);
    mbar_wait_bounded(b_drain, 0, nullptr, kDrainNs);
    __syncwarp();
  } else if (warp == 3) {
    // ================================================================ query rows of groups that TMA does not box
    constexpr int CPR = H / 8;                       // 16-byte chunks of a row
    const int chunk = lane % CPR, rin = lane / CPR;
    int it = 0;
    bool ok = true;
    for (Wk w(a, sh); ok && !t.q_tma && !w.done(); w.next(a)) {
      if (it > 0 && !(ok = wait_all(b_qempty, (it - 1) & 1))) break;
      ++it;
      const int rows = w.r.rows > kBM ? 2 * kBM : kBM;
#pragma unroll 4
      for (int r0 = 0; r0 < rows; r0 += 32 / CPR) {
        const int r = r0 + rin, x = r / kBM, xr = r % kBM;
        const bool take = r < w.r.rows;
        const int pr = w.r.row0 + (take ? r : 0), tok = group_div(g, pr);
        const T* src = reinterpret_cast<const T*>(a.q.p) + a.q.off(0, w.kvh * g.group + pr - tok * g.group, w.s.t0 + tok) +
                       chunk * 8;
        const uint32_t d = sQ + x * C::kTile + (chunk >> 3) * C::kRegionBytes + xr * 128 + (((chunk & 7) ^ (xr & 7)) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src),
                     "r"(take && SDPA_IN_BOUNDS(w.s.t0 + tok < g.tokens, 602) ? 16 : 0) : "memory");
      }
      cp_async_commit();
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_qready);
    }
  } else if (warp >= 4) {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSmxRegs));
    const int x = (warp - 4) >> 2, sub = warp & 3;
    const int row = sub * 32 + lane;                 // row of the tile == tensor-memory lane
    const uint32_t trow = tmem + ((uint32_t)(sub * 32) << 16);
    const uint32_t tS = trow + 128 * x, tO = trow + (x ? C::kO1 : C::kO0), tP = trow + (x ? C::kP1 : C::kP0);
    const uint32_t sY = sQ + C::kYOff + (uint32_t)(x * 4 + sub) * C::kYWarp;
    const float fac = CAP ? t.cap_in : t.scale_log2;      // of the scores, or of the cap's argument
    const float kfac = CAP || t.pre ? 1.f : fac;
    int cs = 0, co = 0, xc = 0;                      // sfull / odone / joining phases waited
    bool ok = true;
    for (Wk w(a, sh); ok && !w.done(); w.next(a)) {
      const int n = w.take(), kt0 = w.r.tile0 + w.tile;
      const bool narrow = w.r.rows <= kBM;           // both groups have the rows, and every second tile
      const int j0 = narrow ? x : 0, js = narrow ? 2 : 1, tile_row = narrow ? 0 : x * kBM;
      if (j0 >= n) continue;
      const bool valid = tile_row + row < w.r.rows;
      const int pr = w.r.row0 + (valid ? tile_row + row : 0);
      // rows past the unit's: every key, so that they cause no masking; their results go nowhere
      int lo = 0, hi = 0x7fffffff;
      if (valid) row_keys(a, w.s, pr, lo, hi);
      if (tile_row + sub * 32 >= w.r.rows) {
        // no row of this warp: it keeps the barriers' counts, at the pace of the other warps
        for (int j = j0; j < n && ok; j += js) {
          if (!(ok = wait_all(b_sfull(x), cs & 1))) break;
          ++cs;
          if constexpr (!C::kAlias) {
            mbar_arrive(b_sfree(x));
            if (j != j0) {
              if (!(ok = wait_all(b_odone(x), co & 1))) break;
              ++co;
            }
          }
          mbar_arrive(b_pfull(x));
        }
        if (!ok || !(ok = wait_all(b_odone(x), co & 1))) break;
        ++co;
        continue;
      }
      float m = kNone, l = 0.f;
      for (int j = j0; j < n; j += js) {
        if (!(ok = wait_all(b_sfull(x), cs & 1))) break;
        ++cs;
        tc_fence_after();
        const int key0 = (kt0 + j) * kTN;
        // one answer for the warp: the loads from tensor memory below are the whole warp's
        const bool edge = __any_sync(0xffffffffu, !(lo <= key0 && key0 + kTN - 1 <= hi));
        // ---- 64 columns at a time (32 took 1578 us where these take 876: each step waits for its scores and
        // for the warp's vote; all 128 at once 995).  The weights refer to the maximum so far; columns that pass it by
        // more than 2^8 move it, and what has been made with the old one is rescaled.
        float sum = 0.f;
        bool free_p = C::kAlias || j == j0;          // P_X has been read, O_X holds the product
        // the previous PV_X has read P_X and O_X holds it (with P in S's columns, sfull said so)
        auto wait_p = [&]() {
          if (free_p || !ok) return;
          ok = wait_all(b_odone(x), co & 1);
          ++co;
          tc_fence_after();
          free_p = true;
        };
        constexpr int kCols = 64;
#pragma unroll
        for (int c = 0; c < kTN / kCols; ++c) {
          uint32_t pw[32];
          float z[kCols];
          {
            uint32_t u[kCols];
            tmem_ld32(tS + c * kCols, u);
            tmem_ld32(tS + c * kCols + 32, u + 32);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < kCols; ++e) z[e] = __uint_as_float(u[e]);
          }
          if constexpr (!C::kAlias) {
            if (c == 1) {
              tc_fence_before();
              mbar_arrive(b_sfree(x));
            }
          }
          if constexpr (CAP) {
            // cap tanh(u) in log2 units: 1 - 2 / (e^2u + 1), absolute error about 2^-23 of the cap
            const float c2 = 2.f * kLog2e * fac;
#pragma unroll
            for (int e = 0; e < kCols; ++e) z[e] = t.cap_log2 * (1.f - __fdividef(2.f, ex2_approx(z[e] * c2) + 1.f));
          } else if (t.pre) {
#pragma unroll
            for (int e = 0; e < kCols; ++e) z[e] *= fac;
          }
          if (edge) {
            const uint32_t b0 = key_bits(key0 + c * kCols, lo, hi), b1 = key_bits(key0 + c * kCols + 32, lo, hi);
#pragma unroll
            for (int e = 0; e < kCols; ++e) z[e] = ((e < 32 ? b0 : b1) >> (e & 31)) & 1u ? z[e] : -INFINITY;
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kCols; e += 2) top[(e >> 1) & 3] = fmax3(top[(e >> 1) & 3], z[e], z[e + 1]);
          const float mx = fmaxf(fmax3(top[0], top[1], top[2]), top[3]) * kfac;
          const bool need = mx > m + kRescale;       // true for a row's first keys
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = need ? ceilf(mx) : m;
            const float corr = ex2_approx(m - m_new);      // a power of two: rescaled weights keep their bits
            m = m_new;
            l *= corr;
            sum *= corr;
            if (c == 1) {
              tmem_st_wait();
#pragma unroll 1
              for (int i = 0; i < 4; ++i) {
                uint32_t o[8];
                tmem_ld8(tP + i * 8, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = times2<T>(o[e], corr);
                tmem_st8(tP + i * 8, o);
              }
            }
            if (j != j0) {
              wait_p();
              if (ok) {
#pragma unroll 1
                for (int i = 0; i < H / 8; ++i) {
                  uint32_t o[8];
                  tmem_ld8(tO + i * 8, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                  tmem_st8(tO + i * 8, o);
                }
                tmem_st_wait();
              }
            }
          }
          f2_t part[2] = {f2_zero(), f2_zero()};
          const f2_t kf2 = f2_pack(kfac, kfac), nm2 = f2_pack(-m, -m);
#pragma unroll
          for (int e = 0; e < kCols; e += 2) {
            float z0, z1;
            f2_unpack(f2_fma(f2_pack(z[e], z[e + 1]), kf2, nm2), z0, z1);
            const float p0 = ex2_approx(z0), p1 = ex2_approx(z1);
            part[(e >> 1) & 1] = f2_add(part[(e >> 1) & 1], f2_pack(p0, p1));
            pw[e >> 1] = BF ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
          }
          {
            float r0, r1;
            f2_unpack(f2_add(part[0], part[1]), r0, r1);
            sum += r0 + r1;
          }
          wait_p();
          if (!ok) break;
          tmem_st32(tP + c * 32, pw);
        }
        if (!ok) break;
        l += sum;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(b_pfull(x));
      }
      if (!ok) break;

      // ---- the unit's rows, or their partial results
      if (m <= 0.5f * kNone) m = -INFINITY;
      if (!(ok = wait_all(b_odone(x), co & 1))) break;
      ++co;
      tc_fence_after();
      // a narrow unit's odd tiles: group 1 hands its rows to group 0, 32 columns at a time, through its
      // staging (float4 q of lane i at [q][i])
      const bool join = narrow && n > 1;
      const uint32_t sX = sQ + C::kYOff + (uint32_t)(4 + sub) * C::kYWarp;
      const uint32_t b_xfull = smem_u32(&bar_xfull[sub]), b_xfree = smem_u32(&bar_xfree[sub]);
      if (join && x == 1) {
        sm_ml[sub][lane] = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; c < H / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 8; ++q) st_shared_v4(sX + q * 512 + lane * 16, o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          mbar_arrive(b_xfull);
          if (!(ok = wait_all(b_xfree, xc & 1))) break;
          ++xc;
        }
        if (!ok) break;
        continue;
      }
      float f0 = 1.f, f1 = 0.f;
      // columns 32 c and on of this thread's row
      auto read_o = [&](int c, uint32_t* o) {
        tmem_ld32(tO + c * 32, o);
        tmem_ld_wait();
        if (!join) return;
        ok = ok && wait_all(b_xfull, xc & 1);
        if (c == 0) {
          const float2 other = sm_ml[sub][lane];
          const float M = fmaxf(m, other.x);
          if (M != -INFINITY) {
            f0 = ex2_approx(m - M);
            f1 = ex2_approx(other.x - M);
          }
          l = l * f0 + other.y * f1;
          m = M;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t v[4];
          ld_shared_v4(sX + q * 512 + lane * 16, v[0], v[1], v[2], v[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[4 * q + e] = __float_as_uint(fmaf(__uint_as_float(o[4 * q + e]), f0, __uint_as_float(v[e]) * f1));
        }
        mbar_arrive(b_xfree);
        ++xc;
      };
      const bool whole = w.whole();
      const int live = min(32, w.r.rows - tile_row - sub * 32);       // rows of this warp
      if (whole) {
        const int tok = group_div(g, pr), h = w.kvh * g.group + pr - tok * g.group;
        float inv = 0.f;
        const long long yrow = (long long)(reinterpret_cast<uintptr_t>(a.y.p) + (uintptr_t)(a.y.off(0, h, w.s.t0 + tok) * 2));
#pragma unroll 1
        for (int c = 0; c < H / 32; ++c) {
          uint32_t o[32];
          read_o(c, o);
          if (c == 0) inv = row_scale<T>(a, h, m, l);      // m and l are the whole row's now
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t wv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v0 = __uint_as_float(o[q * 8 + 2 * e]) * inv, v1 = __uint_as_float(o[q * 8 + 2 * e + 1]) * inv;
              wv[e] = BF ? pack_bf16x2(v0, v1) : pack_f16x2(v0, v1);
            }
            const int c16 = (c & 1) * 4 + q;
            st_shared_v4(sY + lane * 128 + ((c16 ^ (lane & 7)) << 4), wv[0], wv[1], wv[2], wv[3]);
          }
          if (c & 1) {
            // 64 columns of 32 rows are staged: eight lanes store 128 bytes of a row
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = i * 4 + (lane >> 3), c16 = lane & 7;
              const long long dst = __shfl_sync(0xffffffffu, yrow, rr);
              uint4 v;
              ld_shared_v4(sY + rr * 128 + ((c16 ^ (rr & 7)) << 4), v.x, v.y, v.z, v.w);
              if (rr < live && SDPA_IN_BOUNDS(w.s.t0 + w.s.n <= g.tokens, 603))
                *reinterpret_cast<uint4*>((uintptr_t)dst + (c >> 1) * 128 + c16 * 16) = v;
            }
            __syncwarp();
          }
        }
      } else {
        const int64_t base = (2 * (int64_t)cta + (w.begins() ? 1 : 0)) * kTM + tile_row + sub * 32;
#pragma unroll 1
        for (int c = 0; c < H / 32; ++c) {
          uint32_t o[32];
          read_o(c, o);
          if (c == 0 && lane < live && SDPA_IN_BOUNDS(base + lane < (int64_t)2 * ctas * kTM, 604)) {
            t.ws.ml[(base + lane) * 2] = m;
            t.ws.ml[(base + lane) * 2 + 1] = l;
          }
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_shared_v4(sY + lane * 128 + ((q ^ (lane & 7)) << 4), o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = i * 4 + (lane >> 3), q = lane & 7;
            uint4 v;
            ld_shared_v4(sY + rr * 128 + ((q ^ (rr & 7)) << 4), v.x, v.y, v.z, v.w);
            if (rr < live && SDPA_IN_BOUNDS(base + rr < (int64_t)2 * ctas * kTM, 605))
              *reinterpret_cast<uint4*>(t.ws.o + (base + rr) * H + c * 32 + q * 4) = v;
          }
          __syncwarp();
        }
      }
      // these tensor-memory reads are complete before this thread's next P store, which the MMA
      // warp waits for before the next unit's first PV overwrites O
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && abort_flag) {
    // Some role gave up, perhaps behind the last copy of query tiles: it lands before the CTA, whose
    // shared memory it writes, ends.  Earlier ones landed before their space was filled again.
    if (issued_q > 0) mbar_wait_bounded(b_qready, (issued_q - 1) & 1, nullptr, kDrainNs);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && abort_flag) atomicExch(&g_paged4_words[1], (int)SDPA_ERR_TIMEOUT);
}

// ---------------------------------------------------------------- host side

uint64_t wait_limit_ns() {
  static const uint64_t v = [] {
    const char* e = std::getenv("SDPA_WAIT_LIMIT_NS");
    return e ? std::strtoull(e, nullptr, 10) : 4000000000ull;
  }();
  return v;
}

template <int H, bool BF, bool CAP>
cudaError_t launch_cap(const CUtensorMap& tq, const TcArgs& t, int ctas, cudaStream_t st) {
  using C = Cfg<H>;
  auto* kernel = paged4_tc_kernel<H, BF, CAP>;
  // per device: set at every call (the attribute belongs to the current context)
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  cudaFuncAttributes fa{};
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
  // with fewer registers at launch the softmax warps' request could never be met
  if (e == cudaSuccess && fa.numRegs < kLaunchRegs) e = cudaErrorLaunchOutOfResources;
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)ctas, kThreads, C::kSmem, st>>>(tq, t);
  count_launch(1);
  return cudaGetLastError();
}

template <int H>
cudaError_t launch_h(bool bf, bool cap, const CUtensorMap& tq, const TcArgs& t, int ctas, cudaStream_t st) {
  if (bf) return cap ? launch_cap<H, true, true>(tq, t, ctas, st) : launch_cap<H, true, false>(tq, t, ctas, st);
  return cap ? launch_cap<H, false, true>(tq, t, ctas, st) : launch_cap<H, false, false>(tq, t, ctas, st);
}

}  // namespace

// More rows of a sequence than the widest unit of the warp-level products holds: 16 of 128 channels, 32 of 64.  16
// sequences of 2000 to 30000 keys, 8 key heads of 128 / 64: up to 128 rows 227 / 208 us here; 16 rows 132 / 75, 32 rows 279 /
// 130, 64 rows 493 / 248 there (64 rows, and 32 of 128, before each row and group had a factor of its own).
bool paged4_tc_supported(const PagedAttn& a, sdpa_dtype dt) {
  return paged4_mma_supported(a.g.H, a.g.Hv, dt) && (int64_t)a.max_new * a.g.group > paged4_mma_rows(a.g.H);
}

size_t paged4_tc_workspace(int Hv) { return paged_ws_bytes(kPagedMaxSms, kTM, Hv); }

cudaError_t launch_paged4_tc(const PagedAttn& a, sdpa_dtype dt, void* wsp, cudaStream_t st, const char** name) {
  const int ctas = paged_sms();
  if (ctas <= 0) return cudaErrorInvalidDevice;
  TcArgs t{};
  t.a = a;
  t.ws = paged_ws(wsp, ctas, kTM);
  t.scale_log2 = a.scale * kLog2e;
  t.pre = !(a.scale > 0.f);
  t.cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  t.cap_log2 = a.softcap * kLog2e;
  t.wait_ns = wait_limit_ns();
  const bool bf = dt == SDPA_BF16, cap = a.softcap > 0.f;
  CUtensorMap tq{};
  if (kBM % a.g.group == 0 && a.q.sh <= a.q.ss && a.q.ss < ((int64_t)1 << 38)) {
    // (D, head, token): a box is 64 columns x one group's heads x 128 / group tokens, so its rows lie
    // in packed order
    const cuuint64_t dims[4] = {(cuuint64_t)a.g.H, (cuuint64_t)a.g.Nq, (cuuint64_t)a.g.tokens, 1};
    const int64_t sh = a.g.Nq > 1 ? a.q.sh : a.g.H, ss = a.g.tokens > 1 ? a.q.ss : std::max<int64_t>(a.q.ss, sh * a.g.Nq);
    const cuuint64_t strides[3] = {(cuuint64_t)sh * 2, (cuuint64_t)ss * 2, (cuuint64_t)ss * 2 * a.g.tokens};
    const cuuint32_t box[4] = {64, (cuuint32_t)a.g.group, (cuuint32_t)(kBM / a.g.group), 1}, step[4] = {1, 1, 1, 1};
    auto enc = tc_encode_fn();
    t.q_tma = strides[2] < ((cuuint64_t)1 << 40) && enc &&
              enc(&tq, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(a.q.p),
                  dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  cudaError_t e;
  if (a.g.H == 128) {
    *name = bf ? "paged4_tc_bf16_h128" : "paged4_tc_f16_h128";
    e = launch_h<128>(bf, cap, tq, t, ctas, st);
  } else {
    *name = bf ? "paged4_tc_bf16_h64" : "paged4_tc_f16_h64";
    e = launch_h<64>(bf, cap, tq, t, ctas, st);
  }
  return e == cudaSuccess ? launch_paged_merge(a, dt, t.ws, ctas, kTM, st) : e;
}

cudaError_t take_paged4_tc_status(int* status, int* timeout) {
  int v[2] = {0, 0};
  const cudaError_t e = take_words(g_paged4_words, v);
  *status = v[0];
  *timeout = v[1];
  return e;
}

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_paged4_tc)

}  // namespace sdpa
