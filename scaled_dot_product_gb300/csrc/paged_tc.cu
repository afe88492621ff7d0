// Attention over a paged cache for chunks of new tokens: fp16 / bf16, H == Hv in {64, 128}, page
// sizes that are multiples of 8.
//
// Bound by the tensor cores.  A unit is 256 packed rows (token x group head) of one (sequence,
// kv head): two 128-row tiles that stream the same keys and values.  A unit of at most 128 rows (a
// single token beside chunks) has one tile of rows; there the two softmax warpgroups take turns with
// the keys, even tiles and odd ones with their own maximum, sum and accumulator, joined at its end.
// One CTA per SM walks its share (paged_sched.cuh) of all units' 128-key tiles:
//
//   warp 0      K tiles into the ring by TMA, and query tiles where the group divides 128.  A tile is
//               128 / box boxes of box = gcd(page_size, 128) rows, each inside one page; lane by lane
//               they are looked up and issued
//   warp 1      tensor products (one elected lane issues): S_X = Q_X K^T, O_X += P_X V with P
//               read from tensor memory.  Rows of V past the sequence's keys or below every
//               window of the unit it sets to zero first, since 0 x NaN is not 0
//   warp 2      V tiles into the same ring
//   warp 3      query rows by 16-byte asynchronous copies for the other groups
//   warps 4-7   softmax of tile 0, one thread per row; warps 8-11 softmax of tile 1
//
// A chunk of 2048 tokens over 32000 keys, 32/8 heads of 128: 717 to 768 us, 1430 to 1530 TFLOP/s (76
// to 81 % of the measured bf16 burst rate); a causal prompt of 4096 tokens 125 to 138 us, up to 1090
// TFLOP/s (64/8 heads of 64: 194 us, 709); single tokens through this kernel 6.4 TB/s.  Running maxima
// move only when they grow by more than 2^8.  The weights enter the second product rounded to the
// element type (half a step each), since its operands are 16-bit; their sum takes them unrounded.
// 168 registers at launch, 252 bytes of spills a thread.  paged4_tc.cu has the same roles, waits and abort path over
// records of 4 bits a value: what is mended in one has to be mended in the other.  Every wait is bounded: on expiry the kernel
// raises an abort flag, lets its own copies and products finish, frees its tensor memory and records
// SDPA_ERR_TIMEOUT.
#include <algorithm>
#include <cstdlib>
#include <type_traits>

#include "paged_sched.cuh"
#include "prefill_tc.h"

namespace sdpa {

static __device__ int g_paged_words[2];      // status bits, SDPA_ERR_TIMEOUT after an expired wait

namespace {

using namespace ptx;

constexpr int kBM = 128, kTM = 256, kTN = 128;
constexpr int kThreads = 384;
// A unit's cost beside its tiles (a tile costs 4, or 3 in a narrow unit).  Measured: 4 chunks and 24
// tokens with a window of 1024 81 us (with 4: 84, with 16: 87), a causal prompt of 4096 137 us on the
// same GPU (166, 137).
constexpr int kOV = 8;
// Least cost worth a CTA: 12, 24 and 48 measure alike, down to four prompts of 1000 (61 to 67 us each).
constexpr int kMinShare = 24;
// Register split: the control warpgroup shrinks to kCtlRegs, the softmax warpgroups grow to
// kSmxRegs; the sum stays within the launch's kThreads x kLaunchRegs, which the host checks.
constexpr int kLaunchRegs = 168, kCtlRegs = 88, kSmxRegs = 208;
static_assert(kCtlRegs * 128 + kSmxRegs * 256 <= kLaunchRegs * kThreads, "register split");
constexpr float kRescale = 8.f;      // log2 units

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
  int box, boxes;                    // rows per box, boxes per tile
  int k_ds, k_dn, k_db, v_ds, v_dn, v_db;   // tensor-map dimension of slot / head / page
  float scale_log2, cap_in, cap_log2;
  int q_tma;                         // query rows by TMA: boxes of one group's heads x 128 / group tokens
  int pre;                           // scale <= 0: scores are scaled before the maximum
  uint64_t wait_ns;
};

// Keys outside [elo, ehi] of a 128-key segment take -inf: per 32 columns one bit set, then one
// test and one select per key.
__device__ __forceinline__ void clip(float (&s)[128], int elo, int ehi) {
#pragma unroll
  for (int c0 = 0; c0 < 128; c0 += 32) {
    const int lo = max(elo - c0, 0), hi = min(ehi - c0, 31);
    const uint32_t up = 0xffffffffu >> (31 - max(hi, 0));
    const uint32_t m = (lo <= hi) ? (up & (0xffffffffu << min(lo, 31))) : 0u;
#pragma unroll
    for (int e = 0; e < 32; ++e) s[c0 + e] = ((m >> e) & 1u) ? s[c0 + e] : -INFINITY;
  }
}

// Rows of key tile kt that the boxes (a power of two rows) bring: [first, last) of 128.
__device__ __forceinline__ void box_rows(const TcArgs& t, const SeqInfo& s, const RowBlock& r, int kt, int& first, int& last) {
  first = max(0, min(kTN, (r.lo & -t.box) - kt * kTN));
  last = max(first, min(kTN, s.T - kt * kTN));
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
    paged_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv,
                    const __grid_constant__ TcArgs t) {
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
  __shared__ int issued[2][C::kStages];      // last tile + 1 that K's / V's producer put into a stage
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
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
    if (t.q_tma) prefetch_tmap(&tq);
    abort_flag = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), 1);
      issued[0][s] = issued[1][s] = 0;
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
  const Share sh = find_share<kTM, kTN, kOV, kThreads>(a, cta, ctas, kMinShare, &g_paged_words[0]);
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

  if (warp == 0 || warp == 2) {
    // ================================================================ producers: K and Q, V
    // A lane's box: region = lane / 16, box = lane % 16.  The loads of a warp are issued one lane after
    // the other (about 150 cycles each), so K and V have a warp each: with one for both, narrow units
    // over pages of 16 waited for it.  Page ids are fetched a tile ahead.
    const bool is_v = warp == 2;
    const int region = lane >> 4, row = (lane & 15) * t.box;
    const CUtensorMap* map = is_v ? &tv : &tk;
    const int ds = is_v ? t.v_ds : t.k_ds, dn = is_v ? t.v_dn : t.k_dn;
    int base = 0, it = 0;                // ring position of the unit's first tile, units
    bool ok = true;
    for (Wk w(a, sh); ok && !w.done(); w.next(a)) {
      const int n = w.take(), kt0 = w.r.tile0 + w.tile;
      const int32_t* table = g.table + (int64_t)w.b * g.table_stride;
      auto brought = [&](int j) -> bool {
        int first, last;
        box_rows(t, w.s, w.r, kt0 + j, first, last);
        return j < n && region < C::kRegions && row < kTN && row >= first && row < last;
      };
      int id = 0;
      auto look_up = [&](int j) {
        if (brought(j)) id = table[page_div(g, (kt0 + j) * kTN + row)];
      };
      look_up(0);
      for (int j = 0; j < n; ++j) {
        const int sq = base + (is_v ? v_at<C::kAlias>(j, n) : k_at<C::kAlias>(j)), st = sq % C::kStages;
        if (sq >= C::kStages && !(ok = wait_all(b_empty(st), ((sq / C::kStages) - 1) & 1))) break;
        const bool take = brought(j);
        if (take && (unsigned)id >= (unsigned)g.num_pages) {
          atomicOr(&g_paged_words[0], kPagedBadPage);
          id = g.num_pages;              // outside the map: the box is filled with zeros
        }
        const unsigned all = __ballot_sync(0xffffffffu, take);
        if (lane == 0) {
          mbar_arrive_expect_tx(b_full(st), __popc(all) * t.box * 128);
          issued[is_v][st] = sq + 1;
        }
        __syncwarp();
        if (take && SDPA_IN_BOUNDS(st < C::kStages && row + t.box <= kTN && w.kvh < g.Nkv, 541)) {
          const int key = (kt0 + j) * kTN + row, slot = key - page_div(g, key) * g.page_size;
          const int c1 = ds == 1 ? slot : dn == 1 ? w.kvh : id, c2 = ds == 2 ? slot : dn == 2 ? w.kvh : id,
                    c3 = ds == 3 ? slot : dn == 3 ? w.kvh : id;
          tma_load_4d(sKV + st * C::kTile + region * C::kRegionBytes + row * 128, map, b_full(st), 64 * region, c1, c2, c3);
        }
        __syncwarp();
        look_up(j + 1);
        if (j == 0 && !is_v && t.q_tma) {
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
      const int n = w.take(), kt0 = w.r.tile0 + w.tile, nx = w.r.rows > kBM ? 2 : 1;
      // rows of V tile j past the sequence's keys or below the unit's windows become zeros
      auto zero_v = [&](int j, int st) {
        int first, last;
        box_rows(t, w.s, w.r, kt0 + j, first, last);
        first = max(first, min(kTN, w.r.lo - (kt0 + j) * kTN));
        if (first == 0 && last == kTN) return;
        for (int i = lane; i < kTN * 8; i += 32) {
          const int row = i >> 3;
          if (row < first || row >= last) {
#pragma unroll
            for (int r = 0; r < C::kRegions; ++r)
              st_shared_v4(sKV + st * C::kTile + r * C::kRegionBytes + i * 16, 0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
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
          zero_v(j, vst);
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
          zero_v(j, vst);
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
          zero_v(j, vst);
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
                     "r"(take && SDPA_IN_BOUNDS(w.s.t0 + tok < g.tokens, 542) ? 16 : 0) : "memory");
      }
      cp_async_commit();
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_qready);
    }
  } else {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSmxRegs));
    const int x = (warp - 4) >> 2, sub = warp & 3;
    const int row = sub * 32 + lane;                 // row of the tile == tensor-memory lane
    const uint32_t trow = tmem + ((uint32_t)(sub * 32) << 16);
    const uint32_t tS = trow + 128 * x, tO = trow + (x ? C::kO1 : C::kO0), tP = trow + (x ? C::kP1 : C::kP0);
    const uint32_t sY = sQ + C::kYOff + (uint32_t)(x * 4 + sub) * C::kYWarp;
    const float kfac = CAP || t.pre ? 1.f : t.scale_log2;
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
      float m = -INFINITY, l = 0.f;
      for (int j = j0; j < n; j += js) {
        if (!(ok = wait_all(b_sfull(x), cs & 1))) break;
        ++cs;
        tc_fence_after();
        float s[128];
        {
          uint32_t u[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, u + c * 32);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 128; ++e) s[e] = __uint_as_float(u[e]);
        }
        if constexpr (!C::kAlias) {
          tc_fence_before();
          mbar_arrive(b_sfree(x));
        }
        if constexpr (CAP) {
          // cap tanh(u) in log2 units: 1 - 2 / (e^2u + 1), absolute error about 2^-23 of the cap
          const float c2 = 2.f * kLog2e * t.cap_in;
#pragma unroll
          for (int e = 0; e < 128; ++e)
            s[e] = t.cap_log2 * (1.f - __fdividef(2.f, ex2_approx(s[e] * c2) + 1.f));
        } else if (t.pre) {
#pragma unroll
          for (int e = 0; e < 128; ++e) s[e] *= t.scale_log2;
        }
        const int key0 = (kt0 + j) * kTN;
        if (!(lo <= key0 && key0 + kTN - 1 <= hi)) clip(s, lo - key0, hi - key0);
        float mx8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(s[k], s[k + 8]);
#pragma unroll
        for (int e = 16; e < 128; e += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], s[e + k], s[e + 8 + k]);
        const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        const float m_new = fmaxf(m, mx * kfac);
        const bool need = m_new > m + kRescale;      // true for a row's first keys: m = -inf
        float corr = 1.f;
        if (need) {
          corr = ex2_approx(m - m_new);
          m = m_new;
        }
        // rows with nothing admitted yet: exponent -inf, weight 0
        const float negm = (m == -INFINITY) ? -INFINITY : -m;
        const f2_t kf2 = f2_pack(kfac, kfac), nm2 = f2_pack(negm, negm);
        f2_t acc[4] = {f2_zero(), f2_zero(), f2_zero(), f2_zero()};
        uint32_t pw[64];
#pragma unroll
        for (int e = 0; e < 128; e += 2) {
          float z0, z1;
          f2_unpack(f2_fma(f2_pack(s[e], s[e + 1]), kf2, nm2), z0, z1);
          const float p0 = ex2_approx(z0), p1 = ex2_approx(z1);
          acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3], f2_pack(p0, p1));
          pw[e >> 1] = BF ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
        }
        float r0, r1, r2, r3;
        f2_unpack(f2_add(acc[0], acc[1]), r0, r1);
        f2_unpack(f2_add(acc[2], acc[3]), r2, r3);
        l = l * corr + ((r0 + r1) + (r2 + r3));
        if (j != j0) {
          // the previous PV_X has read P_X and O_X holds it (with P in S's columns, sfull said so)
          if constexpr (!C::kAlias) {
            if (!(ok = wait_all(b_odone(x), co & 1))) break;
            ++co;
            tc_fence_after();
          }
          if (__any_sync(0xffffffffu, need)) {
            const f2_t c2 = f2_pack(corr, corr);
#pragma unroll
            for (int c = 0; c < H / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float v0, v1;
                f2_unpack(f2_mul(f2_pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), c2), v0, v1);
                o[e] = __float_as_uint(v0);
                o[e + 1] = __float_as_uint(v1);
              }
              tmem_st32(tO + c * 32, o);
            }
            tmem_st_wait();
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_st32(tP + c * 32, pw + c * 32);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(b_pfull(x));
      }
      if (!ok) break;

      // ---- the unit's rows, or their partial results
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
#pragma unroll
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
              if (rr < live && SDPA_IN_BOUNDS(w.s.t0 + w.s.n <= g.tokens, 543))
                *reinterpret_cast<uint4*>((uintptr_t)dst + (c >> 1) * 128 + c16 * 16) = v;
            }
            __syncwarp();
          }
        }
      } else {
        const int64_t base = (2 * (int64_t)cta + (w.begins() ? 1 : 0)) * kTM + tile_row + sub * 32;
#pragma unroll
        for (int c = 0; c < H / 32; ++c) {
          uint32_t o[32];
          read_o(c, o);
          if (c == 0 && lane < live && SDPA_IN_BOUNDS(base + lane < (int64_t)2 * ctas * kTM, 544)) {
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
            if (rr < live && SDPA_IN_BOUNDS(base + rr < (int64_t)2 * ctas * kTM, 545))
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
    // Some role gave up, perhaps behind the producers' last copies: every copy lands before the CTA,
    // whose shared memory it writes, ends.  A stage's and the query tiles' earlier copies landed
    // before their space was filled again.
    if (issued_q > 0) mbar_wait_bounded(b_qready, (issued_q - 1) & 1, nullptr, kDrainNs);
    for (int s = 0; s < C::kStages; ++s) {
      const int last = max(issued[0][s], issued[1][s]);
      if (last > 0) mbar_wait_bounded(b_full(s), ((last - 1) / C::kStages) & 1, nullptr, kDrainNs);
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && abort_flag) atomicExch(&g_paged_words[1], (int)SDPA_ERR_TIMEOUT);
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
cudaError_t launch_cap(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TcArgs& t, int ctas,
                       cudaStream_t st) {
  using C = Cfg<H>;
  auto* kernel = paged_tc_kernel<H, BF, CAP>;
  // per device: set at every call (the attribute belongs to the current context)
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  cudaFuncAttributes fa{};
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
  // with fewer registers at launch the softmax warps' request could never be met
  if (e == cudaSuccess && fa.numRegs < kLaunchRegs) e = cudaErrorLaunchOutOfResources;
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)ctas, kThreads, C::kSmem, st>>>(tq, tk, tv, t);
  count_launch(1);
  return cudaGetLastError();
}

template <int H>
cudaError_t launch_h(bool bf, bool cap, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     const TcArgs& t, int ctas, cudaStream_t st) {
  if (bf) return cap ? launch_cap<H, true, true>(tq, tk, tv, t, ctas, st) : launch_cap<H, true, false>(tq, tk, tv, t, ctas, st);
  return cap ? launch_cap<H, false, true>(tq, tk, tv, t, ctas, st) : launch_cap<H, false, false>(tq, tk, tv, t, ctas, st);
}

}  // namespace

// Dimension 0 is the head's channels; 1 to 3 are slot, head and page in the order of their strides
// (ds, dn, db say where each went).  A box is 64 channels of box_rows slots.
bool paged_map(CUtensorMap* map, const Paged& g, const View& v, int D, sdpa_dtype dt, int box_rows, int* ds, int* dn, int* db) {
  auto enc = tc_encode_fn();
  if (!enc) return false;
  int order[3];
  tc_axis_order(v, g.num_pages, g.Nkv, g.page_size, order);
  const int64_t ext[3] = {g.page_size, g.Nkv, g.num_pages}, str[3] = {v.ss, v.sh, v.sb};
  int* where[3] = {ds, dn, db};
  cuuint64_t dims[4] = {(cuuint64_t)D, 1, 1, 1}, strides[3];
  cuuint32_t box[4] = {64, 1, 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  int64_t span = D;                      // elements up to here: a legal stride for an axis of one entry
  for (int k = 0; k < 3; ++k) {
    const int id = order[k];
    const int64_t st = ext[id] > 1 ? str[id] : (span + 7) / 8 * 8;
    dims[k + 1] = (cuuint64_t)ext[id];
    strides[k] = (cuuint64_t)(st * 2);
    span = std::max(span, st * ext[id]);
    if (id == 0) box[k + 1] = (cuuint32_t)box_rows;
    *where[id] = k + 1;
  }
  // a head's row is one 128-byte line at D = 64: fetching 256 bytes would bring another head's (single
  // tokens over 1.06 GB of such pages took 281 us against 203)
  const CUtensorMapL2promotion promote = D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  return enc(map, dt == SDPA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(v.p),
             dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promote,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool paged_boxes(const PagedAttn& a) {
  if (a.g.page_size % 8 || a.g.num_pages < 1) return false;
  for (const View* v : {&a.g.kp, &a.g.vp})
    for (int64_t s : {v->sb, v->sh, v->ss})
      if (s >= ((int64_t)1 << 38)) return false;
  return true;
}

// More rows of a sequence than paged_mma's widest unit holds.  16 sequences of 2000 to 8000 keys, 8
// query heads a key head, H = 64 / 128: 72 rows 54 / 79 us here, 93 / 166 there; 64 rows 54 / 78 here, 54
// / 96 there; 32 rows 52 / 77 here, 42 / 70 there.
bool paged_tc_supported(const PagedAttn& a, sdpa_dtype dt) {
  return paged_mma_supported(a.g.H, a.g.Hv, dt) && paged_boxes(a) && (int64_t)a.max_new * a.g.group > 64;
}

size_t paged_tc_workspace(int Hv) { return paged_ws_bytes(kPagedMaxSms, kTM, Hv); }

cudaError_t launch_paged_tc(const PagedAttn& a, sdpa_dtype dt, void* wsp, cudaStream_t st, const char** name) {
  const int ctas = paged_sms();
  if (ctas <= 0) return cudaErrorInvalidDevice;
  TcArgs t{};
  t.a = a;
  t.ws = paged_ws(wsp, ctas, kTM);
  t.box = kTN;
  while (a.g.page_size % t.box) t.box >>= 1;
  t.boxes = kTN / t.box;
  t.scale_log2 = a.scale * kLog2e;
  t.pre = !(a.scale > 0.f);
  t.cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
  t.cap_log2 = a.softcap * kLog2e;
  t.wait_ns = wait_limit_ns();
  CUtensorMap tk, tv;
  if (!paged_map(&tk, a.g, a.g.kp, a.g.H, dt, t.box, &t.k_ds, &t.k_dn, &t.k_db) ||
      !paged_map(&tv, a.g, a.g.vp, a.g.Hv, dt, t.box, &t.v_ds, &t.v_dn, &t.v_db))
    return cudaErrorInvalidValue;
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
    *name = bf ? "paged_tc_bf16_h128" : "paged_tc_f16_h128";
    e = launch_h<128>(bf, cap, tq, tk, tv, t, ctas, st);
  } else {
    *name = bf ? "paged_tc_bf16_h64" : "paged_tc_f16_h64";
    e = launch_h<64>(bf, cap, tq, tk, tv, t, ctas, st);
  }
  return e == cudaSuccess ? launch_paged_merge(a, dt, t.ws, ctas, kTM, st) : e;
}

cudaError_t take_paged_tc_status(int* status, int* timeout) {
  int v[2] = {0, 0};
  const cudaError_t e = take_words(g_paged_words, v);
  *status = v[0];
  *timeout = v[1];
  return e;
}

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_paged_tc)

}  // namespace sdpa
