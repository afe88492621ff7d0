// RMS norm of every query and key head followed by the position rotation, in one pass, and its
// gradient.  With r = (mean(x^2) + eps)^-1/2 over the D channels of a head and u = x r w:
//
//     y  = Rot(u)                                   (the pairs of class RotaryEmbedding)
//     g  = Rot^T(dy),  dw = sum over rows of g x r,  dx = r (g w - x r mean(g w x r))
//
// All arithmetic is fp32; each output is rounded once to the element type.
//
// Bytes bound both directions: x (and dy) are read once and y (dx) is written once.  LPR lanes
// share one row, one 16-byte vector each; the row's sum is a shuffle over them, and in the split
// pair layout the packed partners come from another lane.  (Two vectors a lane, pairs together,
// save those shuffles but took 118 registers forward and 174 backward, and the loads in flight
// with them: 20.9 and 98.7 us on the first and last of these.)  On the device, bf16, heads of 128:
// 4096 tokens x 40 heads forward 16.5 us (5.1 TB/s), 4503 tokens x 72 float16 heads of 64 15.0 us
// (5.55 TB/s), backward of 8192 tokens x 40 heads 50.7 us (5.0 TB/s); in fp32 29.1 us (5.8 TB/s) and 79.5
// us (6.4 TB/s) for the first and the last.
// Shapes or pointers that do not allow 16-byte vectors take the scalar kernels (one warp per
// row, the row in shared memory), as do fp32 heads of more than 128 channels: 63.0 and 196 us for as
// many bytes as those two fp32 cases, 76.6 us for the first case with 20 of 128 channels rotated.
#include <algorithm>

#include "qk_norm.h"
#include "tc_ptx.cuh"

namespace sdpa {

static __device__ int g_norm_status[1];

namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kFwdThreads = 128;
constexpr int kMaxD = 256;

// 16-byte asynchronous copy, or 16 zero bytes; waits until at most N groups are on their way.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Position of token tok, and its row in the caches: a position outside them is recorded and
// clamped.
__device__ __forceinline__ int64_t position(const NormJob& j, int tok) { return j.positions ? j.positions[tok] : tok; }
__device__ __forceinline__ int64_t cache_row(const NormJob& j, int64_t row) {
  if (row < 0 || row >= j.max_pos) {
    atomicExch(g_norm_status, 1);
    row = row < 0 ? 0 : j.max_pos - 1;
  }
  return row;
}

// (x1, x2) turned by the angle of (c, s)
__device__ __forceinline__ void turn(float& x1, float& x2, float c, float s) {
  const float o1 = fmaf(x1, c, -x2 * s);
  const float o2 = fmaf(x2, c, x1 * s);
  x1 = o1;
  x2 = o2;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// 16 bytes of T as pairs of floats, and back (one rounding).
template <typename T>
__device__ __forceinline__ void to_pairs(const uint4& u, f2_t* f) {
  constexpr int V = 16 / (int)sizeof(T);
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};      // a bf16 is the upper half of its float
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = f2_pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  } else {
    float x[V];
    unpack16<T>(u, x);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) f[e] = f2_pack(x[2 * e], x[2 * e + 1]);
  }
}
template <typename T>
__device__ __forceinline__ uint4 from_pairs(const f2_t* f) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 8 / (int)sizeof(T); ++e) {
    float lo, hi;
    f2_unpack(f[e], lo, hi);
    if constexpr (sizeof(T) == 4) {
      w[2 * e] = __float_as_uint(lo);
      w[2 * e + 1] = __float_as_uint(hi);
    } else {
      w[e] = std::is_same<T, __half>::value ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float pair_sum(f2_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}

// A lane owns one 16-byte vector of its row, channels c0 .. c0 + V - 1.  The rotation of every
// channel is x C + mate(x) S with a signed sine S: the mate is the neighbour in the vector
// (adjacent pairs) or the same place of the vector `half` vectors away, in another lane of the row
// (split pairs; as packed words four shuffles).  Channels that are not rotated have C = 1 and a
// mate of 0.
template <typename T, bool kInter, int LPR>
struct Lane {
  static constexpr int V = 16 / (int)sizeof(T), P = V / 2;
  int c0, mate, ci;                // mate's lane, first cos / sin entry
  bool live, rot, second;          // has channels; is rotated; holds the second of its pairs
  uint4 cw, sw;                    // packed cos and sin (adjacent pairs: the first half)
  __device__ __forceinline__ Lane(int u, int D, int R)
      : c0(u * V), mate(u), ci(0), live(u * V < D), rot(u * V < R), second(false) {
    cw = sw = make_uint4(0u, 0u, 0u, 0u);
    if (kInter) {
      ci = c0 / 2;
    } else if (rot) {
      const int half = R / (2 * V);
      second = u >= half;
      mate = second ? u - half : u + half;
      ci = min(u, mate) * V;
    }
  }
  __device__ __forceinline__ uint4 load(const T* row) const {
    return live ? *reinterpret_cast<const uint4*>(row + c0) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void load_cs(const T* cr, const T* sr) {
    if (!rot) return;
    if constexpr (kInter) {
      const uint2 c = *reinterpret_cast<const uint2*>(cr + ci), s = *reinterpret_cast<const uint2*>(sr + ci);
      cw.x = c.x; cw.y = c.y;
      sw.x = s.x; sw.y = s.y;
    } else {
      cw = *reinterpret_cast<const uint4*>(cr + ci);
      sw = *reinterpret_cast<const uint4*>(sr + ci);
    }
  }
  // C and S of the lane's channels; dir = -1 turns back
  __device__ __forceinline__ void factors(f2_t* C, f2_t* S, float dir) const {
    float c[V], s[V];
    unpack16<T>(cw, c);
    unpack16<T>(sw, s);
    if constexpr (kInter) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        C[e] = f2_pack(rot ? c[e] : 1.f, rot ? c[e] : 1.f);
        S[e] = f2_pack(-dir * s[e], dir * s[e]);
      }
    } else {
      // x1 c - x2 s in the first half, x2 c + x1 s in the second
      const float sg = second ? dir : -dir;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        C[e] = f2_pack(rot ? c[2 * e] : 1.f, rot ? c[2 * e + 1] : 1.f);
        S[e] = f2_pack(sg * s[2 * e], sg * s[2 * e + 1]);
      }
    }
  }
  // The mates of the lane's channels; x are its own pairs, w the same as packed words.
  __device__ __forceinline__ void mates(const uint4& w, const f2_t* x, f2_t* m) const {
    if constexpr (kInter) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        float lo, hi;
        f2_unpack(x[e], lo, hi);
        m[e] = rot ? f2_pack(hi, lo) : f2_zero();
      }
    } else {
      uint4 v = make_uint4(__shfl_sync(0xffffffffu, w.x, mate, LPR), __shfl_sync(0xffffffffu, w.y, mate, LPR),
                           __shfl_sync(0xffffffffu, w.z, mate, LPR), __shfl_sync(0xffffffffu, w.w, mate, LPR));
      if (!rot) v = make_uint4(0u, 0u, 0u, 0u);
      to_pairs<T>(v, m);
    }
  }
  __device__ __forceinline__ void store(T* row, const f2_t* f) const {
    if (live) *reinterpret_cast<uint4*>(row + c0) = from_pairs<T>(f);
  }
};

// ---------------------------------------------------------------- forward

// One group of LPR lanes takes HPG heads of one token: the cos/sin row and the weights are read
// once for them and folded into two factors a channel, y = r (x (w C) + mate(x) (mate(w) S)), and
// HPG x 16 bytes are in flight per lane.
template <typename T, bool kInter, int LPR, int HPG>
__global__ void __launch_bounds__(kFwdThreads, 10) norm_fwd_kernel(const NormJob j, const int q_blocks) {
  constexpr int V = 16 / (int)sizeof(T), P = V / 2;
  const bool is_k = (int)blockIdx.x >= q_blocks;
  const NormSide& sd = j.side[is_k];
  const int chunks = (sd.N + HPG - 1) / HPG;
  const unsigned task = (blockIdx.x - (is_k ? q_blocks : 0)) * (unsigned)(kFwdThreads / LPR) + threadIdx.x / LPR;
  const unsigned tok = task / (unsigned)chunks;
  const int h0 = (int)(task - tok * (unsigned)chunks) * HPG;
  const bool live = tok < (unsigned)j.tokens;
  const int b = live ? (int)(tok / (unsigned)j.S) : 0, s = live ? (int)(tok - (unsigned)b * (unsigned)j.S) : 0;
  const int nh = live ? min(HPG, sd.N - h0) : 0;
  Lane<T, kInter, LPR> ln(threadIdx.x % LPR, j.D, j.R);
  const T* x0 = reinterpret_cast<const T*>(sd.x.p) + sd.x.off(b, h0, s);
  T* y0 = reinterpret_cast<T*>(const_cast<void*>(sd.y.p)) + sd.y.off(b, h0, s);

  uint4 xw[HPG];
#pragma unroll
  for (int i = 0; i < HPG; ++i)
    xw[i] = i < nh && SDPA_IN_BOUNDS(b < j.B && h0 + i < sd.N && s < j.S, 501) ? ln.load(x0 + i * sd.x.sh)
                                                                                : make_uint4(0u, 0u, 0u, 0u);
  const uint4 ww = ln.load(reinterpret_cast<const T*>(sd.w));
  if (j.R > 0 && live) {
    const int64_t row = cache_row(j, position(j, (int)tok)) * (j.R / 2);
    ln.load_cs(reinterpret_cast<const T*>(j.cos_c) + row, reinterpret_cast<const T*>(j.sin_c) + row);
  }
  f2_t A[P], Bf[P], w[P], m[P];
  ln.factors(A, Bf, 1.f);
  to_pairs<T>(ww, w);
  ln.mates(ww, w, m);
#pragma unroll
  for (int e = 0; e < P; ++e) {
    A[e] = f2_mul(A[e], w[e]);
    Bf[e] = f2_mul(Bf[e], m[e]);
  }
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    f2_t x[P];
    to_pairs<T>(xw[i], x);
    ln.mates(xw[i], x, m);
    f2_t ss = f2_zero();
#pragma unroll
    for (int e = 0; e < P; ++e) ss = f2_fma(x[e], x[e], ss);
    const float r = rsqrtf(row_sum<LPR>(pair_sum(ss)) * j.inv_D + j.eps);
    const f2_t r2 = f2_pack(r, r);
#pragma unroll
    for (int e = 0; e < P; ++e) x[e] = f2_mul(f2_fma(x[e], A[e], f2_mul(m[e], Bf[e])), r2);
    if (i < nh) ln.store(y0 + i * sd.y.sh, x);
  }
}

// One warp per row; channels lane, lane + 32, ...; the row sits in shared memory between the
// norm and the rotation.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_fwd_scalar_kernel(const NormJob j, const int interleaved) {
  __shared__ float sh[kThreads / 32][kMaxD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* f = sh[warp];
  const int N = j.side[0].N + j.side[1].N;
  const int64_t rows = (int64_t)j.tokens * N;
  for (int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + warp; row < rows; row += (int64_t)gridDim.x * (kThreads / 32)) {
    const int tok = (int)(row / N);
    int h = (int)(row - (int64_t)tok * N);
    const bool is_k = h >= j.side[0].N;
    if (is_k) h -= j.side[0].N;
    const NormSide& sd = j.side[is_k];
    const int b = tok / j.S, s = tok - b * j.S;
    const T* x = reinterpret_cast<const T*>(sd.x.p) + sd.x.off(b, h, s);
    T* y = reinterpret_cast<T*>(const_cast<void*>(sd.y.p)) + sd.y.off(b, h, s);
    float ss = 0.f;
    for (int d = lane; d < j.D; d += 32) {
      const float v = Elem<T>::to_f32(x[d]);
      f[d] = v;
      ss = fmaf(v, v, ss);
    }
    const float r = rsqrtf(row_sum<32>(ss) * j.inv_D + j.eps);
    const T* w = reinterpret_cast<const T*>(sd.w);
    for (int d = lane; d < j.D; d += 32) f[d] = f[d] * r * Elem<T>::to_f32(w[d]);
    __syncwarp();
    const int half = j.R / 2;
    const int64_t crow = j.R > 0 ? cache_row(j, position(j, tok)) * half : 0;
    for (int d = lane; d < half; d += 32) {
      const int i1 = interleaved ? 2 * d : d, i2 = interleaved ? 2 * d + 1 : d + half;
      float a = f[i1], p = f[i2];
      turn(a, p, Elem<T>::to_f32(reinterpret_cast<const T*>(j.cos_c)[crow + d]),
           Elem<T>::to_f32(reinterpret_cast<const T*>(j.sin_c)[crow + d]));
      y[i1] = Elem<T>::from_f32(a);
      y[i2] = Elem<T>::from_f32(p);
    }
    for (int d = j.R + lane; d < j.D; d += 32) y[d] = Elem<T>::from_f32(f[d]);
    __syncwarp();
  }
}

// ---------------------------------------------------------------- backward

// Persistent: blocks [0, q_blocks) walk the query tasks, the others the key tasks, so a lane
// accumulates dw for the one weight vector of its side.  A task is up to kHeads heads of one
// token, taken kPair at a time, whose sums' shuffles overlap; the next kRing - 1 pairs' x and dy are on
// their way into shared memory meanwhile.  Each block leaves its D sums in part[blockIdx.x]; norm_dw_kernel adds them in
// block order, so results do not vary from run to run.  Bound by instructions in 16-bit types: 68 % of
// the issue slots are busy (DRAM 57 %), and a scheduler's four warps wait for their turn (1.2 of them
// per issued instruction) and for fixed latencies (1.2) more than for memory (0.5) or shuffles (0.4).
// One head at a time took 72 us on 8192 tokens x 40 heads, tasks of 16
// heads 71, three blocks an SM (spills) 90, the next pair in registers instead of the ring 53.3, equal
// contiguous shares of the rows instead of tasks in turn 54.3, this 50.7.
constexpr int kHeads = 8, kPair = 2, kRing = 4;
constexpr int kRingBytes = kRing * kPair * 2 * kThreads * 16;
constexpr int kBwdBlocks = 2;
template <typename T, bool kInter, int LPR>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) norm_bwd_kernel(const NormJob j, const int q_blocks,
                                                                        float* __restrict__ part) {
  constexpr int V = 16 / (int)sizeof(T), P = V / 2;
  constexpr int kGroups = kThreads / LPR;
  __shared__ float red[kGroups][LPR * V + 1];
  extern __shared__ uint4 ring[];    // [kRing][kPair][x, dy][kThreads]
  const bool is_k = (int)blockIdx.x >= q_blocks;
  const NormSide& sd = j.side[is_k];
  const unsigned nblk = is_k ? gridDim.x - q_blocks : q_blocks;
  const unsigned blk = is_k ? blockIdx.x - q_blocks : blockIdx.x;
  const unsigned chunks = (unsigned)(sd.N + kHeads - 1) / kHeads;
  const unsigned tasks = (unsigned)j.tokens * chunks;
  const int u = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  Lane<T, kInter, LPR> ln(u, j.D, j.R);
  f2_t w[P], dw[P], C[P], S[P];
  to_pairs<T>(ln.load(reinterpret_cast<const T*>(sd.w)), w);
#pragma unroll
  for (int e = 0; e < P; ++e) dw[e] = f2_zero();

  // Every group of a block runs kHeads / kPair steps per task (the shuffles need whole warps); heads
  // past the task's, and tasks past the last, touch no memory.  `ahead` brings the steps to come:
  // every thread copies its own vectors into its own slots of the ring, so no barrier is needed.
  const unsigned stride = nblk * kGroups;
  struct Cursor { const T *x, *g; T* d; unsigned tok; int n; };
  auto place = [&](unsigned t0, Cursor& c) {
    const unsigned task = t0 + grp;
    c.n = 0;
    if (t0 >= tasks || task >= tasks) return;
    c.tok = task / chunks;
    const int h0 = (int)(task - c.tok * chunks) * kHeads;
    const int b = (int)(c.tok / (unsigned)j.S), s = (int)(c.tok - (unsigned)b * (unsigned)j.S);
    c.n = min(kHeads, sd.N - h0);
    c.x = reinterpret_cast<const T*>(sd.x.p) + sd.x.off(b, h0, s) + ln.c0;
    c.g = reinterpret_cast<const T*>(sd.dy.p) + sd.dy.off(b, h0, s) + ln.c0;
    c.d = reinterpret_cast<T*>(const_cast<void*>(sd.y.p)) + sd.y.off(b, h0, s);
    if (!SDPA_IN_BOUNDS(b < j.B && h0 + c.n <= sd.N && s < j.S, 502)) c.n = 0;
  };
  unsigned at = blk * kGroups;       // task row of the copies
  int ai = 0, put = 0;               // first head of the copies' step, its ring slot
  Cursor fetch{};
  auto ahead = [&]() {
    if (at < tasks) {
      if (ai == 0) place(at, fetch);
#pragma unroll
      for (int k = 0; k < kPair; ++k) {
        const bool take = ai + k < fetch.n && ln.live;
        const uint32_t slot = smem_u32(ring) + (uint32_t)(((put * kPair + k) * 2) * kThreads + threadIdx.x) * 16;
        cp_async16_or_zero(slot, take ? fetch.x : reinterpret_cast<const T*>(sd.w), take);
        cp_async16_or_zero(slot + kThreads * 16, take ? fetch.g : reinterpret_cast<const T*>(sd.w), take);
        fetch.x += sd.x.sh;
        fetch.g += sd.dy.sh;
      }
      ai += kPair;
      if (ai == kHeads) {
        ai = 0;
        at += stride;
      }
    }
    cp_async_commit();
    put = put + 1 == kRing ? 0 : put + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kRing - 1; ++i) ahead();
  Cursor now{}, next{};
  int64_t pos = 0;                   // position of the next task's token: on its way before it is needed
  place(blk * kGroups, now);
  auto load_cs = [&](const Cursor& c) {
    if (j.R == 0 || c.n == 0) return;
    const int64_t row = cache_row(j, pos) * (j.R / 2);
    ln.load_cs(reinterpret_cast<const T*>(j.cos_c) + row, reinterpret_cast<const T*>(j.sin_c) + row);
  };
  if (j.R > 0 && now.n > 0) pos = position(j, (int)now.tok);
  load_cs(now);
  int get = 0;
  for (unsigned t0 = blk * kGroups; t0 < tasks; t0 += stride) {
    ln.factors(C, S, -1.f);
    T* d = now.d;
    const int n = now.n;
    place(t0 + stride, next);
    if (j.R > 0 && next.n > 0) pos = position(j, (int)next.tok);
#pragma unroll 1
    for (int i = 0; i < kHeads; i += kPair) {
      cp_async_wait<kRing - 2>();
      f2_t f[kPair][P], q[kPair][P], m[kPair][P];
      float ss[kPair], dot[kPair];
#pragma unroll
      for (int k = 0; k < kPair; ++k) {
        const uint4 x = ring[((get * kPair + k) * 2) * kThreads + threadIdx.x];
        const uint4 g = ring[((get * kPair + k) * 2 + 1) * kThreads + threadIdx.x];
        to_pairs<T>(x, f[k]);
        to_pairs<T>(g, q[k]);
        ln.mates(g, q[k], m[k]);
      }
      get = get + 1 == kRing ? 0 : get + 1;
      ahead();
      if (i + kPair >= kHeads) load_cs(next);
#pragma unroll
      for (int k = 0; k < kPair; ++k) {
        f2_t s2 = f2_zero(), d2 = f2_zero();
#pragma unroll
        for (int e = 0; e < P; ++e) {
          q[k][e] = f2_fma(q[k][e], C[e], f2_mul(m[k][e], S[e]));
          m[k][e] = f2_mul(q[k][e], w[e]);
          s2 = f2_fma(f[k][e], f[k][e], s2);
          d2 = f2_fma(m[k][e], f[k][e], d2);
        }
        ss[k] = pair_sum(s2);
        dot[k] = pair_sum(d2);
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          ss[k] += __shfl_xor_sync(0xffffffffu, ss[k], o);
          dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], o);
        }
#pragma unroll
      for (int k = 0; k < kPair; ++k) {
        const float r = rsqrtf(ss[k] * j.inv_D + j.eps);
        const float mean = dot[k] * r * j.inv_D;      // mean(g w xh)
        if (i + k < n) {
          const f2_t r2 = f2_pack(r, r), rm = f2_pack(-r * mean, -r * mean);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const f2_t xh = f2_mul(f[k][e], r2);
            dw[e] = f2_fma(q[k][e], xh, dw[e]);
            f[k][e] = f2_fma(xh, rm, f2_mul(m[k][e], r2));
          }
          ln.store(d, f[k]);
          d += sd.y.sh;
        }
      }
    }
    now = next;
  }
  cp_async_wait_all();
#pragma unroll
  for (int e = 0; e < P; ++e) f2_unpack(dw[e], red[grp][u * V + 2 * e], red[grp][u * V + 2 * e + 1]);
  __syncthreads();
  for (int d = threadIdx.x; d < j.D; d += kThreads) {
    float sum = 0.f;
    for (int k = 0; k < kGroups; ++k) sum += red[k][d];
    part[(int64_t)blockIdx.x * j.D + d] = sum;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd_scalar_kernel(const NormJob j, const int q_blocks,
                                                                   const int interleaved, float* __restrict__ part) {
  constexpr int kWarps = kThreads / 32, kE = kMaxD / 32;
  __shared__ float sx[kWarps][kMaxD], sg[kWarps][kMaxD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *f = sx[warp], *g = sg[warp];
  const bool is_k = (int)blockIdx.x >= q_blocks;
  const NormSide& sd = j.side[is_k];
  const int64_t nblk = is_k ? gridDim.x - q_blocks : q_blocks;
  const int64_t blk = is_k ? blockIdx.x - q_blocks : blockIdx.x;
  const int64_t rows = (int64_t)j.tokens * sd.N;
  const T* w = reinterpret_cast<const T*>(sd.w);
  float dw[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) dw[e] = 0.f;
  for (int64_t row = blk * kWarps + warp; row < rows; row += nblk * kWarps) {
    const int tok = (int)(row / sd.N), h = (int)(row - (int64_t)tok * sd.N);
    const int b = tok / j.S, s = tok - b * j.S;
    const T* x = reinterpret_cast<const T*>(sd.x.p) + sd.x.off(b, h, s);
    const T* dy = reinterpret_cast<const T*>(sd.dy.p) + sd.dy.off(b, h, s);
    T* dx = reinterpret_cast<T*>(const_cast<void*>(sd.y.p)) + sd.y.off(b, h, s);
    float ss = 0.f;
    for (int d = lane; d < j.D; d += 32) {
      const float v = Elem<T>::to_f32(x[d]);
      f[d] = v;
      ss = fmaf(v, v, ss);
      g[d] = Elem<T>::to_f32(dy[d]);
    }
    const float r = rsqrtf(row_sum<32>(ss) * j.inv_D + j.eps);
    __syncwarp();
    const int half = j.R / 2;
    const int64_t crow = j.R > 0 ? cache_row(j, position(j, tok)) * half : 0;
    for (int d = lane; d < half; d += 32) {
      const int i1 = interleaved ? 2 * d : d, i2 = interleaved ? 2 * d + 1 : d + half;
      turn(g[i1], g[i2], Elem<T>::to_f32(reinterpret_cast<const T*>(j.cos_c)[crow + d]),
           -Elem<T>::to_f32(reinterpret_cast<const T*>(j.sin_c)[crow + d]));
    }
    __syncwarp();
    float dot = 0.f;
    for (int d = lane; d < j.D; d += 32) dot = fmaf(g[d] * Elem<T>::to_f32(w[d]), f[d], dot);
    const float mean = row_sum<32>(dot) * r * j.inv_D;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int d = lane + 32 * e;
      if (d < j.D) {
        const float xh = f[d] * r;
        dw[e] = fmaf(g[d], xh, dw[e]);
        dx[d] = Elem<T>::from_f32(r * fmaf(-xh, mean, g[d] * Elem<T>::to_f32(w[d])));
      }
    }
    __syncwarp();
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kE; ++e) sx[warp][lane + 32 * e] = dw[e];
  __syncthreads();
  for (int d = threadIdx.x; d < j.D; d += kThreads) {
    float sum = 0.f;
    for (int k = 0; k < kWarps; ++k) sum += sx[k][d];
    part[(int64_t)blockIdx.x * j.D + d] = sum;
  }
}

// dw of one side: 32 channels per block, the side's partial rows spread over 32 warps.
template <typename T>
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, const int D, const int q_blocks,
                                                       const int blocks, T* __restrict__ dwq, T* __restrict__ dwk) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + lane;
  const bool is_k = blockIdx.y != 0;
  const int lo = is_k ? q_blocks : 0, hi = is_k ? blocks : q_blocks;
  float sum = 0.f;
  if (d < D)
    for (int p = lo + warp; p < hi; p += 32) sum += part[(int64_t)p * D + d];
  red[warp][lane] = sum;
  __syncthreads();
  const float v = row_sum<32>(red[lane][warp]);   // warp w sums channel w of the block
  const int dd = blockIdx.x * 32 + warp;
  if (lane == 0 && dd < D) (is_k ? dwk : dwq)[dd] = Elem<T>::from_f32(v);
}

// ---------------------------------------------------------------- host side

bool vec_view(const View& v, int V) {
  return ((uintptr_t)v.p & 15u) == 0 && v.sb % V == 0 && v.sh % V == 0 && v.ss % V == 0;
}

// Lanes per row: one 16-byte vector each, as a power of two; 0 when the row has more than a warp's.
template <typename T>
int lanes_per_row(const NormJob& j) {
  const int nv = j.D / (16 / (int)sizeof(T));
  int l = 4;
  while (l < nv) l *= 2;
  return l <= 32 ? l : 0;
}

template <typename T>
bool vec_ok(const NormJob& j, bool bwd) {
  constexpr int V = 16 / (int)sizeof(T);
  if (j.D % V || !lanes_per_row<T>(j) || (j.interleaved ? j.R % V : j.R % (2 * V))) return false;
  if (j.R && (((uintptr_t)j.cos_c | (uintptr_t)j.sin_c) & (j.interleaved ? 7u : 15u))) return false;
  for (const NormSide& s : j.side) {
    if (((uintptr_t)s.w & 15u) || !vec_view(s.x, V) || !vec_view(s.y, V) || (bwd && !vec_view(s.dy, V))) return false;
  }
  return true;
}

// Heads per lane group of the forward: four once that still leaves every SM 2048 threads, else one.
// (4096 tokens x 40 heads: two heads 25.3 us, four 21.3, eight as four, before the arithmetic was
// paired.)
int heads_per_group(const NormJob& j, int lpr) {
  const int64_t threads = (int64_t)j.tokens * (j.side[0].N + j.side[1].N) * lpr;
  return threads / 4 >= (int64_t)152 * 2048 ? 4 : 1;
}

int side_blocks(const NormJob& j, int side, int threads, int lpr, int hpg) {
  const int64_t tasks = (int64_t)j.tokens * ((j.side[side].N + hpg - 1) / hpg);
  return (int)((tasks + threads / lpr - 1) / (threads / lpr));
}

template <typename T, bool kInter, int LPR, int HPG>
cudaError_t run_fwd(const NormJob& j, cudaStream_t st) {
  const int qb = side_blocks(j, 0, kFwdThreads, LPR, HPG), kb = side_blocks(j, 1, kFwdThreads, LPR, HPG);
  norm_fwd_kernel<T, kInter, LPR, HPG><<<(unsigned)(qb + kb), kFwdThreads, 0, st>>>(j, qb);
  count_launch(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t finish_dw(const NormJob& j, float* part, const NormBwdBlocks& nb, cudaStream_t st) {
  norm_dw_kernel<T><<<dim3((unsigned)(j.D + 31) / 32, 2), 1024, 0, st>>>(part, j.D, nb.q, nb.q + nb.k,
                                                                         reinterpret_cast<T*>(j.side[0].dw),
                                                                         reinterpret_cast<T*>(j.side[1].dw));
  count_launch(1);
  return cudaGetLastError();
}

template <typename T, bool kInter, int LPR>
cudaError_t run_bwd(const NormJob& j, float* part, cudaStream_t st) {
  const NormBwdBlocks nb = norm_bwd_blocks(j.side[0].N, j.side[1].N, side_blocks(j, 0, kThreads, LPR, kHeads),
                                           side_blocks(j, 1, kThreads, LPR, kHeads));
  // per device: set at every call (the attribute belongs to the current context)
  cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<T, kInter, LPR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return e;
  norm_bwd_kernel<T, kInter, LPR><<<(unsigned)(nb.q + nb.k), kThreads, kRingBytes, st>>>(j, nb.q, part);
  count_launch(1);
  e = cudaGetLastError();
  return e == cudaSuccess ? finish_dw<T>(j, part, nb, st) : e;
}

template <typename T, bool kInter, int LPR>
cudaError_t run_lpr(const NormJob& j, float* part, cudaStream_t st) {
  if (part) return run_bwd<T, kInter, LPR>(j, part, st);
  return heads_per_group(j, LPR) == 4 ? run_fwd<T, kInter, LPR, 4>(j, st) : run_fwd<T, kInter, LPR, 1>(j, st);
}

template <typename T, bool kInter>
cudaError_t run_layout(const NormJob& j, float* part, cudaStream_t st) {
  switch (lanes_per_row<T>(j)) {
    case 4: return run_lpr<T, kInter, 4>(j, part, st);
    case 8: return run_lpr<T, kInter, 8>(j, part, st);
    case 16: return run_lpr<T, kInter, 16>(j, part, st);
    default: return run_lpr<T, kInter, 32>(j, part, st);
  }
}

template <typename T>
cudaError_t run_t(const NormJob& j, float* part, cudaStream_t st) {
  if (vec_ok<T>(j, part != nullptr))
    return j.interleaved ? run_layout<T, true>(j, part, st) : run_layout<T, false>(j, part, st);
  auto want = [&](int side) {
    return (int)std::min<int64_t>(((int64_t)j.tokens * j.side[side].N + 7) / 8, 1 << 20);
  };
  if (!part) {
    norm_fwd_scalar_kernel<T><<<(unsigned)(want(0) + want(1)), kThreads, 0, st>>>(j, j.interleaved);
    count_launch(1);
    return cudaGetLastError();
  }
  const NormBwdBlocks nb = norm_bwd_blocks(j.side[0].N, j.side[1].N, want(0), want(1));
  norm_bwd_scalar_kernel<T><<<(unsigned)(nb.q + nb.k), kThreads, 0, st>>>(j, nb.q, j.interleaved, part);
  count_launch(1);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? finish_dw<T>(j, part, nb, st) : e;
}

}  // namespace

cudaError_t launch_qk_norm(sdpa_dtype dt, const NormJob& j, float* part, cudaStream_t st) {
  switch (dt) {
    case SDPA_F32: return run_t<float>(j, part, st);
    case SDPA_F16: return run_t<__half>(j, part, st);
    default: return run_t<__nv_bfloat16>(j, part, st);
  }
}

cudaError_t take_norm_status(int* status) { return take_words(g_norm_status, status); }

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_norm)

}  // namespace sdpa
