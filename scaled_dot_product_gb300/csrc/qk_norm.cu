// RMS norm of every query and key head followed by the position rotation, in one pass, and its
// gradient.  With r = (mean(x^2) + eps)^-1/2 over the D channels of a head and u = x r w:
//
//     y  = Rot(u)                                   (the pairs of class RotaryEmbedding)
//     g  = Rot^T(dy),  dw = sum over rows of g x r,  dx = r (g w - x r mean(g w x r))
//
// All arithmetic is fp32; each output is rounded once to the element type.
//
// Bytes bound both directions: x (and dy) are read once and y (dx) is written once.  LPR lanes
// share one row; a lane holds two 16-byte vectors, in the split pair layout the two halves of
// the same pairs, so the rotation needs no exchange between lanes and the row's sum is a
// shuffle over LPR lanes.  One group of lanes takes HPG heads of one token, so the cos/sin row
// and the weights are read once for them and HPG x 32 bytes are in flight per lane.
// Shapes or pointers that do not allow 16-byte vectors take the scalar kernels (one warp per
// row, the row in shared memory).
#include <algorithm>

#include "internal.h"

namespace sdpa {

static __device__ int g_norm_status;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 256;

// Cache row of token (b, s); rows outside the cache are recorded and clamped.
__device__ __forceinline__ int64_t cache_row(const NormJob& j, int tok) {
  int64_t row = tok;
  if (j.positions) row = j.positions[tok];
  if (row < 0 || row >= j.max_pos) {
    atomicExch(&g_norm_status, 1);
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

// The two vectors a lane owns: their first channels (-1: none) and whether they are rotated.
template <typename T, bool kInter>
struct Lane {
  static constexpr int V = 16 / (int)sizeof(T);
  int c0, c1;
  bool rot0, rot1;
  __device__ __forceinline__ Lane(int u, int D, int R) {
    if (kInter) {
      c0 = 2 * u * V;
      c1 = c0 + V;
      rot0 = c0 < R;
      rot1 = c1 < R;
    } else {
      const int urot = R / (2 * V);
      rot0 = rot1 = u < urot;
      c0 = rot0 ? u * V : R + 2 * (u - urot) * V;
      c1 = rot0 ? c0 + R / 2 : c0 + V;
    }
    if (c0 >= D) { c0 = -1; rot0 = false; }
    if (c1 >= D) { c1 = -1; rot1 = false; }
  }
  // cos / sin of the lane's V pairs
  __device__ __forceinline__ void load_cs(const T* cr, const T* sr, float* c, float* s) const {
    if (kInter) {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        c[e] = rot0 ? Elem<T>::to_f32(cr[c0 / 2 + e]) : 1.f;
        s[e] = rot0 ? Elem<T>::to_f32(sr[c0 / 2 + e]) : 0.f;
        c[V / 2 + e] = rot1 ? Elem<T>::to_f32(cr[c1 / 2 + e]) : 1.f;
        s[V / 2 + e] = rot1 ? Elem<T>::to_f32(sr[c1 / 2 + e]) : 0.f;
      }
    } else if (rot0) {
      unpack16<T>(*reinterpret_cast<const uint4*>(cr + c0), c);
      unpack16<T>(*reinterpret_cast<const uint4*>(sr + c0), s);
    }
  }
  // f: the lane's 2V channels in place; sgn = -1 turns back
  __device__ __forceinline__ void rotate(float* f, const float* c, const float* s, float sgn) const {
    if (kInter) {
      if (rot0 || rot1) {
#pragma unroll
        for (int e = 0; e < V; ++e) turn(f[2 * e], f[2 * e + 1], c[e], sgn * s[e]);
      }
    } else if (rot0) {
#pragma unroll
      for (int e = 0; e < V; ++e) turn(f[e], f[V + e], c[e], sgn * s[e]);
    }
  }
};

template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int c) {
  return c >= 0 ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, int c, const float* f) {
  if (c < 0) return;
  constexpr int V = 16 / (int)sizeof(T);
  uint4 u;
  T* e = reinterpret_cast<T*>(&u);
#pragma unroll
  for (int x = 0; x < V; ++x) e[x] = Elem<T>::from_f32(f[x]);
  *reinterpret_cast<uint4*>(row + c) = u;
}

// ---------------------------------------------------------------- forward

template <typename T, bool kInter, int LPR, int HPG>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormJob j, const int q_blocks) {
  constexpr int V = 16 / (int)sizeof(T);
  const bool is_k = (int)blockIdx.x >= q_blocks;
  const NormSide& sd = j.side[is_k];
  const int chunks = (sd.N + HPG - 1) / HPG;
  const unsigned task = (blockIdx.x - (is_k ? q_blocks : 0)) * (unsigned)(kThreads / LPR) + threadIdx.x / LPR;
  const int u = threadIdx.x % LPR;
  const unsigned tok = task / (unsigned)chunks;
  const int h0 = (int)(task - tok * (unsigned)chunks) * HPG;
  const bool live = tok < (unsigned)j.tokens;
  const int b = live ? (int)(tok / (unsigned)j.S) : 0, s = live ? (int)(tok - (unsigned)b * (unsigned)j.S) : 0;
  const Lane<T, kInter> ln(u, j.D, j.R);
  const T* x0 = reinterpret_cast<const T*>(sd.x.p) + sd.x.off(b, h0, s);
  T* y0 = reinterpret_cast<T*>(const_cast<void*>(sd.y.p)) + sd.y.off(b, h0, s);
  const int nh = live ? min(HPG, sd.N - h0) : 0;

  uint4 xa[HPG], xb[HPG];
#pragma unroll
  for (int i = 0; i < HPG; ++i)
    if (i < nh && SDPA_IN_BOUNDS(b < j.B && h0 + i < sd.N && ln.c0 + V <= j.D && ln.c1 + V <= j.D, 501)) {
      xa[i] = load_vec(x0 + i * sd.x.sh, ln.c0);
      xb[i] = load_vec(x0 + i * sd.x.sh, ln.c1);
    } else {
      xa[i] = xb[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  float c[V], sn[V], w[2 * V];
  if (j.R > 0 && live) {
    const int64_t row = cache_row(j, (int)tok) * (j.R / 2);
    ln.load_cs(reinterpret_cast<const T*>(j.cos_c) + row, reinterpret_cast<const T*>(j.sin_c) + row, c, sn);
  }
  unpack16<T>(load_vec(reinterpret_cast<const T*>(sd.w), ln.c0), w);
  unpack16<T>(load_vec(reinterpret_cast<const T*>(sd.w), ln.c1), w + V);
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    float f[2 * V];
    unpack16<T>(xa[i], f);
    unpack16<T>(xb[i], f + V);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) ss = fmaf(f[e], f[e], ss);
    const float r = rsqrtf(row_sum<LPR>(ss) * j.inv_D + j.eps);
    if (i < nh) {
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) f[e] = f[e] * r * w[e];
      ln.rotate(f, c, sn, 1.f);
      store_vec(y0 + i * sd.y.sh, ln.c0, f);
      store_vec(y0 + i * sd.y.sh, ln.c1, f + V);
    }
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
    const int64_t crow = j.R > 0 ? cache_row(j, tok) * half : 0;
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
// accumulates dw for the one weight vector of its side.  Each block leaves its D sums in
// part[blockIdx.x]; norm_dw_kernel adds them in block order, so results do not vary from run
// to run.
template <typename T, bool kInter, int LPR, int HPG>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormJob j, const int q_blocks,
                                                            float* __restrict__ part) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int kGroups = kThreads / LPR;
  __shared__ float red[kGroups][LPR * 2 * V + 1];
  const bool is_k = (int)blockIdx.x >= q_blocks;
  const NormSide& sd = j.side[is_k];
  const unsigned nblk = is_k ? gridDim.x - q_blocks : q_blocks;
  const unsigned blk = is_k ? blockIdx.x - q_blocks : blockIdx.x;
  const unsigned chunks = (unsigned)(sd.N + HPG - 1) / HPG;
  const unsigned tasks = (unsigned)j.tokens * chunks;
  const int u = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const Lane<T, kInter> ln(u, j.D, j.R);
  float w[2 * V], dw[2 * V];
  unpack16<T>(load_vec(reinterpret_cast<const T*>(sd.w), ln.c0), w);
  unpack16<T>(load_vec(reinterpret_cast<const T*>(sd.w), ln.c1), w + V);
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) dw[e] = 0.f;

  // every thread of the block runs the same number of passes (the shuffles need whole warps)
  for (unsigned t0 = blk * kGroups; t0 < tasks; t0 += nblk * kGroups) {
    const unsigned task = t0 + grp;
    const bool live = task < tasks;
    const unsigned tok = live ? task / chunks : 0u;
    const int h0 = live ? (int)(task - tok * chunks) * HPG : 0;
    const int b = (int)(tok / (unsigned)j.S), s = (int)(tok - (unsigned)b * (unsigned)j.S);
    const int nh = live ? min(HPG, sd.N - h0) : 0;
    const T* x0 = reinterpret_cast<const T*>(sd.x.p) + sd.x.off(b, h0, s);
    const T* g0 = reinterpret_cast<const T*>(sd.dy.p) + sd.dy.off(b, h0, s);
    T* d0 = reinterpret_cast<T*>(const_cast<void*>(sd.y.p)) + sd.y.off(b, h0, s);
    uint4 xa[HPG], xb[HPG], ga[HPG], gb[HPG];
#pragma unroll
    for (int i = 0; i < HPG; ++i)
      if (i < nh && SDPA_IN_BOUNDS(b < j.B && h0 + i < sd.N && ln.c0 + V <= j.D && ln.c1 + V <= j.D, 502)) {
        xa[i] = load_vec(x0 + i * sd.x.sh, ln.c0);
        xb[i] = load_vec(x0 + i * sd.x.sh, ln.c1);
        ga[i] = load_vec(g0 + i * sd.dy.sh, ln.c0);
        gb[i] = load_vec(g0 + i * sd.dy.sh, ln.c1);
      } else {
        xa[i] = xb[i] = ga[i] = gb[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    float c[V], sn[V];
    if (j.R > 0 && live) {
      const int64_t row = cache_row(j, (int)tok) * (j.R / 2);
      ln.load_cs(reinterpret_cast<const T*>(j.cos_c) + row, reinterpret_cast<const T*>(j.sin_c) + row, c, sn);
    }
#pragma unroll
    for (int i = 0; i < HPG; ++i) {
      float f[2 * V], g[2 * V];
      unpack16<T>(xa[i], f);
      unpack16<T>(xb[i], f + V);
      unpack16<T>(ga[i], g);
      unpack16<T>(gb[i], g + V);
      if (i < nh) ln.rotate(g, c, sn, -1.f);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        ss = fmaf(f[e], f[e], ss);
        dot = fmaf(g[e] * w[e], f[e], dot);
      }
      const float r = rsqrtf(row_sum<LPR>(ss) * j.inv_D + j.eps);
      const float mean = row_sum<LPR>(dot) * r * j.inv_D;      // mean(g w xh)
      if (i < nh) {
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) {
          const float xh = f[e] * r;
          dw[e] = fmaf(g[e], xh, dw[e]);
          f[e] = r * fmaf(-xh, mean, g[e] * w[e]);
        }
        store_vec(d0 + i * sd.y.sh, ln.c0, f);
        store_vec(d0 + i * sd.y.sh, ln.c1, f + V);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) red[grp][u * 2 * V + e] = dw[e];
  __syncthreads();
  for (int x = threadIdx.x; x < LPR * 2 * V; x += kThreads) {
    float sum = 0.f;
    for (int g = 0; g < kGroups; ++g) sum += red[g][x];
    const Lane<T, kInter> lx(x / (2 * V), j.D, j.R);
    const int e = x % (2 * V);
    const int ch = e < V ? lx.c0 : lx.c1;
    if (ch >= 0) part[(int64_t)blockIdx.x * j.D + ch + (e < V ? e : e - V)] = sum;
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
    const int64_t crow = j.R > 0 ? cache_row(j, tok) * half : 0;
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

template <typename T>
bool vec_ok(const NormJob& j, bool bwd) {
  constexpr int V = 16 / (int)sizeof(T);
  if (j.D % V || (j.interleaved ? j.R % V : j.R % (2 * V))) return false;
  if (j.R && !j.interleaved && (((uintptr_t)j.cos_c | (uintptr_t)j.sin_c) & 15u)) return false;
  for (const NormSide& s : j.side) {
    if (((uintptr_t)s.w & 15u) || !vec_view(s.x, V) || !vec_view(s.y, V) || (bwd && !vec_view(s.dy, V))) return false;
  }
  return true;
}

// Lanes per row: the row's 16-byte vectors two to a lane, as a power of two.
template <typename T>
int lanes_per_row(const NormJob& j) {
  constexpr int V = 16 / (int)sizeof(T);
  const int nv = j.D / V;
  const int items = j.interleaved ? (nv + 1) / 2 : j.R / (2 * V) + ((j.D - j.R) / V + 1) / 2;
  int l = 4;
  while (l < items) l *= 2;
  return l;
}

// Heads per lane group: four once that still leaves every SM about 1024 threads, else one.
int heads_per_group(const NormJob& j, int lpr) {
  const int64_t threads = (int64_t)j.tokens * (j.side[0].N + j.side[1].N) * lpr;
  return threads / 4 >= (int64_t)152 * 1024 ? 4 : 1;
}

int side_blocks(const NormJob& j, int side, int lpr, int hpg) {
  const int64_t tasks = (int64_t)j.tokens * ((j.side[side].N + hpg - 1) / hpg);
  return (int)((tasks + kThreads / lpr - 1) / (kThreads / lpr));
}

template <typename T, bool kInter, int LPR, int HPG>
cudaError_t run_fwd(const NormJob& j, cudaStream_t st) {
  const int qb = side_blocks(j, 0, LPR, HPG), kb = side_blocks(j, 1, LPR, HPG);
  norm_fwd_kernel<T, kInter, LPR, HPG><<<(unsigned)(qb + kb), kThreads, 0, st>>>(j, qb);
  count_launch(1);
  return cudaGetLastError();
}

// Blocks of the persistent backward, split between the sides by their rows.
void bwd_blocks(const NormJob& j, int want_q, int want_k, int* qb, int* kb) {
  const int total = std::min(want_q + want_k, kNormBwdMaxBlocks);
  const double share = (double)j.side[1].N / (j.side[0].N + j.side[1].N);
  *kb = std::max(1, std::min(want_k, (int)(share * total + 0.5)));
  *qb = std::max(1, std::min(want_q, total - *kb));
}

template <typename T>
cudaError_t finish_dw(const NormJob& j, float* part, int qb, int kb, cudaStream_t st) {
  norm_dw_kernel<T><<<dim3((unsigned)(j.D + 31) / 32, 2), 1024, 0, st>>>(part, j.D, qb, qb + kb,
                                                                         reinterpret_cast<T*>(j.side[0].dw),
                                                                         reinterpret_cast<T*>(j.side[1].dw));
  count_launch(1);
  return cudaGetLastError();
}

template <typename T, bool kInter, int LPR, int HPG>
cudaError_t run_bwd(const NormJob& j, float* part, cudaStream_t st) {
  int qb, kb;
  bwd_blocks(j, side_blocks(j, 0, LPR, HPG), side_blocks(j, 1, LPR, HPG), &qb, &kb);
  norm_bwd_kernel<T, kInter, LPR, HPG><<<(unsigned)(qb + kb), kThreads, 0, st>>>(j, qb, part);
  count_launch(1);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? finish_dw<T>(j, part, qb, kb, st) : e;
}

template <typename T, bool kInter, int LPR>
cudaError_t run_lpr(const NormJob& j, float* part, cudaStream_t st) {
  const bool many = heads_per_group(j, LPR) == 4;
  if (part) return many ? run_bwd<T, kInter, LPR, 2>(j, part, st) : run_bwd<T, kInter, LPR, 1>(j, part, st);
  return many ? run_fwd<T, kInter, LPR, 4>(j, st) : run_fwd<T, kInter, LPR, 1>(j, st);
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
  int qb, kb;
  bwd_blocks(j, want(0), want(1), &qb, &kb);
  norm_bwd_scalar_kernel<T><<<(unsigned)(qb + kb), kThreads, 0, st>>>(j, qb, j.interleaved, part);
  count_launch(1);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? finish_dw<T>(j, part, qb, kb, st) : e;
}

}  // namespace

cudaError_t launch_qk_norm(sdpa_dtype dt, const NormJob& j, float* part, cudaStream_t st) {
  switch (dt) {
    case SDPA_F32: return run_t<float>(j, part, st);
    case SDPA_F16: return run_t<__half>(j, part, st);
    default: return run_t<__nv_bfloat16>(j, part, st);
  }
}

cudaError_t take_norm_status(int* status) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_norm_status, sizeof v);
  if (e != cudaSuccess) return e;
  *status = v;
  if (v) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_norm_status, &zero, sizeof zero);
  }
  return e;
}

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_norm)

}  // namespace sdpa
