// Appends the new keys and values of a ragged batch to a paged cache, the keys turned by the
// angle of their position on the way (the pairs of class RotaryEmbedding).
//
// A copy: every element is read once and written once.  A block takes kUnits * kThreads units of 32
// bytes: TPB whole tokens, or a part of one wide token.  Its threads first issue their loads,
// which depend on the token alone; meanwhile the block finds the tokens' sequences (a counting
// pass over the offsets by all threads), positions, pages and cache rows, one thread per token.
// A unit is two 16-byte vectors; in the split pair layout those of a rotated key are the two
// halves of the same pairs.  Rotations whose half is not a whole number of vectors take the
// scalar kernel.  12 ragged chunks of 12,000 tokens in all, 8 float16 heads of 64: 11.4 to 11.7 us
// (4.2 TB/s), without rotation 9.6 us (4.9 TB/s), float32 18.6 us (5.2 TB/s); the scalar kernel 43.8
// us.  64 single tokens 3.0 us.  A block's chain of four dependent loads (offsets, length, page,
// cos/sin row) starts anew for each block: its barrier is the longest stall (5.4 to 6.4 of the
// 19 warps that wait per issued instruction), with 60 % of the issue slots busy and DRAM at 25 % (what
// is written stays in L2).
#include <algorithm>

#include "paged.h"

namespace sdpa {

static __device__ int g_append_status[1];

namespace {

constexpr int kThreads = 128;      // (256: 12.0 us against 11.4 on 12,000 ragged tokens)
constexpr int kUnits = 1;        // units per thread (two took 12.3 us against 11.9 on 12,000 ragged tokens)
constexpr int kMaxTpb = 64;      // tokens per block

struct Slot {                    // where one token goes; page < 0: nowhere
  int page, slot;
  int64_t crow;
};

// First sequence whose rows end behind token t, counted by the whole block.
__device__ __forceinline__ int find_seq(const Paged& g, int t) {
  int b = 0;
  for (int base = 0; base < g.B; base += kThreads) {
    const int i = base + (int)threadIdx.x;
    const int c = __syncthreads_count(i < g.B && g.cu[i + 1] <= t);
    b += c;
    if (c < kThreads) break;
  }
  return b;
}

__device__ __forceinline__ Slot find_slot(const Paged& g, const PagedRot& rot, int t, int b) {
  Slot s{-1, 0, 0};
  if (g.cu) {
    while (b < g.B && g.cu[b + 1] <= t) ++b;
  } else {
    b = t / g.uniform;
  }
  if (b >= g.B) return s;                      // rows behind the last sequence
  bool bad = false;
  const SeqInfo q = seq_info(g, b, bad);
  const int pos = q.T - q.n + (t - q.t0);
  if (t < q.t0 || q.T < q.n || bad) {          // before the first sequence, or lengths that contradict
    atomicOr(g_append_status, kPagedBadLength);
    return s;
  }
  const int pg = page_div(g, pos);
  const int id = g.table[(int64_t)b * g.table_stride + pg];
  if (id < 0 || id >= g.num_pages) {
    atomicOr(g_append_status, kPagedBadPage);
    return s;
  }
  s.page = id;
  s.slot = pos - pg * g.page_size;
  if (rot.R) {
    int64_t row = pos;
    if (row >= rot.max_pos) {
      atomicOr(g_append_status, kPagedBadPosition);
      row = rot.max_pos - 1;
    }
    s.crow = row * (rot.R / 2);
  }
  return s;
}

template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const Paged g, const View k, const View v,
                                                                const PagedRot rot, const int tpb, const int ku,
                                                                const int vu) {
  constexpr int V = 16 / (int)sizeof(T);
  __shared__ Slot slots[kMaxTpb];
  const int per_tok = g.Nkv * (ku + vu);
  const int tok0 = blockIdx.x * tpb;
  const int u0 = blockIdx.y * (kThreads * kUnits);

  // this thread's units: token, tensor, head and channels
  int lt[kUnits], head[kUnits], c0[kUnits], c1[kUnits];
  bool isk[kUnits], turned[kUnits];
  uint4 a[kUnits], p[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int x = u0 + i * kThreads + (int)threadIdx.x;
    lt[i] = -1;
    const int t = x / per_tok;
    if (t >= tpb || tok0 + t >= g.tokens) continue;
    int r = x - t * per_tok;
    isk[i] = r < g.Nkv * ku;
    if (!isk[i]) r -= g.Nkv * ku;
    const int per = isk[i] ? ku : vu, D = isk[i] ? g.H : g.Hv;
    head[i] = r / per;
    const int u = r - head[i] * per;
    turned[i] = false;
    c0[i] = 2 * u * V;
    c1[i] = c0[i] + V;
    if (isk[i] && rot.R) {
      if (kInter) {
        turned[i] = c0[i] < rot.R;
      } else {
        const int urot = rot.R / (2 * V);
        turned[i] = u < urot;
        c0[i] = turned[i] ? u * V : rot.R + 2 * (u - urot) * V;
        c1[i] = turned[i] ? c0[i] + rot.R / 2 : c0[i] + V;
      }
    }
    if (c0[i] >= D) continue;
    if (c1[i] >= D) c1[i] = -1;
    lt[i] = t;
    const View& src = isk[i] ? k : v;
    const T* row = reinterpret_cast<const T*>(src.p) + src.off(0, head[i], tok0 + t);
    if (SDPA_IN_BOUNDS(head[i] < g.Nkv && c0[i] + V <= D && c1[i] + V <= D, 511)) {
      a[i] = *reinterpret_cast<const uint4*>(row + c0[i]);
      if (c1[i] >= 0) p[i] = *reinterpret_cast<const uint4*>(row + c1[i]);
    }
  }
  const int b0 = g.cu ? find_seq(g, tok0) : 0;
  if ((int)threadIdx.x < tpb && tok0 + (int)threadIdx.x < g.tokens)
    slots[threadIdx.x] = find_slot(g, rot, tok0 + threadIdx.x, b0);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (lt[i] < 0) continue;
    const Slot s = slots[lt[i]];
    if (s.page < 0) continue;
    if (turned[i]) {
      const T* cr = reinterpret_cast<const T*>(rot.cos_c) + s.crow;
      const T* sr = reinterpret_cast<const T*>(rot.sin_c) + s.crow;
      float f[2 * V];
      unpack16<T>(a[i], f);
      unpack16<T>(p[i], f + V);
      T* ea = reinterpret_cast<T*>(&a[i]);
      T* ep = reinterpret_cast<T*>(&p[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        // x1 cos - x2 sin and x2 cos + x1 sin, rounded once (the order of sdpa_rotary)
        const int ci = kInter ? c0[i] / 2 + e : c0[i] + e;
        if (kInter && 2 * ci >= rot.R) break;
        const float c = Elem<T>::to_f32(cr[ci]), sn = Elem<T>::to_f32(sr[ci]);
        const float x1 = kInter ? f[2 * e] : f[e], x2 = kInter ? f[2 * e + 1] : f[V + e];
        const T o1 = Elem<T>::from_f32(fmaf(x1, c, -x2 * sn)), o2 = Elem<T>::from_f32(fmaf(x2, c, x1 * sn));
        if (kInter) {
          T* d = (2 * e < V) ? ea + 2 * e : ep + 2 * e - V;
          d[0] = o1;
          d[1] = o2;
        } else {
          ea[e] = o1;
          ep[e] = o2;
        }
      }
    }
    const View& dst = isk[i] ? g.kp : g.vp;
    T* row = reinterpret_cast<T*>(const_cast<void*>(dst.p)) + dst.off(s.page, head[i], s.slot);
    if (SDPA_IN_BOUNDS(s.page < g.num_pages && s.slot >= 0 && s.slot < g.page_size, 512)) {
      *reinterpret_cast<uint4*>(row + c0[i]) = a[i];
      if (c1[i] >= 0) *reinterpret_cast<uint4*>(row + c1[i]) = p[i];
    }
  }
}

// One element or pair per step, one token per block.
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_append_scalar_kernel(const Paged g, const View k, const View v,
                                                                       const PagedRot rot) {
  __shared__ Slot slot;
  const int t = blockIdx.x;
  const int b0 = g.cu ? find_seq(g, t) : 0;
  if (threadIdx.x == 0) slot = find_slot(g, rot, t, b0);
  __syncthreads();
  const Slot s = slot;
  if (s.page < 0) return;
  const int half = rot.R / 2, per = half + g.H - rot.R;
  const T* cr = reinterpret_cast<const T*>(rot.cos_c) + s.crow;
  const T* sr = reinterpret_cast<const T*>(rot.sin_c) + s.crow;
  for (int x = threadIdx.x; x < g.Nkv * per; x += kThreads) {
    const int h = x / per, c = x - h * per;
    const T* in = reinterpret_cast<const T*>(k.p) + k.off(0, h, t);
    T* out = reinterpret_cast<T*>(const_cast<void*>(g.kp.p)) + g.kp.off(s.page, h, s.slot);
    if (c >= half) {
      out[rot.R + c - half] = in[rot.R + c - half];
      continue;
    }
    const int i1 = rot.interleaved ? 2 * c : c, i2 = rot.interleaved ? 2 * c + 1 : c + half;
    const float x1 = Elem<T>::to_f32(in[i1]), x2 = Elem<T>::to_f32(in[i2]);
    const float co = Elem<T>::to_f32(cr[c]), si = Elem<T>::to_f32(sr[c]);
    out[i1] = Elem<T>::from_f32(fmaf(x1, co, -x2 * si));
    out[i2] = Elem<T>::from_f32(fmaf(x2, co, x1 * si));
  }
  for (int x = threadIdx.x; x < g.Nkv * g.Hv; x += kThreads) {
    const int h = x / g.Hv, d = x - h * g.Hv;
    (reinterpret_cast<T*>(const_cast<void*>(g.vp.p)) + g.vp.off(s.page, h, s.slot))[d] =
        (reinterpret_cast<const T*>(v.p) + v.off(0, h, t))[d];
  }
}

template <typename T>
cudaError_t launch_t(const Paged& g, const View& k, const View& v, const PagedRot& rot, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  const bool vec = rot.R == 0 || (rot.interleaved ? rot.R % V == 0 : rot.R % (2 * V) == 0);
  if (!vec) {
    paged_append_scalar_kernel<T><<<(unsigned)g.tokens, kThreads, 0, st>>>(g, k, v, rot);
  } else {
    const bool split = rot.R && !rot.interleaved;
    const int ku = split ? rot.R / (2 * V) + ((g.H - rot.R) / V + 1) / 2 : (g.H / V + 1) / 2;
    const int vu = (g.Hv / V + 1) / 2;
    const int64_t per_tok = (int64_t)g.Nkv * (ku + vu);
    const int tpb = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxTpb, kThreads * kUnits / per_tok));
    const unsigned gy = (unsigned)((per_tok * tpb + kThreads * kUnits - 1) / (kThreads * kUnits));
    const dim3 grid((unsigned)((g.tokens + tpb - 1) / tpb), gy);
    if (rot.R && rot.interleaved)
      paged_append_kernel<T, true><<<grid, kThreads, 0, st>>>(g, k, v, rot, tpb, ku, vu);
    else
      paged_append_kernel<T, false><<<grid, kThreads, 0, st>>>(g, k, v, rot, tpb, ku, vu);
  }
  count_launch(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(sdpa_dtype dt, const Paged& g, const View& k, const View& v, const PagedRot& rot,
                                cudaStream_t st) {
  switch (dt) {
    case SDPA_F32: return launch_t<float>(g, k, v, rot, st);
    case SDPA_F16: return launch_t<__half>(g, k, v, rot, st);
    default: return launch_t<__nv_bfloat16>(g, k, v, rot, st);
  }
}

cudaError_t take_paged_append_status(int* status) { return take_words(g_append_status, status); }

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_append)

}  // namespace sdpa
