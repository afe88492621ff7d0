// Appends new keys and values to a paged cache of 4 bits a value, the keys turned by the angle of
// their position on the way (the pairs of class RotaryEmbedding) and rounded to their type.
//
// Per 32 channels: m = min, s = (max - min) / 15 rounded to the type, code = round((x - m) / s) to the
// nearest, ties to even, at most 15; s and m are what the cache holds, so a code makes up for their
// rounding.  All in fp32 with one rounding an operation (no contracted products), which makes the
// record a function of the input alone.  A group with a value that is not finite, or whose spread
// is not, takes a scale and a minimum that are no numbers: it reads as NaN.
//
// Every element is read once and written once at 5/8 byte (and once more, as the cache holds it, where the
// caller wants that). A thread has 8 channels, four lanes a group. The slot and the position of a token are one
// load each: they are made once a step and serve every layer. Bound by instructions (420 a warp of 256 values,
// 72 % of the issue slots) and by waits for loads: two prompts of 2048 tokens, 8 bfloat16 heads of 128, rows as held wanted,
// 17.3 us (2.3 TB/s; 14.1 without rotation, float32 17.9), 12,000 ragged tokens of float16 heads of 64 21.9 us, 64 single
// tokens 2.9 us. Without the rows as held the prompts take 14.6 us for 15.7, the chunks 19.0 for 20.3 (one set of inputs).
#include <algorithm>
#include <type_traits>

#include "paged4.h"
#include "paged_sched.cuh"

namespace sdpa {

static __device__ int g_append4_status[1];

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ int fast_div(int x, uint32_t mul, uint32_t shift) {
  return (int)(((uint64_t)(uint32_t)x * mul) >> shift);
}

// A row's place: strides below 2^31, as nearly all are, take one multiplication each.
template <bool kWide>
__device__ __forceinline__ int64_t place(const View& v, int head, int at) {
  if constexpr (kWide) return v.off(0, head, at);
  else return (int64_t)head * (int)v.sh + (int64_t)at * (int)v.ss;
}

// Channels of a thread, four threads a group (with 16, two prompts of 2048 took 22.5 us against 19.3).
constexpr int kCh = 8;

template <typename T>
__device__ __forceinline__ void load_ch(const T* p, float* f) {
  constexpr int V = Elem<T>::kVec;
#pragma unroll
  for (int i = 0; i < kCh / V; ++i) unpack16<T>(reinterpret_cast<const uint4*>(p)[i], f + i * V);
}

// The next smaller value of the type below x > 0.
template <typename T>
__device__ __forceinline__ float step_down(float x) {
  if constexpr (sizeof(T) == 4) return __int_as_float(__float_as_int(x) - 1);
  else {
    T v = Elem<T>::from_f32(x);
    *reinterpret_cast<uint16_t*>(&v) -= 1;
    return Elem<T>::to_f32(v);
  }
}
template <typename T>
__device__ __forceinline__ auto pair_of(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) return __floats2half2_rn(a, b);
  else return __floats2bfloat162_rn(a, b);
}
// Scales from here on are as exact as the type's normal numbers.
template <typename T>
__device__ __forceinline__ float least_scale() { return std::is_same<T, __half>::value ? 0x1p-14f : 1e-30f; }
template <typename T>
__device__ __forceinline__ float largest() {
  if constexpr (std::is_same<T, __half>::value) return 65504.f;
  else if constexpr (sizeof(T) == 2) return __int_as_float(0x7f7f0000);
  else return __int_as_float(0x7f7fffff);
}

template <typename T>
__device__ __forceinline__ float rounded(float x) { return Elem<T>::to_f32(Elem<T>::from_f32(x)); }

// Channels [c0, c0 + 8) of a key turned.  Whole vectors of pairs (vec_rot), or pair by pair.
template <typename T, bool kInter>
__device__ __forceinline__ void turn(const Paged4Append& a, const T* row, int c0, int64_t crow, float* x) {
  const int half = a.R / 2;
  const T* cr = reinterpret_cast<const T*>(a.cos_c) + crow;
  const T* sr = reinterpret_cast<const T*>(a.sin_c) + crow;
  if constexpr (kInter) {
#pragma unroll
    for (int e = 0; e < kCh; e += 2) {
      const int i = (c0 + e) / 2;
      if (c0 + e >= a.R) break;
      const float c = Elem<T>::to_f32(cr[i]), s = Elem<T>::to_f32(sr[i]);
      const float x1 = x[e], x2 = x[e + 1];
      x[e] = rounded<T>(__fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s)));
      x[e + 1] = rounded<T>(__fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s)));
    }
  } else if (a.vec_rot) {
    const bool low = c0 < half;
    const int i0 = low ? c0 : c0 - half;
    float o[kCh], c[kCh], s[kCh];
    load_ch<T>(row + (low ? c0 + half : i0), o);
    load_ch<T>(cr + i0, c);
    load_ch<T>(sr + i0, s);
#pragma unroll
    for (int e = 0; e < kCh; ++e) {
      // x cos - o sin in the lower half, x cos + o sin in the upper
      const float q = __fmul_rn(o[e], s[e]);
      x[e] = rounded<T>(__fadd_rn(__fmul_rn(x[e], c[e]), low ? -q : q));
    }
  } else {
#pragma unroll
    for (int e = 0; e < kCh; ++e) {
      const int ch = c0 + e;
      if (ch >= a.R) break;
      const bool low = ch < half;
      const int i = low ? ch : ch - half;
      const float p = __fmul_rn(x[e], Elem<T>::to_f32(cr[i]));
      const float q = __fmul_rn(Elem<T>::to_f32(row[low ? ch + half : i]), Elem<T>::to_f32(sr[i]));
      x[e] = rounded<T>(low ? __fsub_rn(p, q) : __fadd_rn(p, q));
    }
  }
}

template <typename T, bool kInter, bool kWide>
__global__ void __launch_bounds__(kThreads) paged4_append_kernel(const Paged4Append a, const int tpb) {
  const int ku = a.Nkv * (a.H / kCh), per_tok = ku + a.Nkv * (a.Hv / kCh);
  const int x0 = (int)blockIdx.y * kThreads + (int)threadIdx.x;
  const int lt = fast_div(x0, a.tok_mul, a.tok_shift), t = (int)blockIdx.x * tpb + lt;
  // the four lanes of a group have the same token, tensor and head
  const bool live = lt < tpb && t < a.tokens;
  int u = x0 - lt * per_tok;
  const bool isk = u < ku;
  if (!isk) u -= ku;
  const int D = isk ? a.H : a.Hv;
  const int head = isk ? fast_div(u, a.k_mul, a.k_shift) : fast_div(u, a.v_mul, a.v_shift), c0 = (u - head * (D / kCh)) * kCh;
  float x[kCh];
#pragma unroll
  for (int e = 0; e < kCh; ++e) x[e] = 0.f;
  int64_t slot = -1;
  if (live) {
    const View& src = isk ? a.k : a.v;
    const T* row = reinterpret_cast<const T*>(src.p) + place<kWide>(src, head, t);
    slot = a.slots[t];
    const bool turned = isk && c0 < a.R;
    int64_t pos = turned ? a.positions[t] : 0;
    if (SDPA_IN_BOUNDS(head < a.Nkv && c0 + kCh <= D, 571)) load_ch<T>(row + c0, x);
    if (turned) {
      // the place of a token that goes nowhere is not looked at
      if (slot >= 0 && (pos < 0 || pos >= a.max_pos)) atomicOr(g_append4_status, kPagedBadPosition);
      pos = min(max(pos, (int64_t)0), a.max_pos - 1);
      turn<T, kInter>(a, row, c0, pos * (a.R / 2), x);
    }
  }
  float lo, hi;
  if constexpr (sizeof(T) == 2) {
    // the values are numbers of the type: two at a time
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    T2 v[kCh / 2], l, h;
#pragma unroll
    for (int e = 0; e < kCh / 2; ++e) v[e] = pair_of<T>(x[2 * e], x[2 * e + 1]);
    l = h = v[0];
#pragma unroll
    for (int e = 1; e < kCh / 2; ++e) {
      l = __hmin2_nan(l, v[e]);
      h = __hmax2_nan(h, v[e]);
    }
    lo = min_nan(Elem<T>::to_f32(l.x), Elem<T>::to_f32(l.y));
    hi = max_nan(Elem<T>::to_f32(h.x), Elem<T>::to_f32(h.y));
  } else {
    lo = hi = x[0];
#pragma unroll
    for (int e = 1; e < kCh; ++e) {
      lo = min_nan(lo, x[e]);
      hi = max_nan(hi, x[e]);
    }
  }
#pragma unroll
  for (int o = 1; o < kQ4Group / kCh; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!live || slot < 0) return;
  if (slot >= (int64_t)a.num_pages * a.page_size) {
    atomicOr(g_append4_status, kPagedBadSlot);
    return;
  }
  const float spread = hi - lo;
  float s = rounded<T>(__fdiv_rn(spread, 15.f));
  // a scale rounded up at the end of the type's range: code 15 would have no value
  if (fmaf(15.f, s, lo) > largest<T>()) s = step_down<T>(s);
  if (!(spread < INFINITY)) s = lo = __int_as_float(0x7fffffff);
  // The quotient by the reciprocal is off by 2^-22 of itself at most, and its integer is the code unless the
  // remainder is half a scale but for that much.  There the remainder, which is exact, decides: more than half a scale is the
  // next code's, half a scale the even one's.  A remainder within 2^-18 of a half but no half leaves it to the
  // division's rounding; so do scales that are no ordinary numbers of the type (whose quotients may pass 15).
  constexpr float kInt = 12582912.f;         // 1.5 2^23: a sum with it is rounded to an integer, the even one at a tie
  const bool ordinary = s >= least_scale<T>() && s < 1e30f;
  const float inv = ordinary ? __frcp_rn(s) : 0.f, near = ordinary ? 0.4999f * s : -1.f;
  float code[kCh];
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < kCh; ++e) {
    const float d = x[e] - lo;
    float i = fmaf(d, inv, kInt);
    code[e] = i - kInt;
    const float r = fmaf(-code[e], s, d);
    if (!(fabsf(r) < near)) {
      const float over = fabsf(r) - 0.5f * s;
      if (ordinary && (over == 0.f || fabsf(over) > 0x1p-18f * s)) {
        if (over > 0.f || (over == 0.f && (__float_as_uint(i) & 1u))) i += r > 0.f ? 1.f : -1.f;
      } else {
        i = (s > 0.f ? fminf(__fdiv_rn(d, s), 15.f) : 0.f) + kInt;      // 0: a constant group, or one that is not a number
      }
      code[e] = i - kInt;
    }
    // the integer is in i's last bits: those above belong to 1.5 2^23
    word += __float_as_uint(i) << (4 * e);
  }
  word -= 0x4b400000u * 0x11111111u;
  const uint64_t page = slot < (1ll << 31) ? (uint64_t)fast_div((int)slot, a.page_mul, a.page_shift) : (uint64_t)slot / (uint32_t)a.page_size;
  const int at = (int)(slot - (int64_t)page * a.page_size);
  const View& dst = isk ? a.kp : a.vp;
  unsigned char* rec = reinterpret_cast<unsigned char*>(const_cast<void*>(dst.p)) + (int64_t)page * dst.sb + place<kWide>(dst, head, at);
  if (SDPA_IN_BOUNDS((int64_t)page < a.num_pages && at >= 0 && at < a.page_size, 572)) {
    *reinterpret_cast<uint32_t*>(rec + c0 / 2) = word;
    if (c0 % kQ4Group == 0) {
      T* side = reinterpret_cast<T*>(rec + D / 2) + c0 / kQ4Group * 2;
      if constexpr (sizeof(T) == 4) {
        side[0] = lo;
        side[1] = s;
      } else {
        T pair[2] = {Elem<T>::from_f32(lo), Elem<T>::from_f32(s)};
        *reinterpret_cast<uint32_t*>(side) = *reinterpret_cast<const uint32_t*>(pair);
      }
    }
  }
  const View& held = isk ? a.k_held : a.v_held;
  if (held.p) {
    T out[kCh];
#pragma unroll
    for (int e = 0; e < kCh; ++e) out[e] = Elem<T>::from_f32(fmaf(code[e], s, lo));      // the product alone may pass fp32
    uint4* h = reinterpret_cast<uint4*>(reinterpret_cast<T*>(const_cast<void*>(held.p)) + place<kWide>(held, head, t) + c0);
#pragma unroll
    for (int i = 0; i < kCh / Elem<T>::kVec; ++i) h[i] = reinterpret_cast<const uint4*>(out)[i];
  }
}

template <typename T>
cudaError_t launch_t(Paged4Append a, cudaStream_t st) {
  const int64_t per_tok = (int64_t)a.Nkv * ((a.H + a.Hv) / kCh);
  const int tpb = (int)std::max<int64_t>(1, std::min<int64_t>(64, kThreads / per_tok));
  const dim3 grid((unsigned)((a.tokens + tpb - 1) / tpb), (unsigned)((per_tok * tpb + kThreads - 1) / kThreads));
  paged_magic((int)per_tok, &a.tok_mul, &a.tok_shift);
  paged_magic(a.H / kCh, &a.k_mul, &a.k_shift);
  paged_magic(a.Hv / kCh, &a.v_mul, &a.v_shift);
  paged_magic(a.page_size, &a.page_mul, &a.page_shift);
  bool wide = false;
  for (const View* v : {&a.k, &a.v, &a.k_held, &a.v_held, &a.kp, &a.vp}) wide = wide || v->sh >= (1ll << 31) || v->ss >= (1ll << 31);
  const bool inter = a.R && a.interleaved;
  auto* kernel = wide ? (inter ? paged4_append_kernel<T, true, true> : paged4_append_kernel<T, false, true>)
                      : (inter ? paged4_append_kernel<T, true, false> : paged4_append_kernel<T, false, false>);
  kernel<<<grid, kThreads, 0, st>>>(a, tpb);
  count_launch(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged4_append(sdpa_dtype dt, const Paged4Append& a, cudaStream_t st) {
  switch (dt) {
    case SDPA_F32: return launch_t<float>(a, st);
    case SDPA_F16: return launch_t<__half>(a, st);
    default: return launch_t<__nv_bfloat16>(a, st);
  }
}

cudaError_t take_paged4_append_status(int* status) { return take_words(g_append4_status, status); }

SDPA_DEFINE_BOUNDS_TAKE(take_bounds_paged4_append)

}  // namespace sdpa
