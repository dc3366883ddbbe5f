// kda_layer.cuh -- what the operators around the recurrence share: argument
// checks (spans, strides), packed-batch lookup and element-vector io.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// ------------------------------------------------------------ host checks
struct Span {
  const void* p;
  int64_t bytes;
};

inline bool spans_overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

inline bool span_aligned(const Span& s) { return ((uintptr_t)s.p & 15u) == 0; }

// every span aligned; no output overlaps an input or another output
template <int NI, int NO>
kda_status check_spans(const Span (&ins)[NI], const Span (&outs)[NO]) {
  for (const Span& s : ins)
    if (!span_aligned(s)) return KDA_ERR_MISALIGNED;
  for (const Span& s : outs)
    if (!span_aligned(s)) return KDA_ERR_MISALIGNED;
  for (int o = 0; o < NO; ++o) {
    for (const Span& s : ins)
      if (spans_overlap(outs[o], s)) return KDA_ERR_INVALID_ARG;
    for (int p = 0; p < o; ++p)
      if (spans_overlap(outs[o], outs[p])) return KDA_ERR_INVALID_ARG;
  }
  return KDA_OK;
}

inline int64_t elem_bytes(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }

// bytes that `rows` rows of `width` elements, `stride` apart, span
inline int64_t row_bytes(int64_t rows, int64_t stride, int64_t width, int64_t esz) {
  return rows > 0 ? ((rows - 1) * stride + width) * esz : 0;
}

// a row stride covers the row, keeps 16-byte alignment and stays addressable
inline bool stride_ok(int64_t stride, int64_t width, int64_t esz) {
  return stride >= width && stride <= ((int64_t)1 << 31) && stride * esz % 16 == 0;
}

// B * T and the number of packed sequences are 32-bit counts, with room above
// them for a kernel's look-ahead
constexpr int64_t kMaxRows = 0x7fff0000LL;

// B, T and the packed batch's arguments
inline kda_status check_batch(const int32_t* cu, int num_seqs, int B, int T) {
  if (B <= 0 || T <= 0) return KDA_ERR_INVALID_ARG;
  if (cu) {
    if (B != 1 || num_seqs <= 0) return KDA_ERR_INVALID_ARG;
  } else if (num_seqs != 0 && num_seqs != B) {
    return KDA_ERR_INVALID_ARG;
  }
  if ((int64_t)B * T > kMaxRows || num_seqs > kMaxRows) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

// ---------------------------------------------------------- device helpers
// The last n in [0, N) with off[n] <= i, for off non-decreasing from 0 and
// i < off[N]: of empty ranges at i it skips all, so off[n] <= i < off[n + 1].
__device__ __forceinline__ int find_range(const int32_t* __restrict__ off, int N, int i) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(off + mid) <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// V consecutive elements as fp32 (16-byte loads where V allows); plain loads, since some
// callers write the same rows afterwards
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[V]);

template <>
__device__ __forceinline__ void load_vec<float, 1>(const float* p, float (&v)[1]) {
  v[0] = *p;
}
template <>
__device__ __forceinline__ void load_vec<float, 2>(const float* p, float (&v)[2]) {
  const float2 a = *(reinterpret_cast<const float2*>(p));
  v[0] = a.x; v[1] = a.y;
}
template <>
__device__ __forceinline__ void load_vec<float, 4>(const float* p, float (&v)[4]) {
  const float4 a = *(reinterpret_cast<const float4*>(p));
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
template <>
__device__ __forceinline__ void load_vec<float, 8>(const float* p, float (&v)[8]) {
  const float4 a = *(reinterpret_cast<const float4*>(p));
  const float4 b = *(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ float2 bf2_to_f2(uint32_t u) {
  // bf16 is the upper half of an fp32
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

template <>
__device__ __forceinline__ void load_vec<__nv_bfloat16, 2>(const __nv_bfloat16* p,
                                                           float (&v)[2]) {
  const float2 a = bf2_to_f2(*(reinterpret_cast<const uint32_t*>(p)));
  v[0] = a.x; v[1] = a.y;
}
template <>
__device__ __forceinline__ void load_vec<__nv_bfloat16, 4>(const __nv_bfloat16* p,
                                                           float (&v)[4]) {
  const uint2 u = *(reinterpret_cast<const uint2*>(p));
  const float2 a = bf2_to_f2(u.x), b = bf2_to_f2(u.y);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
template <>
__device__ __forceinline__ void load_vec<__nv_bfloat16, 8>(const __nv_bfloat16* p,
                                                           float (&v)[8]) {
  const uint4 u = *(reinterpret_cast<const uint4*>(p));
  const float2 a = bf2_to_f2(u.x), b = bf2_to_f2(u.y), c = bf2_to_f2(u.z), d = bf2_to_f2(u.w);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
}

__device__ __forceinline__ uint32_t f2_to_bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[V]) {
  if constexpr (V == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}
template <int V>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[V]) {
  if constexpr (V == 2) {
    *reinterpret_cast<uint32_t*>(p) = f2_to_bf2(v[0], v[1]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(f2_to_bf2(v[0], v[1]), f2_to_bf2(v[2], v[3]));
  } else {
    static_assert(V == 8, "vector width");
    *reinterpret_cast<uint4*>(p) = make_uint4(f2_to_bf2(v[0], v[1]), f2_to_bf2(v[2], v[3]),
                                              f2_to_bf2(v[4], v[5]), f2_to_bf2(v[6], v[7]));
  }
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^-x): e^-x = inf gives 0, NaN stays NaN.  The exponential is off by
// (2 + |x|) 2^-22 of itself at most (the unit and its rounded argument), the sum by
// 2^-24 and the reciprocal by 2^-23: below (3 + |x|) 2^-22 of the result, 2^-18.8
// for |x| <= 6.  That is far below a bf16 rounding (2^-8); fp32 results carry it,
// as the header says.
__device__ __forceinline__ float sigmoid_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + ex2(-kLog2e * x)));
  return y;
}

// two fp32 values side by side, one instruction for both
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
  float a, b;
  unpack2(v, a, b);
  return pack2(ex2(a), ex2(b));
}
__device__ __forceinline__ float sum2(f2 v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}
__device__ __forceinline__ f2 zero2() { return 0ull; }

// four consecutive floats as two pairs (16-byte aligned)
__device__ __forceinline__ void load_pairs(const float* p, f2 (&v)[2]) {
  const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(p);
  v[0] = u.x;
  v[1] = u.y;
}
__device__ __forceinline__ void store_pairs(float* p, const f2 (&v)[2]) {
  *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v[0], v[1]);
}

// sigmoid_fast of both
__device__ __forceinline__ f2 sigmoid2(f2 x) {
  float a, b;
  unpack2(add2(ex2_2(mul2(x, pack2(-kLog2e, -kLog2e))), pack2(1.f, 1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pack2(a, b);
}

// ------------------------------------------------------- asynchronous copies
// BYTES (4, 8 or 16) from global to shared memory without registers; zeros
// where !in (the source is not read then)
template <int BYTES>
__device__ __forceinline__ void copy_in(char* to, const void* from, bool in) {
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from),
                 "r"(in ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(from),
                 "n"(BYTES), "r"(in ? BYTES : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_issued() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copies_landed() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// all but the latest N committed groups of copies have landed
template <int N>
__device__ __forceinline__ void copies_landed_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// V elements of a slot as fp32
template <typename T, int V>
__device__ __forceinline__ void read_slot(const char* p, float (&v)[V]) {
  load_vec<T, V>(reinterpret_cast<const T*>(p), v);
}

// -------------------------------------------------------------- raw values
// V elements as they lie in memory, so that loads stay in flight until their
// first use
template <typename T, int V>
struct Raw {
  static constexpr int BYTES = V * (int)sizeof(T);
  static constexpr int N = BYTES / 4;
  static_assert(BYTES == 8 || BYTES % 16 == 0, "vector width");
  uint32_t r[N];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = 0;
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (BYTES == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      r[0] = u.x; r[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[i / 4];
        r[i] = u.x; r[i + 1] = u.y; r[i + 2] = u.z; r[i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r[i]);
    else return __uint_as_float(i & 1 ? r[i >> 1] & 0xffff0000u : r[i >> 1] << 16);
  }
};

}  // namespace kda
