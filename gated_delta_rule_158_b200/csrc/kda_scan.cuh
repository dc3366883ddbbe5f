// kda_scan.cuh -- shared by the selective scan's forward and gradients: thread
// layout, segments of long sequences, arguments.
#pragma once

#include "kda_layer.cuh"

namespace kda {
namespace scan {

constexpr float kLog2e = 1.4426950408889634f;

// A channel's S states lie in LN lanes, 4 a lane, so that a warp holds 32 / LN
// channels and every thread has four independent recurrences; a CTA of NT
// threads holds CT channels (32, or 16 at S = 128 where 32 would be 1024
// threads).
template <int S>
struct Layout {
  static constexpr int LN = S / 4;
  static constexpr int NT = LN * 32 > 512 ? 512 : LN * 32;
  static constexpr int CT = NT / LN;
};

inline int chan_tile(int S) { return S == 128 ? 16 : 32; }

// The tokens are one flat axis; a unit is one segment (at most seg_len tokens)
// of one sequence.  Dense: segs units per sequence.  Packed: seg_off[n] units
// before sequence n.
struct Segments {
  const int32_t* cu;       // nullptr = dense
  const int32_t* seg_off;  // packed
  int num_seqs, T, seg_len, segs, units;
};

struct Unit {
  int n, k;          // sequence, segment of it
  int64_t t0, t1;    // its tokens
  bool first, last;  // of its sequence
  bool valid;
};

__device__ __forceinline__ Unit resolve(const Segments& m, int unit) {
  Unit u;
  int64_t start, end;
  if (m.cu) {
    u.valid = unit < __ldg(m.seg_off + m.num_seqs);
    if (!u.valid) return u;
    u.n = find_range(m.seg_off, m.num_seqs, unit);
    u.k = unit - __ldg(m.seg_off + u.n);
    u.last = unit + 1 == __ldg(m.seg_off + u.n + 1);
    start = __ldg(m.cu + u.n);
    end = __ldg(m.cu + u.n + 1);
  } else {
    u.valid = true;
    u.n = unit / m.segs;
    u.k = unit - u.n * m.segs;
    u.last = u.k == m.segs - 1;
    start = (int64_t)u.n * m.T;
    end = start + m.T;
  }
  u.first = u.k == 0;
  u.t0 = start + (int64_t)u.k * m.seg_len;
  u.t1 = u.last ? end : u.t0 + m.seg_len;
  return u;
}

struct Args {
  const void* x;
  const void* delta;
  const void* Bm;
  const void* Cm;
  const void* z;
  int64_t x_stride, delta_stride, B_stride, C_stride, z_stride;
  const float* A;
  const float* D_skip;
  const float* delta_bias;
  bool softplus;
  const float* init;
  float* final_state;
  void* out;
  int D, S, G, nblk;
  Segments seg;
  float* h_seg;   // [units][D][S]: a segment's end state from zero, then its incoming state
  float* dt_sum;  // [units][D]: the segment's sum of dt
  StatusBlock* sb;
  // gradients
  const void* dout;
  const float* d_final;
  float* dx;
  float* ddelta;
  float* dz;
  float* d_init;
  float* g_seg;    // [units][D][S]: as h_seg, of the state gradient, from the right
  float* ckpt;     // [tokens / step][D][S]: states in front of every step-th token
  float* dbc_part; // [nblk][tokens][2][S]: dBm, dCm summed over a channel block
  float* da_part;  // [units][D][S]
  float* dd_part;  // [units][2][D]: dD_skip, ddelta_bias
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// dt from the raw step: log(1 + e^v) = max(v, 0) + log1p(e^-|v|)
__device__ __forceinline__ float step_size(float v, bool softplus) {
  return softplus ? fmaxf(v, 0.f) + log1pf(__expf(-fabsf(v))) : v;
}

// Sums of four tokens' values over the LN lanes of a channel.  LN >= 4: lane
// l & 3 returns token l & 3; LN = 2: lane l returns tokens 2 l and 2 l + 1.
template <int LN>
__device__ __forceinline__ float2 sum_lanes(const float (&v)[4], int l) {
  if constexpr (LN == 2) {
    const bool hi = l & 1;
    const float a = __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 1);
    const float b = __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 1);
    return make_float2((hi ? v[2] : v[0]) + a, (hi ? v[3] : v[1]) + b);
  } else {
    const bool hi = l & 2, odd = l & 1;
    const float a = __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 2);
    const float b = __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 2);
    const float p = (hi ? v[2] : v[0]) + a, q = (hi ? v[3] : v[1]) + b;
    float r = (odd ? q : p) + __shfl_xor_sync(0xffffffffu, odd ? p : q, 1);
#pragma unroll
    for (int o = 4; o < LN; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    return make_float2(r, 0.f);
  }
}

// Tokens per segment, the units of a batch, workspace rounding (kda_scan.cu).
Segments plan_segments(const int32_t* cu, int num_seqs, int B, int T, int D, int S);
bool sizes_ok(int D, int S, int G);
inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// The segments' local end states (and, with g_seg, state gradients at their
// starts) and their combination into h_seg, g_seg.
cudaError_t launch_ends(const Args& a, kda_dtype dt, cudaStream_t st);

kda_status check_scan(kda_dtype dt, int D, int S, int G, int64_t xs, int64_t ds, int64_t bs,
                      int64_t cs, const void* z, int64_t zs);
Args scan_args(const void* x, int64_t x_stride, const void* delta, int64_t delta_stride,
               const float* A, const void* Bm, int64_t B_stride, const void* Cm,
               int64_t C_stride, const float* D_skip, const void* z, int64_t z_stride,
               const float* delta_bias, int delta_softplus, int D, int S, int G);

}  // namespace scan
}  // namespace kda
