// kda_scan.cuh -- shared by the selective scan's forward and gradients: units
// of work, arguments, packed fp32 arithmetic.
#pragma once

#include <float.h>

#include "kda_layer.cuh"

namespace kda {
namespace scan {

// The tokens are one flat axis; a unit is one segment (at most seg_len tokens)
// of one sequence.  Dense: segs units per sequence.  Packed: the plan kernel
// has chosen seg_len (in the status block) and written seg_off[n], the units
// before sequence n; with one unit per sequence (a batch left whole) unit u is
// sequence order[u], the longest first.
struct Segments {
  const int32_t* cu;       // nullptr = dense
  const int32_t* seg_off;  // packed
  const int32_t* order;    // packed
  int num_seqs, T, seg_len, segs, units;
  int cut_above;           // packed: only a batch with a longer sequence is cut
  bool wide;               // the outputs' kernel: two channels a thread
};

struct Unit {
  int n;             // sequence
  int slot;          // index of the segment's states, in token order
  int64_t t0, t1;    // its tokens
  bool first, last;  // of its sequence
  bool cut;          // the batch has sequences of several segments
  bool valid;
};

__device__ __forceinline__ Unit resolve(const Segments& m, StatusBlock* sb, int unit) {
  Unit u;
  int64_t start, end;
  int k, len = m.seg_len;
  if (m.cu) {
    const int all = __ldg(m.seg_off + m.num_seqs);
    u.valid = unit < all;
    if (!u.valid) return u;
    len = sb->pad[0];
    u.n = all == m.num_seqs ? __ldg(m.order + unit) : find_range(m.seg_off, m.num_seqs, unit);
    const int before = __ldg(m.seg_off + u.n);
    k = all == m.num_seqs ? 0 : unit - before;
    u.slot = before + k;
    u.last = u.slot + 1 == __ldg(m.seg_off + u.n + 1);
    start = __ldg(m.cu + u.n);
    end = __ldg(m.cu + u.n + 1);
  } else {
    u.valid = true;
    u.n = unit / m.segs;
    k = unit - u.n * m.segs;
    u.slot = unit;
    u.last = k == m.segs - 1;
    start = (int64_t)u.n * m.T;
    end = start + m.T;
  }
  u.first = k == 0;
  u.cut = m.cu ? len < m.T : m.segs > 1;
  u.t0 = start + (int64_t)k * len;
  u.t1 = u.last ? end : u.t0 + len;
  if (m.cu)
    u.valid = in_bounds(sb, u.t1, (int64_t)m.T + 1, kSiteScanUnitRows) &&
              in_bounds(sb, u.t0, u.t1 + 1, kSiteScanUnitRows) &&
              in_bounds(sb, u.slot, m.units, kSiteScanSlot);
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
  int D, S, G;
  Segments seg;
  bool split;     // some sequence may have more than one segment (Unit::cut: has)
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
  float* ckpt;     // [tiles][D][S]: the segment's own states in front of every kStep tokens
  float* ckpt_dt;  // [tiles][D]: its sum of dt up to there
  float* dbc_part; // [channel blocks][tokens][2][S]: dBm, dCm summed over a channel block
  float* da_part;  // [units][D][S]
  float* dd_part;  // [units][2][D]: dD_skip, ddelta_bias
};

constexpr int kStep = 8;  // tokens between the states kept for the gradients

// first checkpoint slot of a unit: units lie in token order by slot, so the
// ranges do not meet
__device__ __forceinline__ int64_t first_tile(const Unit& u) { return u.t0 / kStep + u.slot; }

// A block's channels: block cb of the per_group blocks of each group
struct Channels {
  int g, d0, n;
};
template <int CT>
__device__ __forceinline__ Channels channels_of(const Args& a, int cb) {
  const int Dg = a.D / a.G, per = (Dg + CT - 1) / CT;
  Channels c;
  c.g = cb / per;
  const int k = cb - c.g * per;
  c.d0 = c.g * Dg + k * CT;
  c.n = min(CT, Dg - k * CT);
  return c;
}
inline int channel_blocks(int D, int G, int CT) { return G * ((D / G + CT - 1) / CT); }

// The decay e^{dt A} as 2^(dt A2 + kNudge), A2 = A log2 e.  Over a state's memory
// of 1 / (dt |A|) tokens a mean error of the exponential adds up where its
// scatter does not, and the unit's results lie 2.0e-8 of themselves low on
// average for decays of 0.001 to 1 (measured on a B200 over 8 M values a decade;
// rms error 3.7e-8): the exponent is raised by that much.  dt = 0 still gives
// exactly 1.
constexpr float kNudge = 2.9e-8f;
// A log2 e.  Where that is -inf (a state that keeps nothing) it is the lowest
// finite value: the tokens behind a segment's end have dt = 0, and 0 * inf would
// be NaN; any dt above 2^-120 still gives 0.
__device__ __forceinline__ float rate2(float A) {
  float r;  // NaN stays NaN
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(A * kLog2e), "f"(-FLT_MAX));
  return r;
}
__device__ __forceinline__ float decay(float dt, float A2) { return ex2(fmaf(dt, A2, kNudge)); }
__device__ __forceinline__ f2 decay_exp(f2 dt, f2 A2) {
  return fma2(dt, A2, pack2(kNudge, kNudge));
}

// log(1 + u) for 0 <= u <= 1 as u P(u): P is the polynomial of degree 8 with
// P(0) = 1 nearest to log(1 + u) / u in relative error (weighted least squares on
// 4000 Chebyshev points, the weights raised where the error is largest until it
// is level; each coefficient rounded to fp32 from the lowest on, the others
// fitted again behind it).  With these coefficients it is off by 3.4e-8 at most,
// by 1.5e-7 with the fp32 rounding of the evaluation, and by 1e-9 on average.
// P(0) = 1, so a small u passes exactly: steps of 0.001 come from such u, and a
// constant term of 1 - 2^-24 would make every one of them too short.  log2 of the
// rounded sum 1 + u would lose their relative accuracy.
__device__ __forceinline__ f2 log1p_unit(f2 u) {
  f2 p = pack2(0.005365422461181879f, 0.005365422461181879f);
  p = fma2(p, u, pack2(-0.030068300664424896f, -0.030068300664424896f));
  p = fma2(p, u, pack2(0.07920882850885391f, 0.07920882850885391f));
  p = fma2(p, u, pack2(-0.13754187524318695f, -0.13754187524318695f));
  p = fma2(p, u, pack2(0.1915384829044342f, 0.1915384829044342f));
  p = fma2(p, u, pack2(-0.24857217073440552f, -0.24857217073440552f));
  p = fma2(p, u, pack2(0.33321329951286316f, 0.33321329951286316f));
  p = fma2(p, u, pack2(-0.49999648332595825f, -0.49999648332595825f));
  p = fma2(p, u, pack2(1.0f, 1.0f));
  return mul2(p, u);
}

// dt from the raw steps: log(1 + e^v) = max(v, 0) + log1p(e^-|v|), two at a time
template <int V>
__device__ __forceinline__ void step_sizes(float (&v)[V], bool softplus) {
  if (!softplus) return;
#pragma unroll
  for (int j = 0; j < V; j += 2) {
    const float b = V > 1 ? v[V > 1 ? j + 1 : 0] : 0.f;
    float p, q;
    unpack2(log1p_unit(pack2(ex2(-kLog2e * fabsf(v[j])), ex2(-kLog2e * fabsf(b)))), p, q);
    v[j] = fmaxf(v[j], 0.f) + p;
    if (V > 1) v[V > 1 ? j + 1 : 0] = fmaxf(b, 0.f) + q;
  }
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

// The rows of dt and u: per token an entry of 4 floats (dt, dt', u, u') for two
// neighbouring channels, or of 2 floats (dt, u) for one.  Rows of pairs are 16
// floats longer than their entries, and every second eight entries change
// places in pairs: so the fills (lanes two entries apart), the scan's reads
// (lanes one entry apart) and the sums of four tokens, stored in the first
// half of an entry for the first two and in the second half for the others,
// meet no bank twice.
template <int SC, int CT>
constexpr int kDuRow = SC == 2 ? 2 * CT + 16 : 2 * CT;

// entry of the channel (pair) that starts at channel c of the CTA
template <int SC>
__device__ __forceinline__ int du_entry(int c) {
  if constexpr (SC == 1) return 2 * c;
  const int cp = c >> 1;
  return 4 * (cp ^ ((cp >> 3) & 1));
}

// dt and u of V channels from c on
template <int SC, int V>
__device__ __forceinline__ void store_du(float* row, int c, const float (&dt)[V],
                                         const float (&u)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += SC) {
    float* p = row + du_entry<SC>(c + j);
    if constexpr (SC == 2)
      *reinterpret_cast<float4*>(p) = make_float4(dt[j], dt[j + 1], u[j], u[j + 1]);
    else
      *reinterpret_cast<float2*>(p) = make_float2(dt[j], u[j]);
  }
}
template <int SC>
__device__ __forceinline__ void load_du(const float* entry, float (&dt)[SC], float (&u)[SC]) {
  if constexpr (SC == 2) {
    const float4 v = *reinterpret_cast<const float4*>(entry);
    dt[0] = v.x; dt[1] = v.y; u[0] = v.z; u[1] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(entry);
    dt[0] = v.x; u[0] = v.y;
  }
}

// The sums of tokens t4 .. t4 + 3 (t4 a multiple of 4) over a channel's lanes,
// to the channels' entries of those tokens, P floats between tokens.
template <int SC, int LN, int P>
__device__ __forceinline__ void store_sums(float* entry, const float (&v)[SC][4], int l) {
  float2 r[SC];
#pragma unroll
  for (int q = 0; q < SC; ++q) r[q] = sum_lanes<LN>(v[q], l);
  if constexpr (SC == 2) {
    static_assert(LN >= 4, "8 states have one channel a thread");
    if (l < 4)
      *reinterpret_cast<float2*>(entry + l * P + (l & 2)) = make_float2(r[0].x, r[1].x);
  } else {
    if constexpr (LN == 2) {
      entry[2 * l * P] = r[0].x;
      entry[2 * l * P + P] = r[0].y;
    } else if (l < 4) {
      entry[l * P] = r[0].x;
    }
  }
}
// what store_sums has put there, of V channels from c on of token t
template <int SC, int V>
__device__ __forceinline__ void load_sums(const float* row, int c, int t, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += SC) {
    const float* p = row + du_entry<SC>(c + j);
    if constexpr (SC == 2) {
      const float2 f = *reinterpret_cast<const float2*>(p + (t & 2));
      v[j] = f.x;
      v[j + 1] = f.y;
    } else {
      v[j] = *p;
    }
  }
}

// ------------------------------------------------------------------- host
// Tokens per segment, the units of a batch (kda_scan.cu).
Segments plan_segments(const int32_t* cu, int num_seqs, int B, int T, int D, int S, bool bwd);
bool sizes_ok(int D, int S, int G);
// a packed batch has up to num_seqs + T / kMinSeg units, a 32-bit count
constexpr int kMinSeg = 64;
inline bool units_ok(int num_seqs, int T) { return (int64_t)num_seqs + T / kMinSeg <= kMaxRows; }
inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// Packed batches: validates the offsets, chooses seg_len and writes seg_off and
// order (both [num_seqs + 1]).
cudaError_t launch_scan_plan(const Args& a, int32_t* seg_off, int32_t* order, cudaStream_t st);

// Each segment's own end state (h_seg) and sum of dt, with g_seg the state
// gradient its outputs send to its start, with ckpt its states on the way; then
// with split their combination into incoming h_seg and g_seg.
cudaError_t launch_ends(const Args& a, kda_dtype dt, cudaStream_t st);

kda_status check_scan(kda_dtype dt, int D, int S, int G, int64_t xs, int64_t ds, int64_t bs,
                      int64_t cs, const void* z, int64_t zs);
Args scan_args(const void* x, int64_t x_stride, const void* delta, int64_t delta_stride,
               const float* A, const void* Bm, int64_t B_stride, const void* Cm,
               int64_t C_stride, const float* D_skip, const void* z, int64_t z_stride,
               const float* delta_bias, int delta_softplus, int D, int S, int G);

}  // namespace scan
}  // namespace kda
