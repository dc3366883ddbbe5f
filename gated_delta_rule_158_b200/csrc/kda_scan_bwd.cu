// kda_scan_bwd.cu -- gradients of the selective state space scan.
//
// With dy the output's cotangent behind the gate (dout z sigmoid(z)), a_t =
// e^{dt_t A} and the state gradient g_t = dL/dh_t, from a sequence's end to its
// start
//   g_t = C_t dy_t + a_{t+1} g_{t+1},
//   dC_t = sum_d h_t dy_t,             dB_t = sum_d g_t dt_t x_t,
//   dx_t = dt_t sum_s g_t B_t + D dy_t,
//   d(dt)_t = sum_s g_t a_t h_{t-1} A + x_t sum_s g_t B_t,
//   dA = sum_t g_t a_t h_{t-1} dt_t.
// A CTA takes one segment of a sequence and CT channels.  It runs the states
// forward once, keeping the state in front of every tile (kStep tokens) in the
// workspace, then takes the tiles from last to first: the tile's states and
// decays again into registers, and the reverse recurrence over them.  Three
// sums over a channel's states go over its lanes (sum_lanes), the sums of dB
// and dC over channels over the other lanes, then over the CTA's warps in
// shared memory, and leave as one partial row per channel block; a second
// kernel adds those and the segments' parts of dA, dD and ddelta_bias in a
// fixed order.  Nothing is added atomically.
#include <math.h>

#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

// tokens per tile: their states and decays (8 values a token) are registers
template <int S>
constexpr int kStep = S <= 32 ? 16 : 8;

inline int step_of(int S) { return S <= 32 ? 16 : 8; }

template <int S>
struct Tile {
  using L = Layout<S>;
  static constexpr int T = kStep<S>, P = T + 4, W = L::NT / 32;
  static constexpr int kRows = L::CT * P;  // floats of one [channel][token] tile
  static constexpr size_t bytes() {
    return sizeof(float) * (3 * (size_t)kRows + 2 * T * S + (size_t)W * T * 2 * S);
  }
};

// position of token t in channel c's row of a tile of T tokens: blocks of four
// tokens change places by channel, so that the transposing stores spread over
// the banks
template <int T>
__device__ __forceinline__ int place_b(int c, int t) {
  return t ^ (((c >> 3) & (T / 4 - 1)) << 2);
}

// Sums v[0..7] of one token over the channel lanes of the warp (lane bits from
// LN up), storing the sums each lane ends with: v[0..3] belong to dB, states
// 4 nl .., v[4..7] to dC, at row[0 .. S) and row[S .. 2 S).
template <int S>
__device__ __forceinline__ void sum_channels(float (&v)[8], int lane, float* row) {
  constexpr int LN = S / 4, LC = 32 / LN;
  const int nl = lane % LN;
  int first = 0;
  if constexpr (LC >= 2) {
    const bool hi = lane & 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, hi ? v[i] : v[i + 4], 16);
      v[i] = (hi ? v[i + 4] : v[i]) + o;
    }
    first = hi ? 4 : 0;
  }
  if constexpr (LC >= 4) {
    const bool hi = lane & 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, hi ? v[i] : v[i + 2], 8);
      v[i] = (hi ? v[i + 2] : v[i]) + o;
    }
    first += hi ? 2 : 0;
  }
  if constexpr (LC >= 8) {
    const bool hi = lane & 4;
    const float o = __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], 4);
    v[0] = (hi ? v[1] : v[0]) + o;
    first += hi ? 1 : 0;
  }
  if constexpr (LC >= 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  constexpr int KEEP = LC >= 8 ? 1 : 8 / LC;
  if (LC < 16 || !(lane & 2)) {
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      const int k = first + i;
      row[(k >> 2) * S + nl * 4 + (k & 3)] = v[i];
    }
  }
}

template <typename Tin, int S>
__global__ void __launch_bounds__(Layout<S>::NT) scan_bwd_kernel(const Args a) {
  using L = Layout<S>;
  using TL = Tile<S>;
  constexpr int LN = L::LN, NT = L::NT, CT = L::CT, T = TL::T, P = TL::P;
  constexpr int PER = T * CT / NT;
  constexpr int VEC = PER < 1 ? 1 : PER;
  static_assert(VEC <= 8, "one item per thread");
  constexpr int CV = CT / VEC;
  extern __shared__ __align__(16) float sm[];
  float* sdt = sm;
  float* su = sdt + TL::kRows;
  float* sdy = su + TL::kRows;
  float* sB = sdy + TL::kRows;
  float* sC = sB + T * S;
  float* sred = sC + T * S;  // [warp][T][2 S]

  if (a.seg.cu) {
    if (!a.sb->seqlens_ok) return;
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.sb->status = KDA_OK;
    a.sb->detail = 0;
  }
  const int unit = blockIdx.x / a.nblk, cb = blockIdx.x % a.nblk;
  const Unit un = resolve(a.seg, unit);
  if (!un.valid) return;
  const int tid = threadIdx.x, lane = tid & 31, nl = tid % LN, c = tid / LN;
  const int d0 = cb * CT, d = d0 + c;
  const bool live = d < a.D;
  const int grp = d0 / (a.D / a.G);
  const int64_t so = (int64_t)d * S + nl * 4, ds = (int64_t)a.D * S;

  float A[4], A2[4], h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] = h[i] = 0.f;
  if (live) {
    load_vec<float, 4>(a.A + so, A);
    if (a.h_seg)
      load_vec<float, 4>(a.h_seg + unit * ds + so, h);
    else if (a.init)
      load_vec<float, 4>(a.init + un.n * ds + so, h);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = A[i] * kLog2e;

  // the thread's element group of a tile: token it, channels ic ..
  const int ic = tid % CV * VEC, it = tid / CV;
  const bool item = it < T;
  const bool ilive = item && d0 + ic < a.D;
  float bias[VEC], skip[VEC], sum_d[VEC], sum_b[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) bias[j] = skip[j] = sum_d[j] = sum_b[j] = 0.f;
  if (ilive && a.delta_bias) load_vec<float, VEC>(a.delta_bias + d0 + ic, bias);
  if (ilive && a.D_skip) load_vec<float, VEC>(a.D_skip + d0 + ic, skip);

  const int tiles = (int)((un.t1 - un.t0 + T - 1) / T);
  // slot of a unit's first tile: units lie in token order, so slots do not meet
  float* ckpt = a.ckpt + (un.t0 / T + unit) * ds + so;

  // ---- forward: the state in front of every tile
  for (int i0 = 0; i0 < tiles; ++i0) {
    if (live) store_vec<4>(ckpt + i0 * ds, h);
    if (i0 + 1 == tiles) break;
    const int64_t t0 = un.t0 + (int64_t)i0 * T;  // a whole tile
    if (item) {
      float x[VEC], dt[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[j] = dt[j] = 0.f;
      if (ilive) {
        load_vec<Tin, VEC>(static_cast<const Tin*>(a.x) + (t0 + it) * a.x_stride + d0 + ic, x);
        load_vec<Tin, VEC>(static_cast<const Tin*>(a.delta) + (t0 + it) * a.delta_stride + d0 + ic,
                           dt);
#pragma unroll
        for (int j = 0; j < VEC; ++j) dt[j] = step_size(dt[j] + bias[j], a.softplus);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int p = (ic + j) * P + place_b<T>(ic + j, it);
        sdt[p] = dt[j];
        su[p] = dt[j] * x[j];
      }
    }
    for (int e = tid * 2; e < T * S; e += NT * 2) {
      float b[2];
      load_vec<Tin, 2>(static_cast<const Tin*>(a.Bm) + (t0 + e / S) * a.B_stride + grp * S + e % S,
                       b);
      store_vec<2>(sB + e, b);
    }
    __syncthreads();
#pragma unroll
    for (int t4 = 0; t4 < T; t4 += 4) {
      const int p = c * P + place_b<T>(c, t4);
      const float4 dt4 = *reinterpret_cast<const float4*>(sdt + p);
      const float4 u4 = *reinterpret_cast<const float4*>(su + p);
      const float dts[4] = {dt4.x, dt4.y, dt4.z, dt4.w}, us[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 b4 = *reinterpret_cast<const float4*>(sB + (t4 + k) * S + nl * 4);
        const float bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = fmaf(ex2(dts[k] * A2[i]), h[i], us[k] * bs[i]);
      }
    }
    __syncthreads();
  }

  // ---- backward, last tile first; carry = dL/dh of the state in front of the
  // tiles already taken
  float carry[4], dA[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) carry[i] = dA[i] = 0.f;
  if (live) {
    if (a.g_seg)
      load_vec<float, 4>(a.g_seg + unit * ds + so, carry);
    else if (a.d_final)
      load_vec<float, 4>(a.d_final + un.n * ds + so, carry);
  }
  const int64_t total_row = 2 * S;
  const int64_t tokens = a.seg.cu ? a.seg.T : (int64_t)a.seg.num_seqs * a.seg.T;
  for (int i0 = tiles - 1; i0 >= 0; --i0) {
    const int64_t t0 = un.t0 + (int64_t)i0 * T;
    const int64_t t = t0 + it;
    const bool here = ilive && t < un.t1;
    float x[VEC], v[VEC], dt[VEC], dy[VEC], zz[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = v[j] = dt[j] = dy[j] = zz[j] = 0.f;
    if (here) {
      load_vec<Tin, VEC>(static_cast<const Tin*>(a.x) + t * a.x_stride + d0 + ic, x);
      load_vec<Tin, VEC>(static_cast<const Tin*>(a.delta) + t * a.delta_stride + d0 + ic, v);
      load_vec<Tin, VEC>(static_cast<const Tin*>(a.dout) + t * a.D + d0 + ic, dy);
      if (a.z) load_vec<Tin, VEC>(static_cast<const Tin*>(a.z) + t * a.z_stride + d0 + ic, zz);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[j] += bias[j];
        dt[j] = step_size(v[j], a.softplus);
      }
    }
    if (item) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int p = (ic + j) * P + place_b<T>(ic + j, it);
        sdt[p] = dt[j];
        su[p] = dt[j] * x[j];
        sdy[p] = a.z ? dy[j] * (zz[j] * sigmoid_fast(zz[j])) : dy[j];
      }
    }
    for (int e = tid * 2; e < T * S; e += NT * 2) {
      float b[2] = {0.f, 0.f}, cc[2] = {0.f, 0.f};
      const int64_t tt = t0 + e / S;
      if (tt < un.t1) {
        load_vec<Tin, 2>(static_cast<const Tin*>(a.Bm) + tt * a.B_stride + grp * S + e % S, b);
        load_vec<Tin, 2>(static_cast<const Tin*>(a.Cm) + tt * a.C_stride + grp * S + e % S, cc);
      }
      store_vec<2>(sB + e, b);
      store_vec<2>(sC + e, cc);
    }
    float h0[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) load_vec<float, 4>(ckpt + i0 * ds, h0);
    __syncthreads();
    float hs[T][4], dec[T][4];
#pragma unroll
    for (int t4 = 0; t4 < T; t4 += 4) {
      const int p = c * P + place_b<T>(c, t4);
      const float4 dt4 = *reinterpret_cast<const float4*>(sdt + p);
      const float4 u4 = *reinterpret_cast<const float4*>(su + p);
      const float dts[4] = {dt4.x, dt4.y, dt4.z, dt4.w}, us[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 b4 = *reinterpret_cast<const float4*>(sB + (t4 + k) * S + nl * 4);
        const float bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dec[t4 + k][i] = ex2(dts[k] * A2[i]);
          const float hp = t4 + k == 0 ? h0[i] : hs[t4 + k > 0 ? t4 + k - 1 : 0][i];
          hs[t4 + k][i] = fmaf(dec[t4 + k][i], hp, us[k] * bs[i]);
        }
      }
    }
    float* wred = sred + (tid >> 5) * T * 2 * S;
#pragma unroll
    for (int t4 = T - 4; t4 >= 0; t4 -= 4) {
      const int p = c * P + place_b<T>(c, t4);
      const float4 dt4 = *reinterpret_cast<const float4*>(sdt + p);
      const float4 u4 = *reinterpret_cast<const float4*>(su + p);
      const float4 dy4 = *reinterpret_cast<const float4*>(sdy + p);
      const float dts[4] = {dt4.x, dt4.y, dt4.z, dt4.w}, us[4] = {u4.x, u4.y, u4.z, u4.w};
      const float dys[4] = {dy4.x, dy4.y, dy4.z, dy4.w};
      float sgB[4], sgA[4], sy[4];
#pragma unroll
      for (int k = 3; k >= 0; --k) {
        const float4 b4 = *reinterpret_cast<const float4*>(sB + (t4 + k) * S + nl * 4);
        const float4 c4 = *reinterpret_cast<const float4*>(sC + (t4 + k) * S + nl * 4);
        const float bs[4] = {b4.x, b4.y, b4.z, b4.w}, cs[4] = {c4.x, c4.y, c4.z, c4.w};
        float part[8];
        sgB[k] = sgA[k] = sy[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float hp = t4 + k == 0 ? h0[i] : hs[t4 + k > 0 ? t4 + k - 1 : 0][i];
          const float g = fmaf(cs[i], dys[k], carry[i]);
          part[i] = g * us[k];
          part[4 + i] = hs[t4 + k][i] * dys[k];
          sgB[k] = fmaf(g, bs[i], sgB[k]);
          sy[k] = fmaf(cs[i], hs[t4 + k][i], sy[k]);
          carry[i] = g * dec[t4 + k][i];
          const float ga = carry[i] * hp;
          dA[i] = fmaf(ga, dts[k], dA[i]);
          sgA[k] = fmaf(ga, A[i], sgA[k]);
        }
        sum_channels<S>(part, lane, wred + (t4 + k) * 2 * S);
      }
      // the channel's lanes have read these four tokens: the sums take their place
      const float2 rB = sum_lanes<LN>(sgB, nl), rA = sum_lanes<LN>(sgA, nl),
                   ry = sum_lanes<LN>(sy, nl);
      if (LN == 2) {
        *reinterpret_cast<float2*>(su + p + 2 * nl) = rB;
        *reinterpret_cast<float2*>(sdt + p + 2 * nl) = rA;
        *reinterpret_cast<float2*>(sdy + p + 2 * nl) = ry;
      } else if (nl < 4) {
        su[p + nl] = rB.x;
        sdt[p + nl] = rA.x;
        sdy[p + nl] = ry.x;
      }
    }
    __syncthreads();
    if (here) {
      float gx[VEC], gd[VEC], gz[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int p = (ic + j) * P + place_b<T>(ic + j, it);
        const float gB = su[p], gA = sdt[p], y = fmaf(skip[j], x[j], sdy[p]);
        float dyg = dy[j];
        if (a.z) {
          const float s = sigmoid_fast(zz[j]);
          gz[j] = dy[j] * y * (s * fmaf(zz[j], 1.f - s, 1.f));
          dyg *= zz[j] * s;
        }
        gx[j] = fmaf(gB, dt[j], dyg * skip[j]);
        gd[j] = fmaf(gB, x[j], gA);
        if (a.softplus) gd[j] *= sigmoid_fast(v[j]);
        sum_d[j] = fmaf(dyg, x[j], sum_d[j]);
        sum_b[j] += gd[j];
      }
      store_vec<VEC>(a.dx + t * a.D + d0 + ic, gx);
      store_vec<VEC>(a.ddelta + t * a.D + d0 + ic, gd);
      if (a.z) store_vec<VEC>(a.dz + t * a.D + d0 + ic, gz);
    }
    // dB and dC over the CTA's warps
    for (int e = tid; e < T * 2 * S; e += NT) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < TL::W; ++w) s += sred[w * T * 2 * S + e];
      const int64_t tt = t0 + e / (2 * S);
      if (tt < un.t1) a.dbc_part[((int64_t)cb * tokens + tt) * total_row + e % (2 * S)] = s;
    }
    __syncthreads();
  }
  if (live) {
    store_vec<4>(a.da_part + unit * ds + so, dA);
    if (un.first && a.d_init) store_vec<4>(a.d_init + un.n * ds + so, carry);
  }
  // dD and ddelta_bias: over the threads of a channel group, in token order
  float* red = sm;  // [T][2][CT]
  if (item) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      red[(it * 2 + 0) * CT + ic + j] = sum_d[j];
      red[(it * 2 + 1) * CT + ic + j] = sum_b[j];
    }
  }
  __syncthreads();
  for (int e = tid; e < 2 * CT; e += NT) {
    const int cc = e % CT;
    if (d0 + cc >= a.D) continue;
    float s = 0.f;
    for (int r = 0; r < T; ++r) s += red[r * 2 * CT + e];
    a.dd_part[((int64_t)unit * 2 + e / CT) * a.D + d0 + cc] = s;
  }
}

// Adds the partial sums in a fixed order: blocks [0, tok_blocks) the channel
// blocks of dB and dC, four values a thread; the others the units of dA, dD
// and ddelta_bias.
__global__ void __launch_bounds__(256) scan_bwd_sum_kernel(const Args a, int64_t tokens,
                                                           int64_t tok_blocks,
                                                           float* __restrict__ dA,
                                                           float* __restrict__ dB,
                                                           float* __restrict__ dC,
                                                           float* __restrict__ dD,
                                                           float* __restrict__ dbias) {
  if (a.seg.cu && !a.sb->seqlens_ok) return;
  if (blockIdx.x < tok_blocks) {
    const int per = 2 * a.S / 4;  // float4s of a token and group
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int e = (int)(idx % per) * 4;
    const int64_t tg = idx / per;
    const int g = (int)(tg % a.G);
    const int64_t t = tg / a.G;
    if (t >= tokens) return;
    const int per_group = a.G == 1 ? a.nblk : a.nblk / a.G;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int b = g * per_group; b < (g + 1) * per_group; ++b) {
      float v[4];
      load_vec<float, 4>(a.dbc_part + ((int64_t)b * tokens + t) * 2 * a.S + e, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += v[i];
    }
    float* to = (e < a.S ? dB : dC) + (t * a.G + g) * a.S + (e < a.S ? e : e - a.S);
    store_vec<4>(to, s);
    return;
  }
  const int units = a.seg.cu ? __ldg(a.seg.seg_off + a.seg.num_seqs) : a.seg.units;
  const int64_t ds = (int64_t)a.D * a.S;
  const int64_t e = ((int64_t)(blockIdx.x - tok_blocks) * 256 + threadIdx.x);
  if (e < ds) {
    float s = 0.f;
#pragma unroll 4
    for (int u = 0; u < units; ++u) s += a.da_part[u * ds + e];
    dA[e] = s;
  } else if (e < ds + 2 * a.D) {
    const int64_t k = e - ds;
    float s = 0.f;
#pragma unroll 4
    for (int u = 0; u < units; ++u) s += a.dd_part[(int64_t)u * 2 * a.D + k];
    float* to = k < a.D ? dD : dbias;
    if (to) to[k < a.D ? k : k - a.D] = s;
  }
}

template <typename Tin, int S>
cudaError_t launch_bwd_s(const Args& a, cudaStream_t st) {
  constexpr size_t bytes = Tile<S>::bytes();
  if (bytes > 48 * 1024)
    if (cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<Tin, S>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)bytes))
      return e;
  const unsigned grid = (unsigned)((int64_t)a.seg.units * a.nblk);
  scan_bwd_kernel<Tin, S><<<grid, Layout<S>::NT, bytes, st>>>(a);
  return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_bwd(const Args& a, cudaStream_t st) {
  switch (a.S) {
    case 8: return launch_bwd_s<Tin, 8>(a, st);
    case 16: return launch_bwd_s<Tin, 16>(a, st);
    case 32: return launch_bwd_s<Tin, 32>(a, st);
    case 64: return launch_bwd_s<Tin, 64>(a, st);
    default: return launch_bwd_s<Tin, 128>(a, st);
  }
}

// byte offsets of the workspace's parts
struct Plan {
  Segments m;
  size_t seg_off, h_seg, g_seg, dt_sum, ckpt, dbc, da, dd, total;
  int64_t tokens;
  int nblk;
};

Plan plan_bwd(const int32_t* cu, int num_seqs, int B, int T, int D, int S) {
  Plan p{};
  p.m = plan_segments(cu, num_seqs, B, T, D, S);
  p.tokens = (int64_t)B * T;
  p.nblk = (D + chan_tile(S) - 1) / chan_tile(S);
  const size_t state = sizeof(float) * (size_t)D * S;
  size_t at = kStatusBytes;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  if (cu) p.seg_off = take(sizeof(int32_t) * ((size_t)num_seqs + 1));
  if (p.m.segs > 1) {
    p.h_seg = take(state * p.m.units);
    p.g_seg = take(state * p.m.units);
    p.dt_sum = take(sizeof(float) * (size_t)p.m.units * D);
  }
  p.ckpt = take(state * (size_t)(p.tokens / step_of(S) + p.m.units + 1));
  p.dbc = take(sizeof(float) * (size_t)p.nblk * p.tokens * 2 * S);
  p.da = take(state * p.m.units);
  p.dd = take(sizeof(float) * (size_t)p.m.units * 2 * D);
  p.total = at;
  return p;
}

}  // namespace
}  // namespace scan
}  // namespace kda

using namespace kda;
using namespace kda::scan;

extern "C" {

size_t kda_selective_scan_bwd_workspace_size(int B, int T, int D, int S, int G, int num_seqs) {
  if (B <= 0 || T <= 0 || D <= 0 || G <= 0 || num_seqs < 0 || !sizes_ok(D, S, G) ||
      (int64_t)B * T > kMaxRows)
    return 0;
  static const int32_t packed = 0;  // only whether there are offsets matters here
  return plan_bwd(num_seqs > 0 && B == 1 ? &packed : nullptr, num_seqs, B, T, D, S).total;
}

kda_status kda_selective_scan_bwd(const void* x, int64_t x_stride, const void* delta,
                                  int64_t delta_stride, const float* A, const void* Bm,
                                  int64_t B_stride, const void* Cm, int64_t C_stride,
                                  const float* D_skip, const void* z, int64_t z_stride,
                                  const float* delta_bias, int delta_softplus,
                                  kda_dtype in_dtype, const float* init_state, const void* dout,
                                  const float* d_final, const int32_t* cu_seqlens, int num_seqs,
                                  int B, int T, int D, int S, int G, float* dx, float* ddelta,
                                  float* dA, float* dBm, float* dCm, float* dD_skip, float* dz,
                                  float* ddelta_bias, float* d_init, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!x || !delta || !A || !Bm || !Cm || !dout || !dx || !ddelta || !dA || !dBm || !dCm ||
      !workspace)
    return KDA_ERR_INVALID_ARG;
  if ((z != nullptr) != (dz != nullptr)) return KDA_ERR_INVALID_ARG;
  if (kda_status s = check_batch(cu_seqlens, num_seqs, B, T)) return s;
  if (kda_status s = check_scan(in_dtype, D, S, G, x_stride, delta_stride, B_stride, C_stride, z,
                                z_stride))
    return s;
  const int64_t n = (int64_t)B * T, es = elem_bytes(in_dtype), w = (int64_t)G * S;
  const int64_t N = cu_seqlens ? num_seqs : B, state = N * D * S * 4;
  const Plan p = plan_bwd(cu_seqlens, num_seqs, B, T, D, S);
  const Span ins[] = {{x, row_bytes(n, x_stride, D, es)},
                      {delta, row_bytes(n, delta_stride, D, es)},
                      {A, (int64_t)D * S * 4},
                      {Bm, row_bytes(n, B_stride, w, es)},
                      {Cm, row_bytes(n, C_stride, w, es)},
                      {D_skip, (int64_t)D * 4},
                      {z, row_bytes(n, z_stride, D, es)},
                      {delta_bias, (int64_t)D * 4},
                      {init_state, state},
                      {dout, n * D * es},
                      {d_final, state},
                      {cu_seqlens, (N + 1) * 4}};
  const Span outs[] = {{dx, n * D * 4},       {ddelta, n * D * 4},
                       {dA, (int64_t)D * S * 4}, {dBm, n * w * 4},
                       {dCm, n * w * 4},      {dD_skip, (int64_t)D * 4},
                       {dz, n * D * 4},       {ddelta_bias, (int64_t)D * 4},
                       {d_init, state},       {workspace, (int64_t)p.total}};
  if (kda_status s = check_spans(ins, outs)) return s;
  if (workspace_bytes < p.total) return KDA_ERR_WORKSPACE;
  Args a = scan_args(x, x_stride, delta, delta_stride, A, Bm, B_stride, Cm, C_stride, D_skip, z,
                     z_stride, delta_bias, delta_softplus, D, S, G);
  a.seg = p.m;
  const int64_t tok_blocks = (n * G * (2 * S / 4) + 255) / 256;
  const int64_t sum_blocks = ((int64_t)D * S + 2 * D + 255) / 256;
  if ((int64_t)a.seg.units * a.nblk > 0x7fffffffLL || tok_blocks + sum_blocks > 0x7fffffffLL ||
      N * D / 256 * (S / 4) > 0x7ffffff0LL)
    return KDA_ERR_UNSUPPORTED;
  char* ws = static_cast<char*>(workspace);
  a.init = init_state;
  a.dout = dout;
  a.d_final = d_final;
  a.dx = dx;
  a.ddelta = ddelta;
  a.dz = dz;
  a.d_init = d_init;
  a.sb = static_cast<StatusBlock*>(workspace);
  a.ckpt = reinterpret_cast<float*>(ws + p.ckpt);
  a.dbc_part = reinterpret_cast<float*>(ws + p.dbc);
  a.da_part = reinterpret_cast<float*>(ws + p.da);
  a.dd_part = reinterpret_cast<float*>(ws + p.dd);
  cudaStream_t st = (cudaStream_t)stream;
  if (cu_seqlens) {
    int32_t* off = reinterpret_cast<int32_t*>(ws + p.seg_off);
    a.seg.seg_off = off;
    if (cudaError_t e = launch_seqlens_plan(cu_seqlens, num_seqs, T, a.sb, a.seg.seg_len, off, st))
      return cuda_failure(e);
  }
  if (a.seg.segs > 1) {
    a.h_seg = reinterpret_cast<float*>(ws + p.h_seg);
    a.g_seg = reinterpret_cast<float*>(ws + p.g_seg);
    a.dt_sum = reinterpret_cast<float*>(ws + p.dt_sum);
    if (cudaError_t e = launch_ends(a, in_dtype, st)) return cuda_failure(e);
  }
  cudaError_t e = in_dtype == KDA_BF16 ? launch_bwd<__nv_bfloat16>(a, st) : launch_bwd<float>(a, st);
  if (e != cudaSuccess) return cuda_failure(e);
  scan_bwd_sum_kernel<<<(unsigned)(tok_blocks + sum_blocks), 256, 0, st>>>(
      a, n, tok_blocks, dA, dBm, dCm, dD_skip, ddelta_bias);
  e = cudaGetLastError();
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

}  // extern "C"
