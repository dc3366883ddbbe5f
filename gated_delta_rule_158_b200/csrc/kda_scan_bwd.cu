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
// Three kernels.  The forward scan's segment pass (scan_fwd_kernel, kEnd or
// kEnds) keeps the states in front of every kStep tokens; with a sequence in
// several segments it starts each from zero and also gives the state gradient
// that a segment's outputs send to its start, and the segments' incoming
// states and gradients follow from one combination.  Then every segment walks
// its tiles of kStep tokens from last to first: the tile's states and decays
// again into registers, and the reverse recurrence over them.  Last, the
// partial sums of dB, dC (one per channel block), dA, dD and ddelta_bias (one
// per segment) are added in a fixed order.  Nothing is added atomically.
//
// The walk is bound by its instructions (24 per state element and token)
// at the two warps per scheduler that its registers leave: a thread has 4
// states of 2 channels, so that the sums over channels (dB, dC: 8 values a
// token) and over states (3 per channel) are halved before they cross lanes,
// where each exchanged value costs a shuffle, two selects and an addition.
//
// Measured on a B200, bf16, 16 states, 4 x 4096 tokens x 2048 channels: 287 us
// for the segments' pass, 669 us for the walk (55 % of the issue slots at two
// warps a scheduler; 255 registers, 8 bytes of them spilled), 20 us for the sums.  One channel a thread and 16 tokens a
// tile took 1715 us; the walk in one wave of CTAs instead of four, 750 us; three
// warps a scheduler at 168 registers spill (800 us); dt, u and dy stored twice,
// so that the pairs need no moves, load half as much again (771 us).
#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

constexpr int kWalk = 2 * kStep;  // tokens per tile: two steps from kept states

template <int S>
struct Walk {
  static constexpr int LN = S / 4;                 // lanes of a channel
  static constexpr int NT = S <= 32 ? 128 : 256;
  static constexpr int CT = 2 * NT / LN;           // channels of a CTA
  static constexpr int W = NT / 32;
  static constexpr int kCtas = S <= 32 ? 2 : 1;    // per SM, by registers
  static constexpr int T = kWalk;
  static constexpr int PER = T * CT / NT;          // elements of a tile per thread
  static constexpr int VEC = PER > 4 ? 4 : PER < 2 ? 2 : PER;
  static constexpr int ITEMS = PER < 2 ? 1 : PER / VEC, CV = CT / VEC;
  static constexpr int BPT = T * S / NT < 2 ? 2 : T * S / NT > 4 ? 4 : T * S / NT;
  static constexpr int BIT = T * S / NT < BPT ? 1 : T * S / NT / BPT;
  // fp32 rows of the tile, offsets in floats
  static constexpr int kDu = 0;                    // store_du; then the sums of dx, d(dt)
  static constexpr int kRow = kDuRow<2, CT>;
  static constexpr int kDy = kDu + T * kRow;       // [token][channel]; then y
  static constexpr int kB = kDy + T * CT;
  static constexpr int kC = kB + T * S;
  static constexpr int kRed = kC + T * S;          // dB, dC [warp][T][2 S]
  static constexpr int kDt = kRed + W * T * 2 * S; // the threads' own dt
  static constexpr int kKeep = kDt + NT * ITEMS * VEC;  // kept states of two steps, 8 a thread
  static constexpr int kKeepDt = kKeep + 2 * 8 * NT;    // and their sums of dt
  static constexpr int kHin = kKeepDt + 2 * 2 * NT;     // the segment's incoming states
  static constexpr int kRows = kHin + 8 * NT;
};

// bytes of a CTA: the rows, and the threads' slots of two tiles (x, delta, z,
// dout; B, C)
template <typename Tin, int S>
struct WalkSmem {
  using L = Walk<S>;
  static constexpr int kItem = L::VEC * (int)sizeof(Tin), kBitem = L::BPT * (int)sizeof(Tin);
  static constexpr int kSlots = L::NT * L::ITEMS * kItem * 4;
  static constexpr int kStage = kSlots + L::NT * L::BIT * kBitem * 2;
  static constexpr size_t bytes() { return sizeof(float) * (size_t)L::kRows + 2 * (size_t)kStage; }
};

// Sums v[0..7] of one token over the channel lanes of the warp (lane bits from
// LN up); v[0..3] belong to dB, states 4 nl .., v[4..7] to dC.  A lane ends with
// kKept<S> of the sums, in v[0 ..), from v[kept_from()] on.
template <int S>
constexpr int kKept = 128 / S >= 8 ? 1 : S / 16;  // 8 values over 32 / (S / 4) lanes

template <int S>
__device__ __forceinline__ int kept_from(int lane) {
  constexpr int LC = 32 / (S / 4);
  return (LC >= 2 && lane & 16 ? 4 : 0) + (LC >= 4 && lane & 8 ? 2 : 0) +
         (LC >= 8 && lane & 4 ? 1 : 0);
}

template <int S>
__device__ __forceinline__ void sum_channels(float (&v)[8], int lane) {
  constexpr int LN = S / 4, LC = 32 / LN;
  if constexpr (LC >= 2) {
    const bool hi = lane & 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, hi ? v[i] : v[i + 4], 16);
      v[i] = (hi ? v[i + 4] : v[i]) + o;
    }
  }
  if constexpr (LC >= 4) {
    const bool hi = lane & 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, hi ? v[i] : v[i + 2], 8);
      v[i] = (hi ? v[i + 2] : v[i]) + o;
    }
  }
  if constexpr (LC >= 8) {
    const bool hi = lane & 4;
    const float o = __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], 4);
    v[0] = (hi ? v[1] : v[0]) + o;
  }
  if constexpr (LC >= 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
}

// the kept sums of a token to its row: dB at [0, S), dC at [S, 2 S)
template <int S>
__device__ __forceinline__ void store_kept(float* row, const float (&v)[kKept<S>], int lane) {
  constexpr int LN = S / 4, LC = 32 / LN;
  if (LC < 16 || !(lane & 2)) {
#pragma unroll
    for (int i = 0; i < kKept<S>; ++i) {
      const int k = kept_from<S>(lane) + i;
      row[(k >> 2) * S + lane % LN * 4 + (k & 3)] = v[i];
    }
  }
}

// Sums of two values over a channel's lanes: lane l returns value l & 1.
template <int LN>
__device__ __forceinline__ float sum_two(const float (&v)[2], int l) {
  const bool odd = l & 1;
  float r = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
#pragma unroll
  for (int o = 2; o < LN; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

// 2^v of both halves, not merged with an earlier one of the same value
__device__ __forceinline__ f2 ex2_again(f2 v) {
  float a, b;
  unpack2(v, a, b);
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pack2(a, b);
}

// an entry of the walk's sums: (gA, gA', gB, gB')
__device__ __forceinline__ void load_pair_sums(const float* p, float* gA, float* gB) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  gA[0] = v.x; gA[1] = v.y;
  gB[0] = v.z; gB[1] = v.w;
}

template <typename Tin, int S>
__global__ void __launch_bounds__(Walk<S>::NT, Walk<S>::kCtas) scan_bwd_kernel(const Args a) {
  using L = Walk<S>;
  using M = WalkSmem<Tin, S>;
  constexpr int LN = L::LN, NT = L::NT, CT = L::CT, T = L::T, VEC = L::VEC, CV = L::CV,
                ITEMS = L::ITEMS, BPT = L::BPT, BIT = L::BIT;
  extern __shared__ __align__(16) float sm[];
  if (a.seg.cu && !a.sb->seqlens_ok) return;
  const int nblk = a.G * ((a.D / a.G + CT - 1) / CT);
  const int ub = blockIdx.x / nblk, cb = blockIdx.x - ub * nblk;
  const Unit un = resolve(a.seg, a.sb, ub);
  if (!un.valid) return;
  const int tid = threadIdx.x, lane = tid & 31, nl = tid % LN, cp = tid / LN;
  const Channels ch = channels_of<CT>(a, cb);
  const int d = ch.d0 + 2 * cp;
  const bool live = 2 * cp < ch.n;  // ch.n is even: both channels or none
  const int64_t ds = (int64_t)a.D * S;
  const int64_t so = (int64_t)d * S + nl * 4;

  f2 A2[2][2], carry[2][2], dA[2][2], dA_err[2][2];
  float* const own_hin = sm + L::kHin + tid * 4;  // of channel q: + 4 q NT
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int i = 0; i < 2; ++i) A2[q][i] = carry[q][i] = dA[q][i] = dA_err[q][i] = zero2();
  if (live) {
    const float* from = un.cut      ? a.g_seg + un.slot * ds
                        : a.d_final ? a.d_final + un.n * ds : nullptr;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      load_pairs(a.A + so + q * S, A2[q]);
      if (from) load_pairs(from + so + q * S, carry[q]);
      if (un.cut) {
        f2 hin[2];
        load_pairs(a.h_seg + un.slot * ds + so + q * S, hin);
        store_pairs(own_hin + q * 4 * NT, hin);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float lo, hi;
        unpack2(A2[q][k], lo, hi);
        A2[q][k] = pack2(rate2(lo), rate2(hi));
      }
    }
  }

  // the thread's elements of a tile: tokens it + m NT / CV, channels ic ..
  const int ic = tid % CV * VEC, it = tid / CV;
  const bool item = it < T;
  const bool ilive = item && ic < ch.n;
  const int col = ch.d0 + ic;
  float sum_d[VEC], sum_b[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) sum_d[j] = sum_b[j] = 0.f;

  const int len = (int)(un.t1 - un.t0);
  const int tiles = (len + T - 1) / T;
  const int64_t tile0 = first_tile(un);
  const int64_t tokens = a.seg.cu ? a.seg.T : (int64_t)a.seg.num_seqs * a.seg.T;

  char* const slots = reinterpret_cast<char*>(sm + L::kRows);
  auto slot = [&](int i, int arr, int m) {
    return slots + (i & 1) * M::kStage + ((arr * ITEMS + m) * NT + tid) * M::kItem;
  };
  auto bslot = [&](int i, int arr, int m) {
    return slots + (i & 1) * M::kStage + M::kSlots + ((arr * BIT + m) * NT + tid) * M::kBitem;
  };
  float* const own_dt = sm + L::kDt + tid * VEC;  // of item m: + m NT VEC

  auto copy_tile = [&](int i) {
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int t = i * T + it + m * (NT / CV);
      const bool in = ilive && t < len;
      const int64_t row = in ? un.t0 + t : un.t0;
      const int at = in ? col : 0;
      copy_in<M::kItem>(slot(i, 0, m), static_cast<const Tin*>(a.x) + row * a.x_stride + at, in);
      copy_in<M::kItem>(slot(i, 1, m), static_cast<const Tin*>(a.delta) + row * a.delta_stride + at,
                        in);
      if (a.z)
        copy_in<M::kItem>(slot(i, 2, m), static_cast<const Tin*>(a.z) + row * a.z_stride + at, in);
      copy_in<M::kItem>(slot(i, 3, m), static_cast<const Tin*>(a.dout) + row * a.D + at, in);
    }
#pragma unroll
    for (int m = 0; m < BIT; ++m) {
      const int e = (tid + m * NT) * BPT, t = i * T + e / S;
      if (e >= T * S) break;
      const bool in = t < len;
      const int64_t row = in ? un.t0 + t : un.t0;
      const int at = ch.g * S + e % S;
      copy_in<M::kBitem>(bslot(i, 0, m), static_cast<const Tin*>(a.Bm) + row * a.B_stride + at, in);
      copy_in<M::kBitem>(bslot(i, 1, m), static_cast<const Tin*>(a.Cm) + row * a.C_stride + at, in);
    }
    copies_issued();
  };
  auto fill_tile = [&](int i) {
    float bias[VEC] = {};
    if (ilive && a.delta_bias) load_vec<float, VEC>(a.delta_bias + col, bias);
    if (item) {
#pragma unroll
      for (int m = 0; m < ITEMS; ++m) {
        const int t = it + m * (NT / CV);
        const bool in = ilive && i * T + t < len;
        float dt[VEC], u[VEC], dy[VEC], z[VEC];
        read_slot<Tin, VEC>(slot(i, 1, m), dt);
        read_slot<Tin, VEC>(slot(i, 0, m), u);
        read_slot<Tin, VEC>(slot(i, 3, m), dy);
#pragma unroll
        for (int j = 0; j < VEC; ++j) dt[j] += bias[j];
        step_sizes<VEC>(dt, a.softplus);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          dt[j] = in ? dt[j] : 0.f;
          u[j] *= dt[j];
        }
        if (a.z) {
          read_slot<Tin, VEC>(slot(i, 2, m), z);
#pragma unroll
          for (int j = 0; j < VEC; ++j) dy[j] *= z[j] * sigmoid_fast(z[j]);
        }
        store_du<2, VEC>(sm + L::kDu + t * L::kRow, ic, dt, u);
        store_vec<VEC>(sm + L::kDy + t * CT + ic, dy);
        store_vec<VEC>(own_dt + m * NT * VEC, dt);
      }
    }
#pragma unroll
    for (int m = 0; m < BIT; ++m) {
      const int e = (tid + m * NT) * BPT;
      if (e >= T * S) break;
      float b[BPT];
      read_slot<Tin, BPT>(bslot(i, 0, m), b);
      store_vec<BPT>(sm + L::kB + e, b);
      read_slot<Tin, BPT>(bslot(i, 1, m), b);
      store_vec<BPT>(sm + L::kC + e, b);
    }
  };
  // the state kept in front of a step's tokens, to this thread's slot
  auto keep_at = [&](int step, int q) {
    return sm + L::kKeep + (step & 1) * 8 * NT + q * 4 * NT + tid * 4;
  };
  auto keep_dt_at = [&](int step, int q) {
    return sm + L::kKeepDt + (step & 1) * 2 * NT + q * NT + tid;
  };
  auto copy_kept = [&](int step) {
    const bool in = live && step >= 0 && step * kStep < len;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      copy_in<16>(reinterpret_cast<char*>(keep_at(step, q)),
                  in ? a.ckpt + (tile0 + step) * ds + so + q * S : a.ckpt, in);
      if (un.cut)
        copy_in<4>(reinterpret_cast<char*>(keep_dt_at(step, q)),
                   in ? a.ckpt_dt + (tile0 + step) * a.D + d + q : a.ckpt_dt, in);
    }
  };
  // tokens [s, s + kStep) of the tile
  auto walk = [&](int s, int step) {
    float* pdu = sm + L::kDu + s * L::kRow + du_entry<2>(2 * cp);
    float* pdy = sm + L::kDy + s * CT + 2 * cp;
    const float* pb = sm + L::kB + s * S + nl * 4;
    const float* pc = sm + L::kC + s * S + nl * 4;
    float* red = sm + L::kRed + ((tid >> 5) * T + s) * 2 * S;
    f2 h0[2][2], hs[kStep][2][2], dAs[2][2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      load_pairs(keep_at(step, q), h0[q]);
      if (un.cut && live) {
        const float past = *keep_dt_at(step, q);
        f2 hin[2];
        load_pairs(own_hin + q * 4 * NT, hin);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          h0[q][k] = fma2(ex2_2(mul2(pack2(past, past), A2[q][k])), hin[k], h0[q][k]);
      }
    }
    copy_kept(step - 2);  // into the slot that has just been read
    copies_issued();
#pragma unroll
    for (int t = 0; t < kStep; ++t) {
      f2 b[2];
      float dt[2], u[2];
      load_pairs(pb + t * S, b);
      load_du<2>(pdu + t * L::kRow, dt, u);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const f2 dd = pack2(dt[q], dt[q]), uu = pack2(u[q], u[q]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          hs[t][q][k] = fma2(ex2_2(decay_exp(dd, A2[q][k])),
                             t == 0 ? h0[q][k] : hs[t > 0 ? t - 1 : 0][q][k], mul2(uu, b[k]));
        }
      }
    }
    // the decays are formed again and their operands loaded again: kept from
    // above they would take as many registers as the states
    asm volatile("" ::: "memory");
#pragma unroll
    for (int t4 = kStep - 4; t4 >= 0; t4 -= 4) {
      // stored behind the four tokens: a store keeps the loads of later tokens
      // behind it
      float kept[4][kKept<S>], y[4];
      float2 gg[4];
#pragma unroll
      for (int m = 3; m >= 0; --m) {
        const int t = t4 + m;
        f2 b[2], cc[2], pB[2], pC[2];
        float dt[2], u[2], dys[2], gA[2], gB[2], yy[2];
        load_pairs(pb + t * S, b);
        load_pairs(pc + t * S, cc);
        load_du<2>(pdu + t * L::kRow, dt, u);
        load_vec<float, 2>(pdy + t * CT, dys);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const f2 dd = pack2(dt[q], dt[q]), uu = pack2(u[q], u[q]), dy = pack2(dys[q], dys[q]);
          f2 sB, sA, sy;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const f2 hp = t == 0 ? h0[q][k] : hs[t > 0 ? t - 1 : 0][q][k];
            const f2 g = fma2(cc[k], dy, carry[q][k]);
            pB[k] = q == 0 ? mul2(g, uu) : fma2(g, uu, pB[k]);
            pC[k] = q == 0 ? mul2(hs[t][q][k], dy) : fma2(hs[t][q][k], dy, pC[k]);
            sB = k == 0 ? mul2(g, b[k]) : fma2(g, b[k], sB);
            sy = k == 0 ? mul2(cc[k], hs[t][q][k]) : fma2(cc[k], hs[t][q][k], sy);
            carry[q][k] = mul2(g, ex2_again(decay_exp(dd, A2[q][k])));
            const f2 ga = mul2(carry[q][k], hp);
            dAs[q][k] = t == kStep - 1 ? mul2(ga, dd) : fma2(ga, dd, dAs[q][k]);
            sA = k == 0 ? mul2(ga, A2[q][k]) : fma2(ga, A2[q][k], sA);
          }
          gA[q] = sum2(sA);
          gB[q] = sum2(sB);
          yy[q] = sum2(sy);
        }
        const float four[4] = {gA[0], gA[1], gB[0], gB[1]};
        gg[m] = sum_lanes<LN>(four, nl);  // lane l: value l, or 2 l and 2 l + 1
        y[m] = sum_two<LN>(yy, nl);
        float part[8];
        unpack2(pB[0], part[0], part[1]);
        unpack2(pB[1], part[2], part[3]);
        unpack2(pC[0], part[4], part[5]);
        unpack2(pC[1], part[6], part[7]);
        sum_channels<S>(part, lane);
#pragma unroll
        for (int v = 0; v < kKept<S>; ++v) kept[m][v] = part[v];
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) store_kept<S>(red + (t4 + m) * 2 * S, kept[m], lane);
      // over the tokens' dt, u and dy, which only the channels' lanes read, all
      // of them in this warp, and have read for the last time
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float* to = pdu + (t4 + m) * L::kRow;
        if constexpr (LN == 2) *reinterpret_cast<float2*>(to + 2 * nl) = gg[m];
        else if (nl < 4) to[nl] = gg[m].x;
        if (nl < 2) pdy[(t4 + m) * CT + nl] = y[m];
      }
    }
    // a segment's tokens are many: the steps' sums are added with the rounding
    // error of each addition carried along
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f2 neg = pack2(-1.f, -1.f);
        const f2 v = fma2(dA_err[q][k], neg, dAs[q][k]);
        const f2 s = add2(dA[q][k], v);
        dA_err[q][k] = fma2(v, neg, fma2(dA[q][k], neg, s));
        dA[q][k] = s;
      }
  };
  auto finish_tile = [&](int i) {
    float skip[VEC] = {}, bias[VEC] = {};
    if (ilive && a.D_skip) load_vec<float, VEC>(a.D_skip + col, skip);
    if (ilive && a.delta_bias) load_vec<float, VEC>(a.delta_bias + col, bias);
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int t = it + m * (NT / CV);
      if (!(ilive && i * T + t < len)) continue;
      float x[VEC], v[VEC], dy[VEC], z[VEC], dt[VEC], gA[VEC], gB[VEC], y[VEC];
      read_slot<Tin, VEC>(slot(i, 0, m), x);
      read_slot<Tin, VEC>(slot(i, 1, m), v);
      read_slot<Tin, VEC>(slot(i, 3, m), dy);
      if (a.z) read_slot<Tin, VEC>(slot(i, 2, m), z);
      load_vec<float, VEC>(own_dt + m * NT * VEC, dt);
#pragma unroll
      for (int j = 0; j < VEC; j += 2)
        load_pair_sums(sm + L::kDu + t * L::kRow + du_entry<2>(ic + j), gA + j, gB + j);
      load_vec<float, VEC>(sm + L::kDy + t * CT + ic, y);
      const int64_t at = (un.t0 + i * T + t) * a.D + col;
      float out[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (a.z) {
          const float s = sigmoid_fast(z[j]), zs = z[j] * s;
          out[j] = dy[j] * fmaf(skip[j], x[j], y[j]) * fmaf(zs, 1.f - s, s);
          dy[j] *= zs;
        }
        sum_d[j] = fmaf(dy[j], x[j], sum_d[j]);
      }
      if (a.z) store_vec<VEC>(a.dz + at, out);
#pragma unroll
      for (int j = 0; j < VEC; ++j) out[j] = fmaf(gB[j], dt[j], dy[j] * skip[j]);
      store_vec<VEC>(a.dx + at, out);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        out[j] = fmaf(gB[j], x[j], gA[j] * (1.f / kLog2e));
        if (a.softplus) out[j] *= sigmoid_fast(v[j] + bias[j]);
        sum_b[j] += out[j];
      }
      store_vec<VEC>(a.ddelta + at, out);
    }
    // dB and dC over the CTA's warps
    float* to = a.dbc_part + ((int64_t)cb * tokens + un.t0 + (int64_t)i * T) * 2 * S;
    const int rows = min(T, len - i * T) * 2 * S;
    for (int e = tid * 4; e < rows; e += NT * 4) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < L::W; ++v) {
        float p[4];
        load_vec<float, 4>(sm + L::kRed + v * T * 2 * S + e, p);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] += p[k];
      }
      store_vec<4>(to + e, s);
    }
  };

  if (tiles > 0) {
    copy_kept(2 * tiles - 1);
    copy_kept(2 * tiles - 2);
    copy_tile(tiles - 1);
  }
  for (int i = tiles - 1; i >= 0; --i) {
    copies_landed();  // this thread's own: nobody else reads its slots
    fill_tile(i);
    __syncthreads();
    if (i > 0) copy_tile(i - 1);
#pragma unroll 1
    for (int step = 2 * i + 1; step >= 2 * i; --step) {
      if (step * kStep < len) walk((step & 1) * kStep, step);
      else copy_kept(step - 2);
    }
    __syncthreads();
    finish_tile(i);
    __syncthreads();  // the warps' sums have been read
  }
  if (live) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      store_pairs(a.da_part + un.slot * ds + so + q * S, dA[q]);
      if (un.first && a.d_init) store_pairs(a.d_init + un.n * ds + so + q * S, carry[q]);
    }
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
  constexpr int ROWS = NT / CV < T ? NT / CV : T;
  for (int e = tid; e < 2 * CT; e += NT) {
    const int c = e % CT;
    if (c >= ch.n) continue;
    float s = 0.f;
    for (int r = 0; r < ROWS; ++r) s += red[r * 2 * CT + e];
    a.dd_part[((int64_t)un.slot * 2 + e / CT) * a.D + ch.d0 + c] = s;
  }
}

// Adds the partial sums in a fixed order: blocks [0, tok_blocks) the channel
// blocks of dB and dC, four values a thread; the others the units of dA, dD
// and ddelta_bias.
__global__ void __launch_bounds__(256) scan_bwd_sum_kernel(const Args a, int64_t tokens,
                                                           int per_group, int64_t tok_blocks,
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
  constexpr size_t bytes = WalkSmem<Tin, S>::bytes();
  if (bytes > 48 * 1024)
    if (cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<Tin, S>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)bytes))
      return e;
  const unsigned grid = (unsigned)((int64_t)a.seg.units * channel_blocks(a.D, a.G, Walk<S>::CT));
  scan_bwd_kernel<Tin, S><<<grid, Walk<S>::NT, bytes, st>>>(a);
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

int walk_channels(int S) {
  switch (S) {
    case 8: return Walk<8>::CT;
    case 16: return Walk<16>::CT;
    case 32: return Walk<32>::CT;
    case 64: return Walk<64>::CT;
    default: return Walk<128>::CT;
  }
}

// byte offsets of the workspace's parts
struct Plan {
  Segments m;
  size_t seg_off, order, h_seg, g_seg, dt_sum, ckpt, ckpt_dt, dbc, da, dd, total;
  int nblk;
};

Plan plan_bwd(const int32_t* cu, int num_seqs, int B, int T, int D, int S, int G) {
  Plan p{};
  p.m = plan_segments(cu, num_seqs, B, T, D, S, true);
  const int64_t tokens = (int64_t)B * T;
  p.nblk = channel_blocks(D, G, walk_channels(S));
  const size_t state = sizeof(float) * (size_t)D * S;
  const size_t tiles = (size_t)(tokens / kStep + p.m.units + 1);
  size_t at = kStatusBytes;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  if (cu) {
    p.seg_off = take(sizeof(int32_t) * ((size_t)num_seqs + 1));
    p.order = take(sizeof(int32_t) * ((size_t)num_seqs + 1));
  }
  if (p.m.segs > 1) {
    p.h_seg = take(state * p.m.units);
    p.g_seg = take(state * p.m.units);
    p.dt_sum = take(sizeof(float) * (size_t)p.m.units * D);
    p.ckpt_dt = take(sizeof(float) * tiles * D);
  }
  p.ckpt = take(state * tiles);
  p.dbc = take(sizeof(float) * (size_t)p.nblk * tokens * 2 * S);
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
      (int64_t)B * T > kMaxRows || !units_ok(num_seqs, T))
    return 0;
  static const int32_t packed = 0;  // only whether there are offsets matters here
  return plan_bwd(num_seqs > 0 && B == 1 ? &packed : nullptr, num_seqs, B, T, D, S, G).total;
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
  if (!units_ok(num_seqs, T)) return KDA_ERR_UNSUPPORTED;
  if (kda_status s = check_scan(in_dtype, D, S, G, x_stride, delta_stride, B_stride, C_stride, z,
                                z_stride))
    return s;
  const int64_t n = (int64_t)B * T, es = elem_bytes(in_dtype), w = (int64_t)G * S;
  const int64_t N = cu_seqlens ? num_seqs : B, state = N * D * S * 4;
  const Plan p = plan_bwd(cu_seqlens, num_seqs, B, T, D, S, G);
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
  if ((int64_t)a.seg.units * channel_blocks(D, G, 8) > 0x7fffffffLL ||
      tok_blocks + sum_blocks > 0x7fffffffLL ||
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
    int32_t* order = reinterpret_cast<int32_t*>(ws + p.order);
    a.seg.seg_off = off;
    a.seg.order = order;
    if (cudaError_t e = launch_scan_plan(a, off, order, st)) return cuda_failure(e);
  }
  a.split = a.seg.segs > 1;
  if (a.split) {
    a.h_seg = reinterpret_cast<float*>(ws + p.h_seg);
    a.g_seg = reinterpret_cast<float*>(ws + p.g_seg);
    a.dt_sum = reinterpret_cast<float*>(ws + p.dt_sum);
    a.ckpt_dt = reinterpret_cast<float*>(ws + p.ckpt_dt);
  }
  cudaError_t e = launch_ends(a, in_dtype, st);
  if (e != cudaSuccess) return cuda_failure(e);
  e = in_dtype == KDA_BF16 ? launch_bwd<__nv_bfloat16>(a, st) : launch_bwd<float>(a, st);
  if (e != cudaSuccess) return cuda_failure(e);
  scan_bwd_sum_kernel<<<(unsigned)(tok_blocks + sum_blocks), 256, 0, st>>>(
      a, n, p.nblk / G, tok_blocks, dA, dBm, dCm, dD_skip, ddelta_bias);
  e = cudaGetLastError();
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

}  // extern "C"
