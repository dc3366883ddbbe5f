// kda_scan.cu -- the selective state space scan: prompts and single tokens.
//
//   h_t[d, s] = e^{dt A[d, s]} h_{t-1}[d, s] + dt x[t, d] B[t, s]
//   y[t, d]   = sum_s C[t, s] h_t[d, s] + D[d] x[t, d],   out = y z sigmoid(z)
//
// An exponential per token, channel and state: the special-function unit (16
// values a clock and SM) bounds it before HBM does (S = 16 states: 2 x 16 / 16
// clocks against 4 x 2 bytes), and the registers that shared memory can fill
// (128 bytes a clock and SM) are next: B and C of a token go to every thread.
// So a thread has 4 states of SC channels: the token's 8 values of B and C
// serve SC channels, its 2 SC values of dt and u = dt x serve 4 states.  With
// two channels that is 12 words for 8 exponentials (three clocks of loads to
// four of exponentials); with one, the loads are the bound, but a batch has
// twice the warps.  Products over pairs of states take one instruction
// (f32x2), and the sums over a channel's lanes are transposed over four tokens
// (sum_lanes).
//
// A CTA has CT channels and walks its tokens in tiles of 32.  While a tile is
// scanned the next one's x, dt, z, B and C are copied to slots of the shared
// memory that only the copying thread reads (cp.async, no registers); each
// thread then turns its own into the fp32 rows that the scan reads, token by
// token.
//
// Measured on a B200, bf16, 16 states: 32,768 tokens x 2048 channels in 794 us.
// Under the profiler, each kernel alone and with cold caches, its 18 segments take
// 355 us for their own end states (79 % of the special-function unit), 9 us for the
// combination and 461 us for the outputs (68 % of that unit, 58 % of the issue
// slots).  Both large kernels take as long as their exponentials and their
// shared-memory words one after the other, and more warps a scheduler gained
// nothing.  Of those words half or more are B and C, which for bf16 inputs are
// widened before shared memory; each tile of 32 tokens forms the decays of 34.
// 12,001 packed tokens x 4096 in 390 to 450 us.  One token of 256 sequences x 4096: 32
// us = 4.4 TB/s (a thread loads its states once, computes and stores: nothing is in
// flight meanwhile, at 68 % of the issue slots).  Tried and not kept: one state a thread (878 us for the long
// prompt's outputs: its loads), a quarter of the exponentials as polynomials on
// the multiply-add units (472 us instead of 460), tiles of 16 tokens (481 us), five
// or six CTAs an SM (462 us).
#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

constexpr int kTile = 32;  // tokens per tile

template <int S, int SC_>
struct Layout {
  static constexpr int SC = SC_;
  static constexpr int LN = S / 4;                 // lanes of a channel
  static constexpr int NT = LN <= 8 ? 128 : 256;
  static constexpr int CT = SC * NT / LN;          // channels of a CTA
  static constexpr int PER = kTile * CT / NT;      // elements of a tile per thread
  static constexpr int VEC = PER > 4 ? 4 : PER < 2 ? 2 : PER;  // of them consecutive channels
  static constexpr int ITEMS = PER < 2 ? 1 : PER / VEC, CV = CT / VEC;
  static constexpr int BPT = kTile * S / NT > 4 ? 4 : kTile * S / NT;  // B, C elements per copy
  static constexpr int BIT = kTile * S / NT / BPT;
  static_assert(LN <= 32 && VEC >= SC, "layout");
};

// kOut: the outputs and the final state.  kEnd: only the state that the segment
// leaves and its sum of dt; kEnds: those, and the state gradient that the
// segment's outputs send to its start, sum_t (prod_{s <= t} e^{dt_s A}) C_t dy_t.
enum Mode { kOut, kEnd, kEnds };

template <typename Tin, int S, int SC, int MODE>
struct Smem {
  using L = Layout<S, SC>;
  // fp32 rows of the tile, offsets in floats
  static constexpr int kDu = 0;  // [token] store_du; behind the scan the outputs y
  static constexpr int kRow = kDuRow<SC, L::CT>;
  static constexpr int kDy = kDu + kTile * kRow;
  static constexpr int kB = kDy + (MODE == kEnds ? kTile * L::CT : 0);
  static constexpr int kC = kB + kTile * S;
  static constexpr int kRows = kC + (MODE == kEnd ? 0 : kTile * S);
  // the threads' slots of two tiles: x, delta, z, dout; B, C
  static constexpr int kArrays = MODE == kEnd ? 2 : MODE == kOut ? 3 : 4;
  static constexpr int kItem = L::VEC * (int)sizeof(Tin), kBitem = L::BPT * (int)sizeof(Tin);
  static constexpr int kSlots = L::NT * L::ITEMS * kItem * kArrays;  // bytes
  static constexpr int kBslots = L::NT * L::BIT * kBitem * (MODE == kEnd ? 1 : 2);
  static constexpr int kStage = kSlots + kBslots;
  static constexpr size_t bytes() { return sizeof(float) * (size_t)kRows + 2 * (size_t)kStage; }
};

template <typename Tin, int S, int SC_, int MODE>
__global__ void __launch_bounds__(Layout<S, SC_>::NT) scan_fwd_kernel(const Args a) {
  using L = Layout<S, SC_>;
  using M = Smem<Tin, S, SC_, MODE>;
  constexpr int LN = L::LN, NT = L::NT, CT = L::CT, VEC = L::VEC, ITEMS = L::ITEMS, CV = L::CV,
                BPT = L::BPT, BIT = L::BIT, SC = L::SC;
  extern __shared__ __align__(16) float sm[];

  if (a.seg.cu) {
    if (!a.sb->seqlens_ok) return;
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.sb->status = KDA_OK;
    a.sb->detail = 0;
  }
  const int nblk = a.G * ((a.D / a.G + CT - 1) / CT);
  const int ub = blockIdx.x / nblk;
  const Unit un = resolve(a.seg, a.sb, ub);
  // of a packed batch's gradients kEnds runs the cut ones and kEnd the others
  if (MODE != kOut && a.g_seg && a.seg.cu && un.valid && un.cut != (MODE == kEnds)) return;
  // a sequence's last segment has no successor that needs its end state; the
  // gradients (with a.ckpt) need what it keeps on the way
  if (!un.valid || (MODE == kEnd && !a.ckpt && un.last)) return;
  const int tid = threadIdx.x, nl = tid % LN, cp = tid / LN;
  const Channels ch = channels_of<CT>(a, blockIdx.x - ub * nblk);
  const int d = ch.d0 + SC * cp;
  const bool live = SC * cp < ch.n;  // ch.n is a multiple of 8: both channels or none
  const int64_t ds = (int64_t)a.D * S;
  const int64_t so = (int64_t)d * S + nl * 4;

  float A2[SC][4];
  f2 h[SC][2], prod[SC][2], gs[SC][2];
  {
    const float* from = MODE == kOut && un.cut ? a.h_seg + un.slot * ds
                        : a.init && !un.cut    ? a.init + un.n * ds : nullptr;
#pragma unroll
    for (int q = 0; q < SC; ++q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) A2[q][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        h[q][i] = gs[q][i] = zero2();
        prod[q][i] = pack2(1.f, 1.f);
      }
      if (live) {
        load_vec<float, 4>(a.A + so + q * S, A2[q]);
        if (from) load_pairs(from + so + q * S, h[q]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) A2[q][i] = rate2(A2[q][i]);
    }
  }

  // the thread's elements of a tile: tokens it + m NT / CV, channels ic ..
  const int ic = tid % CV * VEC, it = tid / CV;
  const bool item = it < kTile;
  const bool ilive = item && ic < ch.n;
  float dsum[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) dsum[j] = 0.f;

  const int len = (int)(un.t1 - un.t0);
  const int tiles = (len + kTile - 1) / kTile;
  const int64_t row0 = un.t0;
  const int col = ch.d0 + ic;
  char* const slots = reinterpret_cast<char*>(sm + M::kRows);
  auto slot = [&](int i, int arr, int m) {
    return slots + (i & 1) * M::kStage + ((arr * ITEMS + m) * NT + tid) * M::kItem;
  };
  auto bslot = [&](int i, int arr, int m) {
    return slots + (i & 1) * M::kStage + M::kSlots + ((arr * BIT + m) * NT + tid) * M::kBitem;
  };

  auto copy_tile = [&](int i) {
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int t = i * kTile + it + m * (NT / CV);
      const bool in = ilive && t < len;
      const int64_t row = in ? row0 + t : row0;
      const int at = in ? col : 0;
      copy_in<M::kItem>(slot(i, 0, m), static_cast<const Tin*>(a.x) + row * a.x_stride + at, in);
      copy_in<M::kItem>(slot(i, 1, m), static_cast<const Tin*>(a.delta) + row * a.delta_stride + at,
                        in);
      if (MODE != kEnd && a.z)
        copy_in<M::kItem>(slot(i, 2, m), static_cast<const Tin*>(a.z) + row * a.z_stride + at, in);
      if (MODE == kEnds)
        copy_in<M::kItem>(slot(i, 3, m), static_cast<const Tin*>(a.dout) + row * a.D + at, in);
    }
#pragma unroll
    for (int m = 0; m < BIT; ++m) {
      const int e = (tid + m * NT) * BPT, t = i * kTile + e / S;
      const bool in = t < len;
      const int64_t row = in ? row0 + t : row0;
      const int at = ch.g * S + e % S;
      copy_in<M::kBitem>(bslot(i, 0, m), static_cast<const Tin*>(a.Bm) + row * a.B_stride + at, in);
      if (MODE != kEnd)
        copy_in<M::kBitem>(bslot(i, 1, m), static_cast<const Tin*>(a.Cm) + row * a.C_stride + at,
                           in);
    }
    copies_issued();
  };
  // the copied tile i as the rows that the scan reads
  auto fill_tile = [&](int i) {
    float bias[VEC] = {};
    if (ilive && a.delta_bias) load_vec<float, VEC>(a.delta_bias + col, bias);
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int t = it + m * (NT / CV);
      // a token behind the end leaves the state as it is: dt = 0
      const bool in = ilive && i * kTile + t < len;
      if (!item) continue;
      float dt[VEC], u[VEC];
      read_slot<Tin, VEC>(slot(i, 1, m), dt);
      read_slot<Tin, VEC>(slot(i, 0, m), u);
#pragma unroll
      for (int j = 0; j < VEC; ++j) dt[j] += bias[j];
      step_sizes<VEC>(dt, a.softplus);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        dt[j] = in ? dt[j] : 0.f;
        u[j] *= dt[j];
        if (MODE != kOut) dsum[j] += dt[j];
      }
      store_du<SC, VEC>(sm + M::kDu + t * M::kRow, ic, dt, u);
      if (MODE == kEnds) {
        float dy[VEC], z[VEC];
        read_slot<Tin, VEC>(slot(i, 3, m), dy);
        if (a.z) {
          read_slot<Tin, VEC>(slot(i, 2, m), z);
#pragma unroll
          for (int j = 0; j < VEC; ++j) dy[j] *= z[j] * sigmoid_fast(z[j]);
        }
        store_vec<VEC>(sm + M::kDy + t * CT + ic, dy);
      }
    }
#pragma unroll
    for (int m = 0; m < BIT; ++m) {
      const int e = (tid + m * NT) * BPT;
      float b[BPT];
      read_slot<Tin, BPT>(bslot(i, 0, m), b);
      store_vec<BPT>(sm + M::kB + e, b);
      if (MODE != kEnd) {
        read_slot<Tin, BPT>(bslot(i, 1, m), b);
        store_vec<BPT>(sm + M::kC + e, b);
      }
    }
  };
  float cum[SC];  // sum of dt in front of the tile's tokens (checkpoints)
#pragma unroll
  for (int q = 0; q < SC; ++q) cum[q] = 0.f;
  const int64_t tile0 = first_tile(un);
  // Two tokens' operands, loaded and their decays formed while the two tokens
  // before are applied: a store to shared memory keeps the compiler from moving
  // later loads in front of it, and a warp alone on its scheduler would wait
  // for every load and exponential.
  struct Pair {
    f2 w[2][SC][2], b[2][2], c[2][2];
    float dt[2][SC], u[2][SC], dy[2][SC];
  };
  float* pdu = sm + M::kDu + du_entry<SC>(SC * cp);
  const float* pdy = sm + M::kDy + SC * cp;
  const float* pb = sm + M::kB + nl * 4;
  const float* pc = sm + M::kC + nl * 4;
  auto fetch = [&](Pair& g, int t) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      load_du<SC>(pdu + (t + k) * M::kRow, g.dt[k], g.u[k]);
      load_pairs(pb + (t + k) * S, g.b[k]);
      if (MODE != kEnd) load_pairs(pc + (t + k) * S, g.c[k]);
      if (MODE == kEnds) load_vec<float, SC>(pdy + (t + k) * CT, g.dy[k]);
    }
  };
  auto decays = [&](Pair& g) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int q = 0; q < SC; ++q)
#pragma unroll
        for (int p = 0; p < 2; ++p)
          g.w[k][q][p] = pack2(decay(g.dt[k][q], A2[q][2 * p]), decay(g.dt[k][q], A2[q][2 * p + 1]));
  };
  auto apply = [&](const Pair& g, float (&y)[SC][4], int at) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int q = 0; q < SC; ++q) {
        const f2 uu = pack2(g.u[k][q], g.u[k][q]);
        f2 yy;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          h[q][p] = fma2(g.w[k][q][p], h[q][p], mul2(uu, g.b[k][p]));
          if (MODE == kOut) yy = p == 0 ? mul2(g.c[k][0], h[q][0]) : fma2(g.c[k][p], h[q][p], yy);
          if (MODE == kEnds) {
            prod[q][p] = mul2(prod[q][p], g.w[k][q][p]);
            gs[q][p] = fma2(mul2(prod[q][p], g.c[k][p]), pack2(g.dy[k][q], g.dy[k][q]), gs[q][p]);
          }
        }
        if (MODE == kOut) y[q][at + k] = sum2(yy);
        else cum[q] += g.dt[k][q];
      }
  };
  auto keep = [&](int t) {  // the states in front of the segment's token t
    if (a.ckpt && t < len && live) {
      const int64_t at = tile0 + t / kStep;
#pragma unroll
      for (int q = 0; q < SC; ++q) {
        store_pairs(a.ckpt + at * ds + so + q * S, h[q]);
        if (un.cut && nl == 0) a.ckpt_dt[at * a.D + d + q] = cum[q];
      }
    }
  };
  auto scan_tile = [&](int i) {
    Pair g0, g1;
    fetch(g0, 0);
    decays(g0);
#pragma unroll 1
    for (int t8 = 0; t8 < kTile; t8 += 8) {
      if (MODE != kOut) keep(i * kTile + t8);
#pragma unroll
      for (int t4 = t8; t4 < t8 + 8; t4 += 4) {
        float y[SC][4];
        fetch(g1, t4 + 2);
        apply(g0, y, 0);
        decays(g1);
        // behind the last tokens their own rows again, unused
        fetch(g0, t4 + 4 < kTile ? t4 + 4 : t4 + 2);
        apply(g1, y, 2);
        decays(g0);
        // y takes the place of the four tokens' dt: only the channel's lanes, all
        // of them in this warp, read it, and they have
        if (MODE == kOut) store_sums<SC, LN, M::kRow>(pdu + t4 * M::kRow, y, nl);
      }
    }
  };
  auto store_tile = [&](int i) {
    float skip[VEC] = {};
    if (ilive && a.D_skip) load_vec<float, VEC>(a.D_skip + col, skip);
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int t = it + m * (NT / CV);
      if (ilive && i * kTile + t < len) {
        float y[VEC], x[VEC], z[VEC];
        read_slot<Tin, VEC>(slot(i, 0, m), x);
        if (a.z) read_slot<Tin, VEC>(slot(i, 2, m), z);
        load_sums<SC, VEC>(sm + M::kDu + t * M::kRow, ic, t, y);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          y[j] = fmaf(skip[j], x[j], y[j]);
          if (a.z) y[j] *= z[j] * sigmoid_fast(z[j]);
        }
        store_vec<VEC>(static_cast<Tin*>(a.out) + (row0 + i * kTile + t) * a.D + col, y);
      }
    }
  };

  if (tiles > 0) copy_tile(0);
  for (int i = 0; i < tiles; ++i) {
    copies_landed();  // this thread's own: nobody else reads its slots
    fill_tile(i);
    __syncthreads();
    if (i + 1 < tiles) copy_tile(i + 1);
    scan_tile(i);
    __syncthreads();
    if (MODE == kOut) store_tile(i);
  }
  if (MODE != kOut) {
    if (!un.cut) return;  // the checkpoints alone were wanted
    if (live) {
#pragma unroll
      for (int q = 0; q < SC; ++q) {
        store_pairs(a.h_seg + un.slot * ds + so + q * S, h[q]);
        if (MODE == kEnds) store_pairs(a.g_seg + un.slot * ds + so + q * S, gs[q]);
      }
    }
    // dt summed over the threads that share a channel group, in order
    float* red = sm;
    if (item) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) red[it * CT + ic + j] = dsum[j];
    }
    __syncthreads();
    constexpr int ROWS = NT / CV < kTile ? NT / CV : kTile;
    for (int e = tid; e < ch.n; e += NT) {
      float s = 0.f;
      for (int r = 0; r < ROWS; ++r) s += red[r * CT + e];
      a.dt_sum[(int64_t)un.slot * a.D + ch.d0 + e] = s;
    }
  } else if (un.last && a.final_state && live) {
#pragma unroll
    for (int q = 0; q < SC; ++q) store_pairs(a.final_state + un.n * ds + so + q * S, h[q]);
  }
}

// Incoming state of every segment of a sequence, in place over the states the
// segments leave from zero: h_in[0] = init, h_in[k+1] = e^{A sum dt_k} h_in[k] + h_k;
// with g_seg the state gradients from the right likewise: g_in[last] = d_final,
// g_in[k-1] = e^{A sum dt_k} g_in[k] + g_k.
__global__ void __launch_bounds__(256) scan_combine_kernel(const Args a) {
  // a batch that was not cut uses neither h_seg nor g_seg
  if (a.seg.cu && (!a.sb->seqlens_ok || a.sb->pad[0] >= a.seg.T)) return;
  const int64_t per = (int64_t)a.D * a.S / 4;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int n = (int)(idx / per);
  if (n >= a.seg.num_seqs) return;
  const int64_t e = (idx % per) * 4;
  const int d = (int)(e / a.S);
  const int u0 = a.seg.cu ? __ldg(a.seg.seg_off + n) : n * a.seg.segs;
  const int u1 = a.seg.cu ? __ldg(a.seg.seg_off + n + 1) : u0 + a.seg.segs;
  const int64_t ds = (int64_t)a.D * a.S;
  float A2[4], in[4] = {};
  load_vec<float, 4>(a.A + e, A2);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = rate2(A2[i]);
  if (a.init) load_vec<float, 4>(a.init + n * ds + e, in);
  // eight segments' values in flight: the chain itself is a multiply-add each
  constexpr int U = 8;
  for (int ua = u0; ua < u1; ua += U) {
    float own[U][4], w[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      w[k] = own[k][0] = own[k][1] = own[k][2] = own[k][3] = 0.f;
      if (ua + k + 1 < u1) {
        load_vec<float, 4>(a.h_seg + (ua + k) * ds + e, own[k]);
        w[k] = a.dt_sum[(int64_t)(ua + k) * a.D + d];
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (ua + k >= u1) break;
      store_vec<4>(a.h_seg + (ua + k) * ds + e, in);
#pragma unroll
      for (int i = 0; i < 4; ++i) in[i] = fmaf(ex2(w[k] * A2[i]), in[i], own[k][i]);
    }
  }
  if (!a.g_seg) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) in[i] = 0.f;
  if (a.d_final) load_vec<float, 4>(a.d_final + n * ds + e, in);
  for (int ua = u1 - 1; ua >= u0; ua -= U) {
    float own[U][4], w[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      w[k] = own[k][0] = own[k][1] = own[k][2] = own[k][3] = 0.f;
      if (ua - k > u0) {
        load_vec<float, 4>(a.g_seg + (ua - k) * ds + e, own[k]);
        w[k] = a.dt_sum[(int64_t)(ua - k) * a.D + d];
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (ua - k < u0) break;
      store_vec<4>(a.g_seg + (ua - k) * ds + e, in);
#pragma unroll
      for (int i = 0; i < 4; ++i) in[i] = fmaf(ex2(w[k] * A2[i]), in[i], own[k][i]);
    }
  }
}

// One token: a thread has 4 states of a channel, of NSEQ sequences.  HBM-bound:
// the fp32 states are read once and written once; A, as large as one
// sequence's states, is kept for the NSEQ sequences.  Lane k of a channel's
// lanes forms dt and u of sequence k for all of them, and receives its sum y
// (transposed over the sequences), so what is per channel is done once.
template <typename Tin, int S, int NSEQ>
__global__ void __launch_bounds__(256) scan_step_kernel(const Args a, float* state, int N) {
  constexpr int LN = S / 4;
  static_assert(NSEQ == 1 || (NSEQ == 4 && LN >= 4), "lanes per channel");
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int nl = (int)(idx % LN);
  const int64_t cn = idx / LN;
  const int64_t n0 = cn / a.D * NSEQ;
  const int d = (int)(cn - n0 / NSEQ * a.D);
  const int ns = n0 < N ? (int)min((int64_t)NSEQ, N - n0) : 0;
  const int g = d / (a.D / a.G);
  const int64_t so = (int64_t)d * S + nl * 4, ds = (int64_t)a.D * S;
  float A2[4] = {};
  f2 h[NSEQ][2];
  Raw<Tin, 4> b[NSEQ], c[NSEQ];
#pragma unroll
  for (int k = 0; k < NSEQ; ++k) {
    h[k][0] = h[k][1] = zero2();
    b[k].zero();
    c[k].zero();
    if (k < ns) {
      load_pairs(state + (n0 + k) * ds + so, h[k]);
      b[k].load(static_cast<const Tin*>(a.Bm) + (n0 + k) * a.B_stride + g * S + nl * 4);
      c[k].load(static_cast<const Tin*>(a.Cm) + (n0 + k) * a.C_stride + g * S + nl * 4);
    }
  }
  // this lane's own sequence (all lanes the only one with NSEQ = 1)
  const int own = NSEQ == 1 ? 0 : nl;
  const bool mine = own < ns;
  float x = 0.f, z = 0.f, dt[1] = {0.f};
  if (mine) {
    const int64_t n = n0 + own;
    x = Elem<Tin>::load(static_cast<const Tin*>(a.x) + n * a.x_stride + d);
    dt[0] = Elem<Tin>::load(static_cast<const Tin*>(a.delta) + n * a.delta_stride + d);
    if (a.z) z = Elem<Tin>::load(static_cast<const Tin*>(a.z) + n * a.z_stride + d);
    if (a.delta_bias) dt[0] += a.delta_bias[d];
  }
  if (ns > 0) load_vec<float, 4>(a.A + so, A2);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = rate2(A2[i]);
  step_sizes<1>(dt, a.softplus);
  const float u = dt[0] * x;
  float y[4] = {};
#pragma unroll
  for (int k = 0; k < NSEQ; ++k) {
    const float sk = NSEQ == 1 ? dt[0] : __shfl_sync(0xffffffffu, dt[0], k, LN);
    const float uk = NSEQ == 1 ? u : __shfl_sync(0xffffffffu, u, k, LN);
    const f2 uu = pack2(uk, uk);
    const f2 w0 = pack2(decay(sk, A2[0]), decay(sk, A2[1]));
    const f2 w1 = pack2(decay(sk, A2[2]), decay(sk, A2[3]));
    h[k][0] = fma2(w0, h[k][0], mul2(uu, pack2(b[k].at(0), b[k].at(1))));
    h[k][1] = fma2(w1, h[k][1], mul2(uu, pack2(b[k].at(2), b[k].at(3))));
    if (k < ns) store_pairs(state + (n0 + k) * ds + so, h[k]);
    y[k] = sum2(fma2(pack2(c[k].at(2), c[k].at(3)), h[k][1],
                     mul2(pack2(c[k].at(0), c[k].at(1)), h[k][0])));
  }
  float out;
  if constexpr (NSEQ == 1) {
    out = y[0];
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
  } else {
    out = sum_lanes<LN>(y, nl).x;
  }
  if (mine && nl < NSEQ) {
    if (a.D_skip) out = fmaf(a.D_skip[d], x, out);
    if (a.z) out *= z * sigmoid_fast(z);
    Elem<Tin>::store(static_cast<Tin*>(a.out) + (n0 + own) * a.D + d, out);
  }
}

// Packed batches: validates the offsets, then chooses the segment length
// (seg_len or more where a sequence is longer than cut_above, else the whole
// batch's length, so that every sequence is one unit) and writes seg_off and, for
// a batch left whole, order.  Longest first pays up to kMaxOrder sequences; the
// ranks take N^2 comparisons of one CTA.  Ordered and not, us, 16,384 tokens x
// 1024 x 16: 159 and 211 with 64 sequences, 140 and 171 with 128, 159 and 175
// with 256, 206 and 210 with 512, 319 and 293 with 1024, 616 and 480 with 2048.
constexpr int kMaxOrder = 512;
constexpr int kMaxSegs = 148;  // of a sequence (plan_segments)

__global__ void __launch_bounds__(1024) scan_plan_kernel(const int32_t* __restrict__ cu, int N,
                                                         int T, StatusBlock* sb, int cut_above,
                                                         int seg_len,
                                                         int32_t* __restrict__ seg_off,
                                                         int32_t* __restrict__ order) {
  __shared__ int bad, longest, carry;
  __shared__ int wsum[32], lens[kMaxOrder];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) {
    bad = (cu[0] != 0 || cu[N] != T) ? 1 : 0;
    longest = 0;
    carry = 0;
  }
  __syncthreads();
  int most = 0;
  for (int n = tid; n < N; n += 1024) {
    const int len = cu[n + 1] - cu[n];
    if (cu[n + 1] < cu[n]) atomicOr(&bad, 1);
    most = max(most, len);
    if (n < kMaxOrder) lens[n] = len;
  }
  atomicMax(&longest, most);
  __syncthreads();
  if (tid == 0) {
    sb->status = bad ? KDA_ERR_BAD_SEQLENS : KDA_OK;
    sb->detail = 0;
    sb->never_set = 0;
    sb->seqlens_ok = bad ? 0 : 1;
  }
  if (bad) return;
  int sl = T;
  if (longest > cut_above) {  // no more than kMaxSegs of any sequence
    sl = (longest - 1) / (kMaxSegs * kTile) * kTile + kTile;
    if (sl < seg_len) sl = seg_len;
  }
  if (tid == 0) sb->pad[0] = sl;
  // longest first; batches of more sequences keep their order
  for (int n = tid; n < N && sl == T; n += 1024) {
    int rank = n;
    if (N <= kMaxOrder) {
      const int len = lens[n];
      rank = 0;
      for (int m = 0; m < N; ++m) rank += lens[m] > len || (lens[m] == len && m < n);
    }
    order[rank] = n;
  }
  // exclusive prefix sums of the segment counts, 1024 sequences a step
  for (int n0 = 0; n0 < N; n0 += 1024) {
    const int n = n0 + tid;
    int c = 0;
    if (n < N) {
      const int len = cu[n + 1] - cu[n];
      c = len > 0 ? 1 + (len - 1) / sl : 1;
    }
    int s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += v;
    }
    if (lane == 31) wsum[wid] = s;
    __syncthreads();
    if (wid == 0) {
      int v = wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      wsum[lane] = v;
    }
    __syncthreads();
    const int before = carry + (wid ? wsum[wid - 1] : 0) + s - c;
    if (n < N) seg_off[n] = before;
    if (n == N - 1) seg_off[N] = before + c;
    __syncthreads();
    if (tid == 0) carry += wsum[31];
    __syncthreads();
  }
}

template <typename Tin, int S, int SC, int MODE>
cudaError_t launch_one(const Args& a, cudaStream_t st) {
  using L = Layout<S, SC>;
  constexpr size_t bytes = Smem<Tin, S, SC, MODE>::bytes();
  if (bytes > 48 * 1024)
    if (cudaError_t e = cudaFuncSetAttribute(scan_fwd_kernel<Tin, S, SC, MODE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)bytes))
      return e;
  const unsigned grid = (unsigned)((int64_t)a.seg.units * channel_blocks(a.D, a.G, L::CT));
  scan_fwd_kernel<Tin, S, SC, MODE><<<grid, L::NT, bytes, st>>>(a);
  return cudaGetLastError();
}

template <typename Tin, int MODE>
cudaError_t launch_mode(const Args& a, cudaStream_t st) {
  if constexpr (MODE == kOut) {  // the other modes' batches fill the GPU with pairs
    if (!a.seg.wide) {
      switch (a.S) {
        case 8: return launch_one<Tin, 8, 1, MODE>(a, st);
        case 16: return launch_one<Tin, 16, 1, MODE>(a, st);
        case 32: return launch_one<Tin, 32, 1, MODE>(a, st);
        case 64: return launch_one<Tin, 64, 1, MODE>(a, st);
        default: return launch_one<Tin, 128, 1, MODE>(a, st);
      }
    }
  }
  switch (a.S) {
    case 8: return launch_one<Tin, 8, 1, MODE>(a, st);  // the lanes of a channel pair are few
    case 16: return launch_one<Tin, 16, 2, MODE>(a, st);
    case 32: return launch_one<Tin, 32, 2, MODE>(a, st);
    case 64: return launch_one<Tin, 64, 2, MODE>(a, st);
    default: return launch_one<Tin, 128, 2, MODE>(a, st);
  }
}

template <int MODE>
cudaError_t launch_typed(const Args& a, kda_dtype dt, cudaStream_t st) {
  return dt == KDA_BF16 ? launch_mode<__nv_bfloat16, MODE>(a, st)
                        : launch_mode<float, MODE>(a, st);
}

template <typename Tin, int S>
cudaError_t launch_step_s(const Args& a, float* state, int N, cudaStream_t st) {
  if constexpr (S >= 16) {
    constexpr int NSEQ = 4;
    // threads with four sequences each
    const int64_t many = ((int64_t)N + NSEQ - 1) / NSEQ * a.D * (S / 4);
    // From 512 such threads an SM on; one sequence a thread against four, D =
    // 4096, S = 16, bf16: 3.1 and 3.2 us at 221 threads an SM (8 sequences), 7.4
    // and 6.4 at 886, 12.3 and 10.7 at 1771, 42.0 and 32.8 at 7085 (256).
    if (many >= 148 * 512) {
      scan_step_kernel<Tin, S, NSEQ><<<(unsigned)((many + 255) / 256), 256, 0, st>>>(a, state, N);
      return cudaGetLastError();
    }
  }
  const int64_t all = (int64_t)N * a.D * (S / 4);
  scan_step_kernel<Tin, S, 1><<<(unsigned)((all + 255) / 256), 256, 0, st>>>(a, state, N);
  return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_step(const Args& a, float* state, int N, cudaStream_t st) {
  switch (a.S) {
    case 8: return launch_step_s<Tin, 8>(a, state, N, st);
    case 16: return launch_step_s<Tin, 16>(a, state, N, st);
    case 32: return launch_step_s<Tin, 32>(a, state, N, st);
    case 64: return launch_step_s<Tin, 64>(a, state, N, st);
    default: return launch_step_s<Tin, 128>(a, state, N, st);
  }
}

}  // namespace

cudaError_t launch_scan_plan(const Args& a, int32_t* seg_off, int32_t* order, cudaStream_t st) {
  scan_plan_kernel<<<1, 1024, 0, st>>>(a.seg.cu, a.seg.num_seqs, a.seg.T, a.sb, a.seg.cut_above,
                                       a.seg.seg_len, seg_off, order);
  return cudaGetLastError();
}

cudaError_t launch_ends(const Args& a, kda_dtype dt, cudaStream_t st) {
  if (!a.g_seg || a.seg.cu)
    if (cudaError_t e = launch_typed<kEnd>(a, dt, st)) return e;
  if (a.g_seg)
    if (cudaError_t e = launch_typed<kEnds>(a, dt, st)) return e;
  if (!a.split) return cudaSuccess;
  const int64_t items = (int64_t)a.seg.num_seqs * a.D * a.S / 4;
  scan_combine_kernel<<<(unsigned)((items + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

bool sizes_ok(int D, int S, int G) {
  if (S != 8 && S != 16 && S != 32 && S != 64 && S != 128) return false;
  return D <= (1 << 24) && D % G == 0 && D / G % 8 == 0;
}

// How a batch is spread over the GPU.  `warps` is its sequences' warps with two
// channels a thread.  Dense batches (us for two channels a thread, one channel,
// and cut; S = 16, T = 2048, D = 2048, that is 128 warps a sequence):
//   from SMs x 6: two channels a thread (289, 324, 406 at 6.9 warps an SM;
//     388, 395, 514 at 8.6);
//   from SMs x 3: one channel a thread, twice the warps (207, 200, 229 at 3.5;
//     289, 258, 311 at 5.2);
//   fewer: the sequences are cut until there are SMs x 16 warps, which costs
//     a second pass over all but the last segments (200, 144, 66 at 0.9; 205,
//     199, 159 at 2.6).
// The gradients' first pass over the segments is needed anyway and their walk
// has two warps a scheduler at most: cut until there are SMs x 32 warps, four
// waves (493 us; 555 with SMs x 8 or 16 at 3.5 warps an SM).  A sequence has
// kMaxSegs segments at most: their combination is one chain, 0.1 us a segment and
// 0.4 in the gradients (65,536 tokens x 64 channels, forward and gradients: 107
// and 226 us, 138 and 552 with 512 and 1024 segments; gradients of 16,384 x 256
// in 202 us, 253 with 256 segments).
// Packed batches do not show their lengths to the host: two channels a thread,
// and a cut (the plan kernel's choice) into halves of the even share of SMs x
// 16 warps, where one sequence is longer than three shares.  12,000 tokens x
// 4096 x 16 in 16 sequences, the longest of 2.3, 3.1, 4.6, 6.9 shares: uncut
// 401, 491, 669, 930 us; cut at half a share 442, 442, 461, 508 (at one share
// 475, 479, 523, 591; at four 409, 499, 953, 1002); gradients uncut 1269, 1532,
// 2084, 2906, cut at half a share 1442, 1457, 1410, 1363.
Segments plan_segments(const int32_t* cu, int num_seqs, int B, int T, int D, int S, bool bwd) {
  constexpr int64_t kSms = 148;
  Segments m{};
  m.cu = cu;
  m.num_seqs = cu ? num_seqs : B;
  m.T = T;
  const int64_t per_seq = ((int64_t)D * S + 255) / 256;
  const int64_t warps = m.num_seqs * per_seq;
  int64_t len = T;
  if (cu) {
    m.wide = true;
    len = T * per_seq / (kSms * 32);
    if (len < kMinSeg) len = kMinSeg;
    len = (len + kTile - 1) / kTile * kTile;
    const int64_t above = 6 * len < 512 ? 512 : 6 * len;  // shorter: the extra launches
    m.cut_above = (int)(above < T ? above : T);
    if (m.cut_above == T) len = T;
  } else {
    m.wide = warps >= kSms * 6;
    if (warps < kSms * (bwd ? 32 : 3)) {
      int64_t segs = kSms * (bwd ? 32 : 16) / warps;
      if (segs > T / kMinSeg) segs = T / kMinSeg;
      if (segs > kMaxSegs) segs = kMaxSegs;
      if (segs >= 2) {
        m.wide = true;
        len = (T + segs - 1) / segs;
      }
    }
    len = (len + kTile - 1) / kTile * kTile;
  }
  m.seg_len = (int)(len < T ? len : T);
  m.segs = (T + m.seg_len - 1) / m.seg_len;
  m.units = cu ? num_seqs + T / m.seg_len : B * m.segs;
  return m;
}

// checks shared by the prompt, step and gradient entries
kda_status check_scan(kda_dtype dt, int D, int S, int G, int64_t xs, int64_t ds, int64_t bs,
                      int64_t cs, const void* z, int64_t zs) {
  if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (D <= 0 || S <= 0 || G <= 0) return KDA_ERR_INVALID_ARG;
  if (!sizes_ok(D, S, G)) return KDA_ERR_UNSUPPORTED;
  const int64_t es = elem_bytes(dt), w = (int64_t)G * S;
  if (!stride_ok(xs, D, es) || !stride_ok(ds, D, es) || !stride_ok(bs, w, es) ||
      !stride_ok(cs, w, es) || (z && !stride_ok(zs, D, es)))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

Args scan_args(const void* x, int64_t x_stride, const void* delta, int64_t delta_stride,
               const float* A, const void* Bm, int64_t B_stride, const void* Cm,
               int64_t C_stride, const float* D_skip, const void* z, int64_t z_stride,
               const float* delta_bias, int delta_softplus, int D, int S, int G) {
  Args a{};
  a.x = x;
  a.delta = delta;
  a.Bm = Bm;
  a.Cm = Cm;
  a.z = z;
  a.x_stride = x_stride;
  a.delta_stride = delta_stride;
  a.B_stride = B_stride;
  a.C_stride = C_stride;
  a.z_stride = z_stride;
  a.A = A;
  a.D_skip = D_skip;
  a.delta_bias = delta_bias;
  a.softplus = delta_softplus != 0;
  a.D = D;
  a.S = S;
  a.G = G;
  return a;
}

}  // namespace scan
}  // namespace kda

using namespace kda;
using namespace kda::scan;

extern "C" {

size_t kda_selective_scan_fwd_workspace_size(int B, int T, int D, int S, int G, int num_seqs) {
  if (B <= 0 || T <= 0 || D <= 0 || G <= 0 || num_seqs < 0 || !sizes_ok(D, S, G) ||
      (int64_t)B * T > kMaxRows || !units_ok(num_seqs, T))
    return 0;
  static const int32_t packed = 0;  // only whether there are offsets matters here
  const Segments m = plan_segments(num_seqs > 0 && B == 1 ? &packed : nullptr, num_seqs, B, T,
                                   D, S, false);
  size_t b = kStatusBytes;
  if (m.cu) b += 2 * align256(sizeof(int32_t) * ((size_t)num_seqs + 1));
  if (m.segs > 1)
    b += align256(sizeof(float) * (size_t)m.units * D * S) +
         align256(sizeof(float) * (size_t)m.units * D);
  return b;
}

kda_status kda_selective_scan_fwd(const void* x, int64_t x_stride, const void* delta,
                                  int64_t delta_stride, const float* A, const void* Bm,
                                  int64_t B_stride, const void* Cm, int64_t C_stride,
                                  const float* D_skip, const void* z, int64_t z_stride,
                                  const float* delta_bias, int delta_softplus,
                                  kda_dtype in_dtype, const float* init_state,
                                  const int32_t* cu_seqlens, int num_seqs, int B, int T, int D,
                                  int S, int G, void* out, float* final_state, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!x || !delta || !A || !Bm || !Cm || !out || !workspace) return KDA_ERR_INVALID_ARG;
  if (kda_status s = check_batch(cu_seqlens, num_seqs, B, T)) return s;
  if (!units_ok(num_seqs, T)) return KDA_ERR_UNSUPPORTED;
  if (kda_status s = check_scan(in_dtype, D, S, G, x_stride, delta_stride, B_stride, C_stride, z,
                                z_stride))
    return s;
  const int64_t n = (int64_t)B * T, es = elem_bytes(in_dtype), w = (int64_t)G * S;
  const int64_t N = cu_seqlens ? num_seqs : B, state = N * D * S * 4;
  const size_t need =
      kda_selective_scan_fwd_workspace_size(B, T, D, S, G, cu_seqlens ? num_seqs : 0);
  const Span ins[] = {{x, row_bytes(n, x_stride, D, es)},
                      {delta, row_bytes(n, delta_stride, D, es)},
                      {A, (int64_t)D * S * 4},
                      {Bm, row_bytes(n, B_stride, w, es)},
                      {Cm, row_bytes(n, C_stride, w, es)},
                      {D_skip, (int64_t)D * 4},
                      {z, row_bytes(n, z_stride, D, es)},
                      {delta_bias, (int64_t)D * 4},
                      {cu_seqlens, (N + 1) * 4}};
  const Span outs[] = {{out, n * D * es}, {final_state, state}, {workspace, (int64_t)need}};
  if (kda_status s = check_spans(ins, outs)) return s;
  // init_state may be final_state: it has been read when that is written
  const Span init = {init_state, state};
  if (!span_aligned(init)) return KDA_ERR_MISALIGNED;
  for (const Span& o : outs)
    if (!(o.p == final_state && init_state == final_state) && spans_overlap(o, init))
      return KDA_ERR_INVALID_ARG;
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
  Args a = scan_args(x, x_stride, delta, delta_stride, A, Bm, B_stride, Cm, C_stride, D_skip, z,
                     z_stride, delta_bias, delta_softplus, D, S, G);
  a.seg = plan_segments(cu_seqlens, num_seqs, B, T, D, S, false);
  if ((int64_t)a.seg.units * channel_blocks(D, G, 8) > 0x7fffffffLL ||
      N * D / 256 * (S / 4) > 0x7ffffff0LL)
    return KDA_ERR_UNSUPPORTED;
  a.init = init_state;
  a.final_state = final_state;
  a.out = out;
  a.sb = static_cast<StatusBlock*>(workspace);
  char* tail = static_cast<char*>(workspace) + kStatusBytes;
  cudaStream_t st = (cudaStream_t)stream;
  if (cu_seqlens) {
    const size_t part = align256(sizeof(int32_t) * ((size_t)num_seqs + 1));
    int32_t* off = reinterpret_cast<int32_t*>(tail);
    int32_t* order = reinterpret_cast<int32_t*>(tail + part);
    tail += 2 * part;
    a.seg.seg_off = off;
    a.seg.order = order;
    if (cudaError_t e = launch_scan_plan(a, off, order, st)) return cuda_failure(e);
  }
  a.split = a.seg.segs > 1;
  if (a.split) {
    a.h_seg = reinterpret_cast<float*>(tail);
    tail += align256(sizeof(float) * (size_t)a.seg.units * D * S);
    a.dt_sum = reinterpret_cast<float*>(tail);
  }
  if (a.split)
    if (cudaError_t e = launch_ends(a, in_dtype, st)) return cuda_failure(e);
  const cudaError_t e = launch_typed<kOut>(a, in_dtype, st);
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

kda_status kda_selective_scan_step(const void* x, int64_t x_stride, const void* delta,
                                   int64_t delta_stride, const float* A, const void* Bm,
                                   int64_t B_stride, const void* Cm, int64_t C_stride,
                                   const float* D_skip, const void* z, int64_t z_stride,
                                   const float* delta_bias, int delta_softplus,
                                   kda_dtype in_dtype, float* state, int N, int D, int S, int G,
                                   void* out, void* stream) {
  if (!x || !delta || !A || !Bm || !Cm || !state || !out) return KDA_ERR_INVALID_ARG;
  if (N <= 0) return KDA_ERR_INVALID_ARG;
  if (kda_status s = check_scan(in_dtype, D, S, G, x_stride, delta_stride, B_stride, C_stride, z,
                                z_stride))
    return s;
  const int64_t es = elem_bytes(in_dtype), w = (int64_t)G * S;
  const Span ins[] = {{x, row_bytes(N, x_stride, D, es)},
                      {delta, row_bytes(N, delta_stride, D, es)},
                      {A, (int64_t)D * S * 4},
                      {Bm, row_bytes(N, B_stride, w, es)},
                      {Cm, row_bytes(N, C_stride, w, es)},
                      {D_skip, (int64_t)D * 4},
                      {z, row_bytes(N, z_stride, D, es)},
                      {delta_bias, (int64_t)D * 4}};
  const Span outs[] = {{out, (int64_t)N * D * es}, {state, (int64_t)N * D * S * 4}};
  if (kda_status s = check_spans(ins, outs)) return s;
  if ((int64_t)N * D / 256 * (S / 4) > 0x7ffffff0LL) return KDA_ERR_UNSUPPORTED;
  Args a = scan_args(x, x_stride, delta, delta_stride, A, Bm, B_stride, Cm, C_stride, D_skip, z,
                     z_stride, delta_bias, delta_softplus, D, S, G);
  a.out = out;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = in_dtype == KDA_BF16 ? launch_step<__nv_bfloat16>(a, state, N, st)
                                             : launch_step<float>(a, state, N, st);
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

}  // extern "C"
