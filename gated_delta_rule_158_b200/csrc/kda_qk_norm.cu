// kda_qk_norm.cu -- norms of query and key rows with the position rotation,
// forward and gradients.
//
//   r = 1 / sqrt(c sum x^2 + eps),  u = x r w,  out = R(position) u
//   du = R^T dout,  dw = sum du x r,  dx = r (du w - x r c sum(du w x r))
//
// HBM-bound: every row is read once and written once (the gradients add one
// fp32 row each way).  A row of d elements lies in a group of L lanes, 8
// elements a lane, so the row's sum is log2 L shuffles; a lane's elements are
// chosen so that both of a turning pair are its own.  Blocks walk over tiles of
// whole tokens, all their heads, so that an angle's cosine and sine are formed
// once per token (fp64 product and reduction to one turn, then fp32 sincospi)
// and read from shared memory by all heads, a tile ahead; the next rows are in
// flight while a step's are worked on.
//
// Measured on a B200 (6455 GB/s copy): unit rows of 16,384 tokens x 64 heads x
// 128, bf16, 90 us = 6.0 TB/s (130 us before the blocks stayed and kept rows in
// flight, 103 us before a group kept to its heads); 8192 tokens x 40 heads with
// half of each row turned 47 us (the instructions of the turn and the weights,
// 74 % of the issue slots; 24 bytes spilled at the 64 registers that four blocks an
// SM leave) and its gradients 79 us = 5.3 TB/s.  16 tokens x 40 heads: 8 us, one
// block a token behind its fp64 angles.
#include <math.h>

#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int kNormThreads = 256;
// rows per lane group and step, and as many in flight: 64 bytes a lane, 96 with
// the gradients' fp32 cotangent beside bf16 rows
template <typename Tin>
constexpr int kRows = 8 / (int)sizeof(Tin);
constexpr int kBwdRows = 2;
constexpr int kMaxTokens = 16;  // rotated tokens per tile (two shared tables: 2 x 16 x 256 floats)

struct NormArgs {
  const void* q;
  const void* k;
  int64_t q_stride, k_stride;
  const float* q_weight;
  const float* k_weight;
  const int32_t* positions;
  const float* inv_freq;
  int tokens, Hq, Hk, d, rot;
  float c, eps;
  bool pairs;
  void* q_out;
  void* k_out;
  int per_block;  // tokens per tile
  int hs, ts;     // heads x tokens of a block's lane groups
  int blocks;
  // gradients
  const float* dq_out;
  const float* dk_out;
  float* dq;
  float* dk;
  float* partial;  // [blocks][2][d]
};

// cos and sin of positions[t0 + i] * inv_freq[j] for the tile's tokens: a token's
// cosines, then its sines
__device__ __forceinline__ void fill_turns(const NormArgs& a, int t0, int nt, float* tab) {
  const int half = a.rot >> 1;
  for (int e = threadIdx.x; e < nt * half; e += kNormThreads) {
    const int i = e / half, j = e - i * half;
    // in half turns; |product| < 2^31 * inv_freq, so the fraction keeps about
    // 2^-22 of a half turn or better for any 32-bit position at inv_freq <= 1
    const double x = (double)a.positions[t0 + i] * (double)a.inv_freq[j] * 0.31830988618379067154;
    const double f = x - 2.0 * rint(0.5 * x);
    float s, co;
    sincospif((float)f, &s, &co);
    tab[i * a.rot + j] = co;
    tab[i * a.rot + half + j] = s;
  }
}

enum Rot { kNoRot, kHalves, kPairs };

// A lane's 8 elements of a row are two pieces of 4: neighbours, but with the
// halves of the rotated part turning together, piece 0 from its first half and
// piece 1 from the second, so that both elements of a pair are in the lane.
struct Pieces {
  int o0, o1;
};
template <int ROT>
__device__ __forceinline__ Pieces pieces_of(const NormArgs& a, int l) {
  Pieces p;
  p.o0 = 8 * l;
  p.o1 = 8 * l + 4;
  if (ROT == kHalves && 8 * l < a.rot) {
    p.o0 = 4 * l;
    p.o1 = a.rot / 2 + 4 * l;
  }
  return p;
}

template <typename T, int ROT>
struct RowRaw {  // 8 elements as they lie in memory
  static constexpr int N = ROT == kHalves ? 2 : 1;
  Raw<T, 8 / N> r[N];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i].zero();
  }
  __device__ __forceinline__ void load(const T* row, const Pieces& p) {
    r[0].load(row + p.o0);
    if constexpr (N == 2) r[1].load(row + p.o1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r[i / (8 / N)].at(i % (8 / N));
  }
};

template <int ROT, typename T>
__device__ __forceinline__ void store_row(T* row, const Pieces& p, const float (&v)[8]) {
  if constexpr (ROT == kHalves) {
    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    store_vec<4>(row + p.o0, lo);
    store_vec<4>(row + p.o1, hi);
  } else {
    store_vec<8>(row + p.o0, v);
  }
}

template <int ROT>
__device__ __forceinline__ void load_weight(const float* w, const Pieces& p, float (&v)[8]) {
  float lo[4], hi[4];
  load_vec<float, 4>(w + p.o0, lo);
  load_vec<float, 4>(w + p.o1, hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = lo[i];
    v[4 + i] = hi[i];
  }
}

// Turns the lane's four pairs, numbers 4 l .. of the row, by the angles of the
// tile's token tok; sgn = 1 forward, -1 back.
template <int ROT>
__device__ __forceinline__ void turn(const NormArgs& a, const float* tab, int tok, int l,
                                     float sgn, float (&v)[8]) {
  if (ROT == kNoRot || 8 * l >= a.rot) return;
  const float* at = tab + tok * a.rot + 4 * l;
  if constexpr (ROT == kHalves) {
    f2 c[2], s[2];
    load_pairs(at, c);
    load_pairs(at + (a.rot >> 1), s);
    const f2 one = pack2(sgn, sgn), neg = pack2(-sgn, -sgn);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f2 p = pack2(v[2 * i], v[2 * i + 1]), q = pack2(v[4 + 2 * i], v[5 + 2 * i]);
      unpack2(fma2(p, c[i], mul2(q, mul2(s[i], neg))), v[2 * i], v[2 * i + 1]);
      unpack2(fma2(q, c[i], mul2(p, mul2(s[i], one))), v[4 + 2 * i], v[5 + 2 * i]);
    }
  } else {
    float c[4], s[4];
    load_vec<float, 4>(at, c);
    load_vec<float, 4>(at + (a.rot >> 1), s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = v[2 * i], q = v[2 * i + 1], sn = sgn * s[i];
      v[2 * i] = p * c[i] - q * sn;
      v[2 * i + 1] = q * c[i] + p * sn;
    }
  }
}

template <int L>
__device__ __forceinline__ float group_sum(float s) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o, L);
  return s;
}

// A block's lane groups stand for HS heads x TS tokens of its tile; a group
// takes every HS-th head and, of a head, U tokens TS apart at a time.  What
// depends on the head (its tensor, row length, weight) is chosen once per head.
template <typename Tin>
struct Head {
  const Tin* in;       // the group's first row of the tile
  int64_t step;        // to its next
  bool isq;
};

template <typename Tin>
__device__ __forceinline__ Head<Tin> head_of(const NormArgs& a, int h, int64_t t) {
  Head<Tin> r;
  r.isq = h < a.Hq;
  const int64_t stride = r.isq ? a.q_stride : a.k_stride;
  r.in = static_cast<const Tin*>(r.isq ? a.q : a.k) + (r.isq ? h : h - a.Hq) * a.d + t * stride;
  r.step = a.ts * stride;
  return r;
}

// the same of a dense q- or k-shaped tensor
__device__ __forceinline__ int64_t dense_row(const NormArgs& a, int h, int64_t t) {
  return h < a.Hq ? (t * a.Hq + h) * a.d : (t * a.Hk + h - a.Hq) * a.d;
}
__device__ __forceinline__ int64_t dense_step(const NormArgs& a, int h) {
  return (int64_t)a.ts * (h < a.Hq ? a.Hq : a.Hk) * a.d;
}

// Blocks walk over tiles of per_block <= U TS tokens; the next head's rows (of
// this tile or the next) are in flight while a head's are worked on.
template <typename Tin, int L, int ROT>
__global__ void __launch_bounds__(kNormThreads, 4) qk_norm_fwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) float tab[];
  constexpr int U = kRows<Tin>;
  const int l = threadIdx.x % L, grp = threadIdx.x / L;
  const int hs = grp % a.hs, ts = grp / a.hs;
  const bool act = 8 * l < a.d && ts < a.ts;
  const Pieces pc = pieces_of<ROT>(a, l);
  const int H = a.Hq + a.Hk;
  const int tiles = (int)(((int64_t)a.tokens + a.per_block - 1) / a.per_block);
  RowRaw<Tin, ROT> next[U];
  auto fetch = [&](int tile, int h) {
    const int t0 = tile * a.per_block, nt = min(a.per_block, a.tokens - t0);
    const Head<Tin> r = head_of<Tin>(a, h, t0 + ts);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      next[u].zero();
      if (act && h < H && ts + u * a.ts < nt) next[u].load(r.in + u * r.step, pc);
    }
  };
  if ((int)blockIdx.x < tiles) {
    fetch(blockIdx.x, hs);
    if (ROT != kNoRot) {
      const int t0 = blockIdx.x * a.per_block;
      fill_turns(a, t0, min(a.per_block, a.tokens - t0), tab);
    }
  }
  for (int tile = blockIdx.x, k = 0; tile < tiles; tile += gridDim.x, ++k) {
    const int t0 = tile * a.per_block, nt = min(a.per_block, a.tokens - t0);
    const float* tb = tab;
    if (ROT != kNoRot) {
      // the table of the tile after this one is formed while this is worked on:
      // two tables, one barrier per tile
      tb = tab + (k & 1) * a.per_block * a.rot;
      __syncthreads();
      const int64_t t2 = ((int64_t)tile + gridDim.x) * a.per_block;
      if (t2 < a.tokens)
        fill_turns(a, (int)t2, (int)min((int64_t)a.per_block, a.tokens - t2),
                   tab + (~k & 1) * a.per_block * a.rot);
    }
    for (int h0 = 0; h0 < H; h0 += a.hs) {
      const int h = h0 + hs;
      RowRaw<Tin, ROT> cur[U];
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = next[u];
      if (h0 + a.hs < H) fetch(tile, h + a.hs);
      else if (tile + (int)gridDim.x < tiles) fetch(tile + gridDim.x, hs);
      const bool isq = h < a.Hq;
      Tin* out = static_cast<Tin*>(isq ? a.q_out : a.k_out) + dense_row(a, h, t0 + ts);
      const int64_t step = dense_step(a, h);
      const float* wp = isq ? a.q_weight : a.k_weight;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = ts + u * a.ts;
        float x[8], ss = 0.f;
        cur[u].get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        const float f = rsqrtf(fmaf(a.c, group_sum<L>(ss), a.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= f;
        if (act && h < H && t < nt) {
          if (wp) {
            float w[8];
            load_weight<ROT>(wp, pc, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= w[i];
          }
          turn<ROT>(a, tb, t, l, 1.f, x);
          store_row<ROT>(out + u * step, pc, x);
        }
      }
    }
  }
}

// A lane's share of dweight (its 8 columns, the rows of its group) stays in
// registers over the walk, is added over the block's groups in order, and
// leaves as one partial row per block.
template <typename Tin, int L, int ROT>
__global__ void __launch_bounds__(kNormThreads, 2) qk_norm_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) float tab[];
  constexpr int G = kNormThreads / L;
  constexpr int U = kBwdRows;
  const int l = threadIdx.x % L, grp = threadIdx.x / L;
  const int hs = grp % a.hs, ts = grp / a.hs;
  const bool act = 8 * l < a.d && ts < a.ts;
  const Pieces pc = pieces_of<ROT>(a, l);
  const int H = a.Hq + a.Hk;
  const int tiles = (int)(((int64_t)a.tokens + a.per_block - 1) / a.per_block);
  float gq[8], gk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) gq[i] = gk[i] = 0.f;
  RowRaw<Tin, ROT> nx[U];
  RowRaw<float, ROT> nd[U];
  auto fetch = [&](int tile, int h) {
    const int t0 = tile * a.per_block, nt = min(a.per_block, a.tokens - t0);
    const Head<Tin> r = head_of<Tin>(a, h, t0 + ts);
    const float* dy = (r.isq ? a.dq_out : a.dk_out) + dense_row(a, h, t0 + ts);
    const int64_t step = dense_step(a, h);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      nx[u].zero();
      nd[u].zero();
      if (act && h < H && ts + u * a.ts < nt) {
        nx[u].load(r.in + u * r.step, pc);
        nd[u].load(dy + u * step, pc);
      }
    }
  };
  if ((int)blockIdx.x < tiles) {
    fetch(blockIdx.x, hs);
    if (ROT != kNoRot) {
      const int t0 = blockIdx.x * a.per_block;
      fill_turns(a, t0, min(a.per_block, a.tokens - t0), tab);
    }
  }
  for (int tile = blockIdx.x, k = 0; tile < tiles; tile += a.blocks, ++k) {
    const int t0 = tile * a.per_block, nt = min(a.per_block, a.tokens - t0);
    const float* tb = tab;
    if (ROT != kNoRot) {
      tb = tab + (k & 1) * a.per_block * a.rot;
      __syncthreads();
      const int64_t t2 = ((int64_t)tile + a.blocks) * a.per_block;
      if (t2 < a.tokens)
        fill_turns(a, (int)t2, (int)min((int64_t)a.per_block, a.tokens - t2),
                   tab + (~k & 1) * a.per_block * a.rot);
    }
    for (int h0 = 0; h0 < H; h0 += a.hs) {
      const int h = h0 + hs;
      RowRaw<Tin, ROT> cx[U];
      RowRaw<float, ROT> cd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        cx[u] = nx[u];
        cd[u] = nd[u];
      }
      if (h0 + a.hs < H) fetch(tile, h + a.hs);
      else if (tile + a.blocks < tiles) fetch(tile + a.blocks, hs);
      const bool isq = h < a.Hq;
      float* out = (isq ? a.dq : a.dk) + dense_row(a, h, t0 + ts);
      const int64_t step = dense_step(a, h);
      const float* wp = isq ? a.q_weight : a.k_weight;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.f;
      if (wp && act) load_weight<ROT>(wp, pc, w);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = ts + u * a.ts;
        const bool in = act && h < H && t < nt;
        float x[8], dy[8], ss = 0.f;
        cx[u].get(x);
        cd[u].get(dy);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        const float f = rsqrtf(fmaf(a.c, group_sum<L>(ss), a.eps));
        if (in) turn<ROT>(a, tb, t, l, -1.f, dy);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= f;
        if (a.partial) {  // rows past the end are zero
          if (isq) {
#pragma unroll
            for (int i = 0; i < 8; ++i) gq[i] = fmaf(dy[i], x[i], gq[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) gk[i] = fmaf(dy[i], x[i], gk[i]);
          }
        }
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dy[i] *= w[i];
          m = fmaf(dy[i], x[i], m);
        }
        m = a.c * group_sum<L>(m);
#pragma unroll
        for (int i = 0; i < 8; ++i) dy[i] = f * fmaf(-x[i], m, dy[i]);
        if (in) store_row<ROT>(out + u * step, pc, dy);
      }
    }
  }
  if (!a.partial) return;
  // [group][2][8 L] over the shared memory of the table
  float* red = tab;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int col = i < 4 ? pc.o0 + i : pc.o1 + i - 4;
    red[(grp * 2 + 0) * 8 * L + col] = gq[i];
    red[(grp * 2 + 1) * 8 * L + col] = gk[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * 8 * L; e += kNormThreads) {
    const int which = e / (8 * L), col = e % (8 * L);
    if (col >= a.d) continue;
    float s = 0.f;
    for (int g = 0; g < G; ++g) s += red[(g * 2 + which) * 8 * L + col];
    a.partial[((int64_t)blockIdx.x * 2 + which) * a.d + col] = s;
  }
}

// dweight column e of q or k: the blocks' partial sums, 32 lanes taking every
// 32nd block each and a fixed tree over the lanes
__global__ void __launch_bounds__(256) qk_norm_bwd_sum_kernel(const float* __restrict__ partial,
                                                              int blocks, int d,
                                                              float* __restrict__ dq_weight,
                                                              float* __restrict__ dk_weight) {
  const int e = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x & 31;
  if (e >= 2 * d) return;
  float s = 0.f;
  for (int b = lane; b < blocks; b += 32) s += partial[(int64_t)b * 2 * d + e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane != 0) return;
  if (e < d) {
    if (dq_weight) dq_weight[e] = s;
  } else if (dk_weight) {
    dk_weight[e - d] = s;
  }
}

int lane_group(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }

constexpr int kFwdBlocks = 148 * 4, kBwdBlocks = 148 * 2;  // as many as are resident

// The split of a block's lane groups into HS heads x TS tokens, and the tokens
// per tile: up to U TS, no more than give every resident block one, nor (with a
// rotation) than the tables hold.  The split with the most rows in flight in a
// block is taken, the one with the most heads of several.  Measured, bf16, forward
// and gradients: 16,384 tokens x 2 heads x 32, 8 and 12 us (with one token a step
// as soon as TS is above a block's share, 22 and 55); 9000 x 9 x 128, 16 and 33 us
// (16 and 43; with the split that leaves the fewest lanes idle, 23 and 33).
void tile_shape(NormArgs& a, int rows, int blocks) {
  const int H = a.Hq + a.Hk, groups = kNormThreads / lane_group(a.d);
  int most = (int)(((int64_t)a.tokens + blocks - 1) / blocks);
  if (a.rot && most > kMaxTokens) most = kMaxTokens;
  int64_t best = 0;
  for (int hs = 1; hs <= groups && hs <= H; ++hs) {
    const int ts = groups / hs < most ? groups / hs : most;
    const int n = rows * ts < most ? rows * ts : most;
    // heads per step, times 2^20, by tokens
    const int64_t rows_in_flight = ((int64_t)H << 20) / ((H + hs - 1) / hs) * n;
    if (rows_in_flight >= best) {
      best = rows_in_flight;
      a.hs = hs;
      a.ts = ts;
      a.per_block = n;
    }
  }
}

size_t table_bytes(const NormArgs& a) { return 2 * sizeof(float) * (size_t)a.per_block * a.rot; }

template <typename Tin, int ROT>
cudaError_t dispatch_fwd_rot(const NormArgs& a, cudaStream_t st) {
  const int64_t tiles = ((int64_t)a.tokens + a.per_block - 1) / a.per_block;
  const unsigned grid = (unsigned)(tiles < kFwdBlocks ? tiles : kFwdBlocks);
  const size_t sm = table_bytes(a);
  switch (lane_group(a.d)) {
    case 4: qk_norm_fwd_kernel<Tin, 4, ROT><<<grid, kNormThreads, sm, st>>>(a); break;
    case 8: qk_norm_fwd_kernel<Tin, 8, ROT><<<grid, kNormThreads, sm, st>>>(a); break;
    case 16: qk_norm_fwd_kernel<Tin, 16, ROT><<<grid, kNormThreads, sm, st>>>(a); break;
    default: qk_norm_fwd_kernel<Tin, 32, ROT><<<grid, kNormThreads, sm, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <typename Tin, int ROT>
cudaError_t dispatch_bwd_rot(const NormArgs& a, cudaStream_t st) {
  const size_t red = a.partial ? sizeof(float) * kNormThreads * 16 : 0;
  const size_t sm = table_bytes(a) > red ? table_bytes(a) : red;
  switch (lane_group(a.d)) {
    case 4: qk_norm_bwd_kernel<Tin, 4, ROT><<<a.blocks, kNormThreads, sm, st>>>(a); break;
    case 8: qk_norm_bwd_kernel<Tin, 8, ROT><<<a.blocks, kNormThreads, sm, st>>>(a); break;
    case 16: qk_norm_bwd_kernel<Tin, 16, ROT><<<a.blocks, kNormThreads, sm, st>>>(a); break;
    default: qk_norm_bwd_kernel<Tin, 32, ROT><<<a.blocks, kNormThreads, sm, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <typename Tin>
cudaError_t dispatch_fwd(const NormArgs& a, cudaStream_t st) {
  if (a.rot == 0) return dispatch_fwd_rot<Tin, kNoRot>(a, st);
  return a.pairs ? dispatch_fwd_rot<Tin, kPairs>(a, st) : dispatch_fwd_rot<Tin, kHalves>(a, st);
}

template <typename Tin>
cudaError_t dispatch_bwd(const NormArgs& a, cudaStream_t st) {
  if (a.rot == 0) return dispatch_bwd_rot<Tin, kNoRot>(a, st);
  return a.pairs ? dispatch_bwd_rot<Tin, kPairs>(a, st) : dispatch_bwd_rot<Tin, kHalves>(a, st);
}

kda_status check_norm(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const int32_t* positions, const float* inv_freq, kda_dtype dt, int tokens,
                      int Hq, int Hk, int d, int rot_dim, kda_norm norm, kda_rotation rotation,
                      float eps) {
  if (!q || !k) return KDA_ERR_INVALID_ARG;
  if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (norm != KDA_NORM_RMS && norm != KDA_NORM_L2) return KDA_ERR_INVALID_ARG;
  if (rotation != KDA_ROT_HALVES && rotation != KDA_ROT_PAIRS) return KDA_ERR_INVALID_ARG;
  if (tokens <= 0 || Hq <= 0 || Hk <= 0 || d <= 0 || rot_dim < 0) return KDA_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !isfinite(eps)) return KDA_ERR_INVALID_ARG;
  if (rot_dim > d) return KDA_ERR_INVALID_ARG;
  if ((rot_dim > 0) != (positions != nullptr) || (rot_dim > 0) != (inv_freq != nullptr))
    return KDA_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > 256 || rot_dim % 16 != 0) return KDA_ERR_UNSUPPORTED;
  if (Hq > (1 << 16) || Hk > (1 << 16)) return KDA_ERR_UNSUPPORTED;
  const int64_t es = elem_bytes(dt);
  if (!stride_ok(q_stride, (int64_t)Hq * d, es) || !stride_ok(k_stride, (int64_t)Hk * d, es))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

NormArgs norm_args(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                   const float* q_weight, const float* k_weight, const int32_t* positions,
                   const float* inv_freq, int tokens, int Hq, int Hk, int d, int rot_dim,
                   kda_norm norm, kda_rotation rotation, float eps) {
  NormArgs a{};
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.tokens = tokens;
  a.Hq = Hq;
  a.Hk = Hk;
  a.d = d;
  a.rot = rot_dim;
  a.c = norm == KDA_NORM_RMS ? 1.0f / (float)d : 1.0f;
  a.eps = eps;
  a.pairs = rotation == KDA_ROT_PAIRS;
  return a;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_qk_norm_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const float* q_weight, const float* k_weight,
                           const int32_t* positions, const float* inv_freq, kda_dtype in_dtype,
                           int tokens, int Hq, int Hk, int d, int rot_dim, kda_norm norm,
                           kda_rotation rotation, float eps, void* q_out, void* k_out,
                           void* stream) {
  if (!q_out || !k_out) return KDA_ERR_INVALID_ARG;
  if (kda_status s = check_norm(q, q_stride, k, k_stride, positions, inv_freq, in_dtype, tokens,
                                Hq, Hk, d, rot_dim, norm, rotation, eps))
    return s;
  const int64_t es = elem_bytes(in_dtype), n = tokens;
  const int64_t wq = (int64_t)Hq * d, wk = (int64_t)Hk * d;
  // in place: a dense input that is its own output is read before it is written
  const bool q_in_place = q == q_out && q_stride == wq;
  const bool k_in_place = k == k_out && k_stride == wk;
  const Span qs = {q, row_bytes(n, q_stride, wq, es)}, ks = {k, row_bytes(n, k_stride, wk, es)};
  const Span qo = {q_out, n * wq * es}, ko = {k_out, n * wk * es};
  const Span ins[] = {{q_weight, (int64_t)d * 4},
                      {k_weight, (int64_t)d * 4},
                      {positions, n * 4},
                      {inv_freq, (int64_t)rot_dim * 2}};
  const Span outs[] = {qo, ko};
  if (kda_status s = check_spans(ins, outs)) return s;
  if (!span_aligned(qs) || !span_aligned(ks)) return KDA_ERR_MISALIGNED;
  if ((!q_in_place && spans_overlap(qo, qs)) || (!k_in_place && spans_overlap(ko, ks)) ||
      spans_overlap(qo, ks) || spans_overlap(ko, qs))
    return KDA_ERR_INVALID_ARG;
  NormArgs a = norm_args(q, q_stride, k, k_stride, q_weight, k_weight, positions, inv_freq,
                         tokens, Hq, Hk, d, rot_dim, norm, rotation, eps);
  a.q_out = q_out;
  a.k_out = k_out;
  tile_shape(a, in_dtype == KDA_BF16 ? kRows<__nv_bfloat16> : kRows<float>, kFwdBlocks);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = in_dtype == KDA_BF16 ? dispatch_fwd<__nv_bfloat16>(a, st)
                                             : dispatch_fwd<float>(a, st);
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

size_t kda_qk_norm_bwd_workspace_size(int tokens, int Hq, int Hk, int d) {
  if (tokens <= 0 || Hq <= 0 || Hk <= 0 || d <= 0 || d % 8 != 0 || d > 256 || Hq > (1 << 16) ||
      Hk > (1 << 16))
    return 0;
  return sizeof(float) * (size_t)(tokens < kBwdBlocks ? tokens : kBwdBlocks) * 2 * d;
}

kda_status kda_qk_norm_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const float* q_weight, const float* k_weight,
                           const int32_t* positions, const float* inv_freq, kda_dtype in_dtype,
                           int tokens, int Hq, int Hk, int d, int rot_dim, kda_norm norm,
                           kda_rotation rotation, float eps, const float* dq_out,
                           const float* dk_out, float* dq, float* dk, float* dq_weight,
                           float* dk_weight, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (!dq_out || !dk_out || !dq || !dk) return KDA_ERR_INVALID_ARG;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return KDA_ERR_INVALID_ARG;
  if (kda_status s = check_norm(q, q_stride, k, k_stride, positions, inv_freq, in_dtype, tokens,
                                Hq, Hk, d, rot_dim, norm, rotation, eps))
    return s;
  const bool sums = dq_weight || dk_weight;
  const size_t need = sums ? kda_qk_norm_bwd_workspace_size(tokens, Hq, Hk, d) : 0;
  if (sums && !workspace) return KDA_ERR_WORKSPACE;
  const int64_t es = elem_bytes(in_dtype), n = tokens;
  const int64_t wq = (int64_t)Hq * d, wk = (int64_t)Hk * d;
  const Span dqo = {dq_out, n * wq * 4}, dko = {dk_out, n * wk * 4};
  const Span dqs = {dq, n * wq * 4}, dks = {dk, n * wk * 4};
  const Span ins[] = {{q, row_bytes(n, q_stride, wq, es)},
                      {k, row_bytes(n, k_stride, wk, es)},
                      {q_weight, (int64_t)d * 4},
                      {k_weight, (int64_t)d * 4},
                      {positions, n * 4},
                      {inv_freq, (int64_t)rot_dim * 2}};
  const Span outs[] = {dqs, dks, {dq_weight, (int64_t)d * 4}, {dk_weight, (int64_t)d * 4},
                       {sums ? workspace : nullptr, (int64_t)need}};
  if (kda_status s = check_spans(ins, outs)) return s;
  if (!span_aligned(dqo) || !span_aligned(dko)) return KDA_ERR_MISALIGNED;
  for (int i = 0; i < 5; ++i) {
    // dq may overwrite dq_out and dk dk_out, exactly
    if (!(i == 0 && dq == dq_out) && spans_overlap(outs[i], dqo)) return KDA_ERR_INVALID_ARG;
    if (!(i == 1 && dk == dk_out) && spans_overlap(outs[i], dko)) return KDA_ERR_INVALID_ARG;
  }
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
  NormArgs a = norm_args(q, q_stride, k, k_stride, q_weight, k_weight, positions, inv_freq,
                         tokens, Hq, Hk, d, rot_dim, norm, rotation, eps);
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.dq = dq;
  a.dk = dk;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  tile_shape(a, kBwdRows, kBwdBlocks);
  const int64_t tiles = ((int64_t)tokens + a.per_block - 1) / a.per_block;
  a.blocks = (int)(tiles < kBwdBlocks ? tiles : kBwdBlocks);
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = in_dtype == KDA_BF16 ? dispatch_bwd<__nv_bfloat16>(a, st)
                                       : dispatch_bwd<float>(a, st);
  if (e == cudaSuccess && sums) {
    qk_norm_bwd_sum_kernel<<<(unsigned)((2 * d + 7) / 8), 256, 0, st>>>(
        a.partial, a.blocks, d, dq_weight, dk_weight);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

}  // extern "C"
