// kda_scan.cu -- the selective state space scan: prompts and single tokens.
//
//   h_t[d, s] = e^{dt A[d, s]} h_{t-1}[d, s] + dt x[t, d] B[t, s]
//   y[t, d]   = sum_s C[t, s] h_t[d, s] + D[d] x[t, d],   out = y z sigmoid(z)
#include <math.h>

#include "kda_scan.cuh"

namespace kda {
namespace scan {
namespace {

constexpr int kTile = 32;            // tokens per tile
constexpr int kPitch = kTile + 4;    // of a channel's row of a tile, in floats

// position of token t in channel c's row of a tile: blocks of 4 or 8 tokens
// change places by channel, so that the transposing stores (neighbouring lanes
// hold neighbouring channel groups) spread over the banks
template <int VEC>
__device__ __forceinline__ int place(int c, int t) {
  return VEC == 8 ? t ^ (((c >> 3) & 3) << 3) : t ^ (((c >> 2) & 7) << 2);
}

// kOut: the outputs and the final state.  kEnd: only the state that the segment
// leaves from a zero state, and its sum of dt (for all but a sequence's last
// segment).  kEnds: those, and the state gradient that the segment's outputs
// send to its start, sum_t (prod_{s <= t} e^{dt_s A}) C_t dy_t.
enum Mode { kOut, kEnd, kEnds };

template <typename Tin, int S, int MODE>
__global__ void __launch_bounds__(Layout<S>::NT) scan_fwd_kernel(const Args a) {
  using L = Layout<S>;
  constexpr int LN = L::LN, NT = L::NT, CT = L::CT;
  constexpr int PER = kTile * CT / NT;             // elements of a tile per thread
  constexpr int VEC = PER > 8 ? 8 : PER;           // of them consecutive channels
  constexpr int ITEMS = PER / VEC, CV = CT / VEC;
  constexpr int BPT = kTile * S / NT >= 4 ? 4 : kTile * S / NT;  // B, C elements per load
  __shared__ __align__(16) float sdt[CT * kPitch], su[CT * kPitch];
  __shared__ __align__(16) float sB[kTile * S], sC[MODE == kEnd ? 4 : kTile * S];
  __shared__ __align__(16) float sdy[MODE == kEnds ? CT * kPitch : 4];

  if (a.seg.cu) {
    if (!a.sb->seqlens_ok) return;
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.sb->status = KDA_OK;
    a.sb->detail = 0;
  }
  const int unit = blockIdx.x / a.nblk, cb = blockIdx.x % a.nblk;
  const Unit un = resolve(a.seg, unit);
  if (!un.valid || (MODE != kOut && un.last && (MODE == kEnd || un.first))) return;
  const int tid = threadIdx.x, nl = tid % LN, c = tid / LN;
  const int d0 = cb * CT, d = d0 + c;
  const bool live = d < a.D;
  const int g = d0 / (a.D / a.G);

  float A2[4], h[4], prod[4], gs[4];
  const int64_t so = (int64_t)d * S + nl * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    A2[i] = h[i] = gs[i] = 0.f;
    prod[i] = 1.f;
  }
  if (live) {
    load_vec<float, 4>(a.A + so, A2);
    if (MODE == kOut) {
      if (a.h_seg)
        load_vec<float, 4>(a.h_seg + (int64_t)unit * a.D * S + so, h);
      else if (a.init)
        load_vec<float, 4>(a.init + (int64_t)un.n * a.D * S + so, h);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;

  const int icv = tid % CV, it = tid / CV;  // the thread's channel group, first token
  const int ic = icv * VEC;
  const bool ilive = d0 + ic < a.D;  // D is a multiple of 8
  float bias[VEC], skip[VEC], dsum[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) bias[j] = skip[j] = dsum[j] = 0.f;
  if (ilive && a.delta_bias) load_vec<float, VEC>(a.delta_bias + d0 + ic, bias);
  if (ilive && a.D_skip) load_vec<float, VEC>(a.D_skip + d0 + ic, skip);

  for (int64_t t0 = un.t0; t0 < un.t1; t0 += kTile) {
    float x[ITEMS][VEC];
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int t = it + m * (NT / CV);
      float dt[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[m][j] = dt[j] = 0.f;
      if (ilive && t0 + t < un.t1) {
        load_vec<Tin, VEC>(static_cast<const Tin*>(a.x) + (t0 + t) * a.x_stride + d0 + ic, x[m]);
        load_vec<Tin, VEC>(static_cast<const Tin*>(a.delta) + (t0 + t) * a.delta_stride + d0 + ic,
                           dt);
#pragma unroll
        for (int j = 0; j < VEC; ++j) dt[j] = step_size(dt[j] + bias[j], a.softplus);
      }
      if (MODE == kEnds) {
        float dy[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) dy[j] = 0.f;
        if (ilive && t0 + t < un.t1) {
          load_vec<Tin, VEC>(static_cast<const Tin*>(a.dout) + (t0 + t) * a.D + d0 + ic, dy);
          if (a.z) {
            float zz[VEC];
            load_vec<Tin, VEC>(static_cast<const Tin*>(a.z) + (t0 + t) * a.z_stride + d0 + ic, zz);
#pragma unroll
            for (int j = 0; j < VEC; ++j) dy[j] *= zz[j] * sigmoid_fast(zz[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) sdy[(ic + j) * kPitch + place<VEC>(ic + j, t)] = dy[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int p = (ic + j) * kPitch + place<VEC>(ic + j, t);
        sdt[p] = dt[j];
        su[p] = dt[j] * x[m][j];
        dsum[j] += dt[j];
      }
    }
    for (int e = tid * BPT; e < kTile * S; e += NT * BPT) {
      const int t = e / S, s = e % S;
      float b[BPT], cc[BPT];
#pragma unroll
      for (int j = 0; j < BPT; ++j) b[j] = cc[j] = 0.f;
      if (t0 + t < un.t1) {
        load_vec<Tin, BPT>(static_cast<const Tin*>(a.Bm) + (t0 + t) * a.B_stride + g * S + s, b);
        if (MODE != kEnd)
          load_vec<Tin, BPT>(static_cast<const Tin*>(a.Cm) + (t0 + t) * a.C_stride + g * S + s,
                             cc);
      }
      store_vec<BPT>(sB + e, b);
      if (MODE != kEnd) store_vec<BPT>(sC + e, cc);
    }
    __syncthreads();
#pragma unroll 2
    for (int t4 = 0; t4 < kTile; t4 += 4) {
      const int p = c * kPitch + place<VEC>(c, t4);
      const float4 dt4 = *reinterpret_cast<const float4*>(sdt + p);
      const float4 u4 = *reinterpret_cast<const float4*>(su + p);
      const float dts[4] = {dt4.x, dt4.y, dt4.z, dt4.w}, us[4] = {u4.x, u4.y, u4.z, u4.w};
      float4 dy4 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (MODE == kEnds) dy4 = *reinterpret_cast<const float4*>(sdy + p);
      const float dys[4] = {dy4.x, dy4.y, dy4.z, dy4.w};
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 b4 = *reinterpret_cast<const float4*>(sB + (t4 + k) * S + nl * 4);
        const float bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = ex2(dts[k] * A2[i]);
          h[i] = fmaf(w, h[i], us[k] * bs[i]);
          if (MODE == kEnds) prod[i] *= w;
        }
        if (MODE == kEnds) {
          const float4 c4 = *reinterpret_cast<const float4*>(sC + (t4 + k) * S + nl * 4);
          const float cs[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) gs[i] = fmaf(prod[i] * cs[i], dys[k], gs[i]);
        }
        if (MODE == kOut) {
          const float4 c4 = *reinterpret_cast<const float4*>(sC + (t4 + k) * S + nl * 4);
          y[k] = fmaf(c4.x, h[0], c4.y * h[1]) + fmaf(c4.z, h[2], c4.w * h[3]);
        }
      }
      if (MODE == kOut) {
        // the channel's lanes have read their u: y takes its place
        const float2 r = sum_lanes<LN>(y, nl);
        if (LN == 2)
          *reinterpret_cast<float2*>(su + p + 2 * nl) = r;
        else if (nl < 4)
          su[p + nl] = r.x;
      }
    }
    __syncthreads();
    if (MODE == kOut) {
#pragma unroll
      for (int m = 0; m < ITEMS; ++m) {
        const int t = it + m * (NT / CV);
        if (ilive && t0 + t < un.t1) {
          float y[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            y[j] = fmaf(skip[j], x[m][j], su[(ic + j) * kPitch + place<VEC>(ic + j, t)]);
          if (a.z) {
            float zz[VEC];
            load_vec<Tin, VEC>(static_cast<const Tin*>(a.z) + (t0 + t) * a.z_stride + d0 + ic, zz);
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[j] *= zz[j] * sigmoid_fast(zz[j]);
          }
          store_vec<VEC>(static_cast<Tin*>(a.out) + (t0 + t) * a.D + d0 + ic, y);
        }
      }
      __syncthreads();  // su is written again
    }
  }
  if (MODE != kOut) {
    if (live) store_vec<4>(a.h_seg + (int64_t)unit * a.D * S + so, h);
    if (MODE == kEnds && live) store_vec<4>(a.g_seg + (int64_t)unit * a.D * S + so, gs);
    // dt summed over the threads that share a channel group, in order
    float* red = su;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[it * CT + ic + j] = dsum[j];
    __syncthreads();
    if (tid < CT && d0 + tid < a.D) {
      float s = 0.f;
      for (int r = 0; r < NT / CV; ++r) s += red[r * CT + tid];
      a.dt_sum[(int64_t)unit * a.D + d0 + tid] = s;
    }
  } else if (un.last && a.final_state && live) {
    store_vec<4>(a.final_state + (int64_t)un.n * a.D * S + so, h);
  }
}

// Incoming state of every segment of a sequence, in place over the states the
// segments leave from zero: h_in[0] = init, h_in[k+1] = e^{A sum dt_k} h_in[k] + h_k;
// with g_seg the state gradients from the right likewise: g_in[last] = d_final,
// g_in[k-1] = e^{A sum dt_k} g_in[k] + g_k.
__global__ void __launch_bounds__(256) scan_combine_kernel(const Args a) {
  if (a.seg.cu && !a.sb->seqlens_ok) return;
  const int64_t per = (int64_t)a.D * a.S / 4;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int n = (int)(idx / per);
  if (n >= a.seg.num_seqs) return;
  const int64_t e = (idx % per) * 4;
  const int d = (int)(e / a.S);
  const int u0 = a.seg.cu ? __ldg(a.seg.seg_off + n) : n * a.seg.segs;
  const int u1 = a.seg.cu ? __ldg(a.seg.seg_off + n + 1) : u0 + a.seg.segs;
  const int64_t ds = (int64_t)a.D * a.S;
  float A[4], in[4] = {};
  load_vec<float, 4>(a.A + e, A);
  if (a.init) load_vec<float, 4>(a.init + n * ds + e, in);
  for (int u = u0; u < u1; ++u) {
    float* at = a.h_seg + u * ds + e;
    float own[4] = {}, w = 0.f;
    if (u + 1 < u1) {
      load_vec<float, 4>(at, own);
      w = a.dt_sum[(int64_t)u * a.D + d];
    }
    store_vec<4>(at, in);
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i] = fmaf(ex2(w * (A[i] * kLog2e)), in[i], own[i]);
  }
  if (!a.g_seg) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) in[i] = 0.f;
  if (a.d_final) load_vec<float, 4>(a.d_final + n * ds + e, in);
  for (int u = u1 - 1; u >= u0; --u) {
    float* at = a.g_seg + u * ds + e;
    float own[4] = {}, w = 0.f;
    if (u > u0) {
      load_vec<float, 4>(at, own);
      w = a.dt_sum[(int64_t)u * a.D + d];
    }
    store_vec<4>(at, in);
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i] = fmaf(ex2(w * (A[i] * kLog2e)), in[i], own[i]);
  }
}

// One token: a thread has 4 states of a channel of a sequence.  HBM-bound: the
// fp32 states are read once and written once.
template <typename Tin, int S>
__global__ void __launch_bounds__(256) scan_step_kernel(const Args a, float* state, int N) {
  constexpr int LN = S / 4;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int nl = (int)(idx % LN);
  const int64_t cn = idx / LN;
  const int64_t n = cn / a.D;
  const bool live = n < N;  // LN divides 32: a channel's lanes share this
  const int d = (int)(cn % a.D);
  float y = 0.f, x = 0.f;
  if (live) {
    const int g = d / (a.D / a.G);
    float h[4], A[4], b[4], c[4];
    float* st = state + (n * a.D + d) * S + nl * 4;
    load_vec<float, 4>(st, h);
    load_vec<float, 4>(a.A + (int64_t)d * S + nl * 4, A);
    load_vec<Tin, 4>(static_cast<const Tin*>(a.Bm) + n * a.B_stride + g * S + nl * 4, b);
    load_vec<Tin, 4>(static_cast<const Tin*>(a.Cm) + n * a.C_stride + g * S + nl * 4, c);
    x = Elem<Tin>::load(static_cast<const Tin*>(a.x) + n * a.x_stride + d);
    float dt = Elem<Tin>::load(static_cast<const Tin*>(a.delta) + n * a.delta_stride + d);
    if (a.delta_bias) dt += a.delta_bias[d];
    dt = step_size(dt, a.softplus);
    const float u = dt * x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(ex2(dt * (A[i] * kLog2e)), h[i], u * b[i]);
      y = fmaf(c[i], h[i], y);
    }
    store_vec<4>(st, h);
  }
#pragma unroll
  for (int o = LN / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  if (live && nl == 0) {
    if (a.D_skip) y = fmaf(a.D_skip[d], x, y);
    if (a.z) {
      const float zz = Elem<Tin>::load(static_cast<const Tin*>(a.z) + n * a.z_stride + d);
      y *= zz * sigmoid_fast(zz);
    }
    Elem<Tin>::store(static_cast<Tin*>(a.out) + n * a.D + d, y);
  }
}

template <typename Tin, int MODE>
cudaError_t launch_mode(const Args& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.seg.units * a.nblk);
  switch (a.S) {
    case 8: scan_fwd_kernel<Tin, 8, MODE><<<grid, Layout<8>::NT, 0, st>>>(a); break;
    case 16: scan_fwd_kernel<Tin, 16, MODE><<<grid, Layout<16>::NT, 0, st>>>(a); break;
    case 32: scan_fwd_kernel<Tin, 32, MODE><<<grid, Layout<32>::NT, 0, st>>>(a); break;
    case 64: scan_fwd_kernel<Tin, 64, MODE><<<grid, Layout<64>::NT, 0, st>>>(a); break;
    default: scan_fwd_kernel<Tin, 128, MODE><<<grid, Layout<128>::NT, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_typed(const Args& a, kda_dtype dt, cudaStream_t st) {
  return dt == KDA_BF16 ? launch_mode<__nv_bfloat16, MODE>(a, st)
                        : launch_mode<float, MODE>(a, st);
}

template <typename Tin>
cudaError_t launch_step(const Args& a, float* state, int N, cudaStream_t st) {
  const int64_t items = (int64_t)N * a.D * a.S / 4;
  const unsigned grid = (unsigned)((items + 255) / 256);
  switch (a.S) {
    case 8: scan_step_kernel<Tin, 8><<<grid, 256, 0, st>>>(a, state, N); break;
    case 16: scan_step_kernel<Tin, 16><<<grid, 256, 0, st>>>(a, state, N); break;
    case 32: scan_step_kernel<Tin, 32><<<grid, 256, 0, st>>>(a, state, N); break;
    case 64: scan_step_kernel<Tin, 64><<<grid, 256, 0, st>>>(a, state, N); break;
    default: scan_step_kernel<Tin, 128><<<grid, 256, 0, st>>>(a, state, N); break;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ends(const Args& a, kda_dtype dt, cudaStream_t st) {
  if (cudaError_t e = a.g_seg ? launch_typed<kEnds>(a, dt, st) : launch_typed<kEnd>(a, dt, st))
    return e;
  const int64_t items = (int64_t)a.seg.num_seqs * a.D * a.S / 4;
  scan_combine_kernel<<<(unsigned)((items + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

bool sizes_ok(int D, int S, int G) {
  if (S != 8 && S != 16 && S != 32 && S != 64 && S != 128) return false;
  if (D % 8 != 0 || D > (1 << 24) || D % G != 0) return false;
  return G == 1 || D / G % 32 == 0;
}

// Tokens per segment.  A segment costs a second pass over its tokens, so a
// sequence is cut only where the channel blocks of the sequences do not fill
// the GPU.
int segment_len(int B, int T, int D, int S, bool packed) {
  const int64_t blocks = (D + chan_tile(S) - 1) / chan_tile(S);
  const int64_t slots = 148 * 4;
  int64_t len;
  if (packed) {
    len = (int64_t)T * blocks / (slots * 2);
  } else {
    if (B * blocks >= slots / 2) return T;
    const int64_t cuts = (slots + B * blocks - 1) / (B * blocks);
    len = (T + cuts - 1) / cuts;
  }
  if (len < 256) len = 256;
  len = (len + 31) / 32 * 32;
  return (int)(len < T ? len : T);
}

Segments plan_segments(const int32_t* cu, int num_seqs, int B, int T, int D, int S) {
  Segments m{};
  m.cu = cu;
  m.num_seqs = cu ? num_seqs : B;
  m.T = T;
  m.seg_len = segment_len(B, T, D, S, cu != nullptr);
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
  a.nblk = (D + chan_tile(S) - 1) / chan_tile(S);
  return a;
}

}  // namespace scan
}  // namespace kda

using namespace kda;
using namespace kda::scan;

extern "C" {

size_t kda_selective_scan_fwd_workspace_size(int B, int T, int D, int S, int G, int num_seqs) {
  if (B <= 0 || T <= 0 || D <= 0 || G <= 0 || num_seqs < 0 || !sizes_ok(D, S, G) ||
      (int64_t)B * T > kMaxRows)
    return 0;
  static const int32_t packed = 0;  // only whether there are offsets matters here
  const Segments m = plan_segments(num_seqs > 0 && B == 1 ? &packed : nullptr, num_seqs, B, T, D, S);
  size_t b = kStatusBytes;
  if (m.cu) b += align256(sizeof(int32_t) * ((size_t)num_seqs + 1));
  if (m.segs > 1)
    b += align256(sizeof(float) * (size_t)m.units * D * S) +
         align256(sizeof(float) * (size_t)m.units * D);
  return b;
}

}  // extern "C"

extern "C" {

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
  a.seg = plan_segments(cu_seqlens, num_seqs, B, T, D, S);
  if ((int64_t)a.seg.units * a.nblk > 0x7fffffffLL || N * D / 256 * (S / 4) > 0x7ffffff0LL)
    return KDA_ERR_UNSUPPORTED;
  a.init = init_state;
  a.final_state = final_state;
  a.out = out;
  a.sb = static_cast<StatusBlock*>(workspace);
  char* tail = static_cast<char*>(workspace) + kStatusBytes;
  cudaStream_t st = (cudaStream_t)stream;
  if (cu_seqlens) {
    int32_t* off = reinterpret_cast<int32_t*>(tail);
    tail += align256(sizeof(int32_t) * ((size_t)num_seqs + 1));
    a.seg.seg_off = off;
    if (cudaError_t e = launch_seqlens_plan(cu_seqlens, num_seqs, T, a.sb, a.seg.seg_len, off, st))
      return cuda_failure(e);
  }
  if (a.seg.segs > 1) {
    a.h_seg = reinterpret_cast<float*>(tail);
    tail += align256(sizeof(float) * (size_t)a.seg.units * D * S);
    a.dt_sum = reinterpret_cast<float*>(tail);
  }
  if (a.h_seg)
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
