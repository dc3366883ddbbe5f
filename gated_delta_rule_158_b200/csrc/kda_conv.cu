// kda_conv.cu -- the short causal convolution: prompt, single token, gradients.
//
//   p[t, d] = bias[d] + sum_j w[d, j] x[t - (W-1) + j, d],  out = p or p sigmoid(p)
//
// W multiply-adds per element: HBM-bound (x read once, out written once).  A
// thread owns one 16-byte group of channels and a strip of consecutive
// tokens, and slides the window over the strip in registers, so a row is
// loaded once per strip plus W - 1 rows at its head (which the strip before
// has just read: L2 hits).  The batch is one flat axis of B * T tokens; a
// strip that crosses a sequence boundary starts a new run there.
#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int kConvThreads = 256;
constexpr int kUnroll = 8;  // rows in flight per thread

// ------------------------------------------------------------ packed batch
__global__ void seqlens_plan_kernel(const int32_t* __restrict__ cu, int N, int T,
                                    StatusBlock* sb, int seg_len,
                                    int32_t* __restrict__ seg_off) {
  __shared__ int bad, carry;
  __shared__ int wsum[32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) {
    bad = (cu[0] != 0 || cu[N] != T) ? 1 : 0;
    carry = 0;
  }
  __syncthreads();
  for (int n = tid; n < N; n += blockDim.x)
    if (cu[n + 1] < cu[n]) atomicOr(&bad, 1);
  __syncthreads();
  if (tid == 0) {
    sb->status = bad ? KDA_ERR_BAD_SEQLENS : KDA_OK;
    sb->detail = 0;
    sb->never_set = 0;
    sb->seqlens_ok = bad ? 0 : 1;
  }
  if (bad || seg_off == nullptr) return;
  // exclusive prefix sums of the segment counts, blockDim.x sequences a step
  for (int n0 = 0; n0 < N; n0 += blockDim.x) {
    const int n = n0 + tid;
    int c = 0;
    if (n < N) {
      const int len = cu[n + 1] - cu[n];
      c = len > 0 ? 1 + (len - 1) / seg_len : 1;
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

struct ConvArgs {
  const void* x;
  int64_t x_stride;
  const float* weight;
  const float* bias;
  const void* init;
  const int32_t* cu;
  int num_seqs;  // N (packed), or B
  int64_t total; // B * T
  int T, D;
  bool silu;
  void* out;
  void* final_state;
  // gradients
  const float* dout;
  const float* d_final;
  float* dx;
  float* d_init;
  float* partial;
  int strip, strips;
  StatusBlock* sb;
};

// the run of tokens [t, end) of one sequence n that starts at `start`
struct Run {
  int n;
  int64_t start, end;
};

__device__ __forceinline__ Run run_at(const ConvArgs& a, int64_t t) {
  Run r;
  if (a.cu) {
    r.n = find_range(a.cu, a.num_seqs, (int)t);
    r.start = __ldg(a.cu + r.n);
    r.end = __ldg(a.cu + r.n + 1);
  } else {
    r.n = (int)(t / a.T);
    r.start = (int64_t)r.n * a.T;
    r.end = r.start + a.T;
  }
  return r;
}

// the row `back` places before the run's start (1 = the newest kept row)
template <typename Tin, int W, int V>
__device__ __forceinline__ void kept_row(const ConvArgs& a, int n, int back, int c,
                                         float (&v)[V]) {
  if (a.init) {
    load_vec<Tin, V>(static_cast<const Tin*>(a.init) +
                         ((int64_t)n * (W - 1) + (W - 1 - back)) * a.D + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.f;
  }
}

// win = the W - 1 rows before token t of run r, oldest first
template <typename Tin, int W, int V>
__device__ __forceinline__ void fill_window(const ConvArgs& a, const Run& r, int64_t t, int c,
                                            float (&win)[W - 1][V]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t s = t - (W - 1) + j;
    if (s >= r.start)
      load_vec<Tin, V>(static_cast<const Tin*>(a.x) + s * a.x_stride + c, win[j]);
    else
      kept_row<Tin, W, V>(a, r.n, (int)(r.start - s), c, win[j]);
  }
}

template <int W, int V>
__device__ __forceinline__ void push_row(float (&win)[W - 1][V], const float (&row)[V]) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
#pragma unroll
  for (int i = 0; i < V; ++i) win[W - 2][i] = row[i];
}

template <int W, int V>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int c, float (&w)[V][W],
                                          float (&b)[V]) {
  // V * W consecutive floats from a 16-byte boundary (c is a multiple of 4)
  float flat[V * W];
#pragma unroll
  for (int i = 0; i < V * W; i += 4) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(a.weight + (int64_t)c * W + i));
    flat[i] = f.x; flat[i + 1] = f.y; flat[i + 2] = f.z; flat[i + 3] = f.w;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) w[i][j] = flat[i * W + j];
  if (a.bias) {
    load_vec<float, V>(a.bias + c, b);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.f;
  }
}

template <int W, int V>
__device__ __forceinline__ void taps_dot(const float (&w)[V][W], const float (&b)[V],
                                         const float (&win)[W - 1][V], const float (&row)[V],
                                         float (&p)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float s = b[i];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s = fmaf(w[i][j], win[j][i], s);
    p[i] = fmaf(w[i][W - 1], row[i], s);
  }
}

// rows of the final state: row j of sequence n is place len - (W-1) + j
template <typename Tin, int W, int V>
__device__ __forceinline__ void store_final(const ConvArgs& a, int64_t item) {
  const int CG = a.D / V;
  const int c = (int)(item % CG) * V;
  const int64_t r = item / CG;
  const int n = (int)(r / (W - 1)), j = (int)(r % (W - 1));
  if (n >= a.num_seqs) return;
  int64_t start, len;
  if (a.cu) {
    start = __ldg(a.cu + n);
    len = __ldg(a.cu + n + 1) - start;
  } else {
    start = (int64_t)n * a.T;
    len = a.T;
  }
  const int64_t s = len - (W - 1) + j;
  float v[V];
  if (s >= 0)
    load_vec<Tin, V>(static_cast<const Tin*>(a.x) + (start + s) * a.x_stride + c, v);
  else
    kept_row<Tin, W, V>(a, n, (int)-s, c, v);
  store_vec<V>(static_cast<Tin*>(a.final_state) + r * a.D + c, v);  // exact: the type is the same
}

// Threads [0, strips * D / V) take a strip each, channel groups fastest; the
// blocks behind them write the final state.
template <typename Tin, int W>
__global__ void __launch_bounds__(kConvThreads) conv_fwd_kernel(const ConvArgs a,
                                                                unsigned strip_blocks) {
  constexpr int V = 16 / sizeof(Tin);
  if (a.cu) {
    if (!a.sb->seqlens_ok) return;
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.sb->status = KDA_OK;
    a.sb->detail = 0;
  }
  if (blockIdx.x >= strip_blocks) {
    store_final<Tin, W, V>(a, (int64_t)(blockIdx.x - strip_blocks) * kConvThreads + threadIdx.x);
    return;
  }
  const int CG = a.D / V;
  const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  const int64_t strip = idx / CG;
  if (strip >= a.strips) return;
  const int c = (int)(idx % CG) * V;
  const int64_t t0 = strip * a.strip;
  const int64_t t1 = min(t0 + a.strip, a.total);
  const Tin* x = static_cast<const Tin*>(a.x);
  Tin* out = static_cast<Tin*>(a.out);

  float w[V][W], b[V], win[W - 1][V];
  load_taps<W, V>(a, c, w, b);
  Run r = run_at(a, t0);
  fill_window<Tin, W, V>(a, r, t0, c, win);
  for (int64_t t = t0; t < t1; t += kUnroll) {
    float row[kUnroll][V];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (t + u < t1) load_vec<Tin, V>(x + (t + u) * a.x_stride + c, row[u]);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (t + u < t1) {
        if (t + u >= r.end) {  // the next sequence that has tokens
          r = run_at(a, t + u);
          fill_window<Tin, W, V>(a, r, t + u, c, win);
        }
        float p[V];
        taps_dot<W, V>(w, b, win, row[u], p);
        if (a.silu) {
#pragma unroll
          for (int i = 0; i < V; ++i) p[i] *= sigmoid_fast(p[i]);
        }
        store_vec<V>(out + (t + u) * a.D + c, p);
        push_row<W, V>(win, row[u]);
      }
    }
  }
}

// One token of one sequence per thread and channel group; the state's rows
// move one place up.
template <typename Tin, int W>
__global__ void __launch_bounds__(kConvThreads)
    conv_step_kernel(const Tin* __restrict__ x, int64_t x_stride,
                     const float* __restrict__ weight, const float* __restrict__ bias,
                     Tin* __restrict__ state, int N, int D, bool silu, Tin* __restrict__ out) {
  constexpr int V = 16 / sizeof(Tin);
  const int CG = D / V;
  const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  const int64_t n = idx / CG;
  if (n >= N) return;
  const int c = (int)(idx % CG) * V;
  ConvArgs a{};
  a.weight = weight;
  a.bias = bias;
  float win[W - 1][V], row[V], w[V][W], b[V], p[V];
  Tin* st = state + n * (W - 1) * D + c;
  load_vec<Tin, V>(x + n * x_stride + c, row);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_vec<Tin, V>(st + (int64_t)j * D, win[j]);
  load_taps<W, V>(a, c, w, b);
  taps_dot<W, V>(w, b, win, row, p);
  if (silu) {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= sigmoid_fast(p[i]);
  }
  store_vec<V>(out + n * D + c, p);
  push_row<W, V>(win, row);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_vec<V>(st + (int64_t)j * D, win[j]);
}

// --------------------------------------------------------------- gradients
// A strip [t0, t1) is walked forward, run by run.  Token t gives ds[t]; the
// gradient of row s is complete once ds[s .. s + W - 1] are known, so the walk
// goes W - 1 tokens past the run (into the next strip's tokens, whose ds it
// forms again, or past the sequence's end, where ds is 0), and a window of
// the last W - 1 values of ds stays in registers.  dweight and dbias are
// summed in registers over the strip's own tokens and leave as one partial
// row per strip, added in strip order by conv_bwd_sum_kernel.
constexpr int kBV = 4;  // channels per thread: fp32 16-byte accesses

template <typename Tin, int W>
__global__ void __launch_bounds__(kConvThreads) conv_bwd_kernel(const ConvArgs a,
                                                                unsigned strip_blocks) {
  constexpr int V = kBV;
  if (a.cu) {
    if (!a.sb->seqlens_ok) return;
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.sb->status = KDA_OK;
    a.sb->detail = 0;
  }
  const int CG = a.D / V;
  if (blockIdx.x >= strip_blocks) {
    // d_init of sequences without a token: their kept rows are the final ones
    const int64_t item = (int64_t)(blockIdx.x - strip_blocks) * kConvThreads + threadIdx.x;
    const int64_t row = item / CG;
    const int64_t n = row / (W - 1);
    if (n >= a.num_seqs || __ldg(a.cu + n + 1) != __ldg(a.cu + n)) return;
    const int c = (int)(item % CG) * V;
    float v[V] = {};
    if (a.d_final) load_vec<float, V>(a.d_final + row * a.D + c, v);
    store_vec<V>(a.d_init + row * a.D + c, v);
    return;
  }
  const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  const int64_t strip = idx / CG;
  if (strip >= a.strips) return;
  const int c = (int)(idx % CG) * V;
  const int64_t t0 = strip * a.strip;
  const int64_t t1 = min(t0 + a.strip, a.total);
  const Tin* x = static_cast<const Tin*>(a.x);

  float w[V][W], b[V], win[W - 1][V], dsw[W - 1][V], dw[V][W], db[V];
  load_taps<W, V>(a, c, w, b);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[i][j] = 0.f;
  }
  for (int64_t ta = t0; ta < t1;) {
    const Run r = run_at(a, ta);
    const int64_t tb = min(t1, r.end);
    fill_window<Tin, W, V>(a, r, ta, c, win);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) dsw[j][i] = 0.f;
    const bool head = ta == r.start;
    constexpr int U = 4;  // tokens whose rows are in flight
    for (int64_t tt = ta; tt < tb + W - 1; tt += U) {
      float rows[U][V], dos[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = tt + u;
#pragma unroll
        for (int i = 0; i < V; ++i) rows[u][i] = dos[u][i] = 0.f;
        if (t < tb + W - 1 && t < r.end) {
          load_vec<Tin, V>(x + t * a.x_stride + c, rows[u]);
          load_vec<float, V>(a.dout + t * a.D + c, dos[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = tt + u;
        if (t >= tb + W - 1) continue;
        float ds[V];
#pragma unroll
        for (int i = 0; i < V; ++i) ds[i] = 0.f;
        if (t < r.end) {
          if (a.silu) {
            float p[V];
            taps_dot<W, V>(w, b, win, rows[u], p);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float sg = sigmoid_fast(p[i]);
              ds[i] = dos[u][i] * (sg * fmaf(p[i], 1.f - sg, 1.f));
            }
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) ds[i] = dos[u][i];
          }
          if (t < tb) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              db[i] += ds[i];
#pragma unroll
              for (int j = 0; j < W - 1; ++j) dw[i][j] = fmaf(ds[i], win[j][i], dw[i][j]);
              dw[i][W - 1] = fmaf(ds[i], rows[u][i], dw[i][W - 1]);
            }
          }
          push_row<W, V>(win, rows[u]);
        }
        const int64_t s = t - (W - 1);  // its gradient is complete
        if (s >= ta || (head && a.d_init)) {
          float g[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            g[i] = w[i][0] * ds[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) g[i] = fmaf(w[i][W - 1 - j], dsw[j][i], g[i]);
          }
          const int64_t f = s - (r.end - (W - 1));  // its row of the final state
          if (f >= 0 && a.d_final) {
            float d[V];
            load_vec<float, V>(a.d_final + ((int64_t)r.n * (W - 1) + f) * a.D + c, d);
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] += d[i];
          }
          float* to = s >= ta ? a.dx + s * a.D
                              : a.d_init + ((int64_t)r.n * (W - 1) + (s - ta + W - 1)) * a.D;
          store_vec<V>(to + c, g);
        }
        push_row<W, V>(dsw, ds);
      }
    }
    ta = tb;
  }
  // [strip][W + 1][D]: tap j of all channels, then the bias
  float* part = a.partial + strip * (W + 1) * a.D + c;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = dw[i][j];
    store_vec<V>(part + (int64_t)j * a.D, v);
  }
  store_vec<V>(part + (int64_t)W * a.D, db);
}

// Element e = (j, d) of the partial rows, added over the strips: eight threads
// take every eighth strip each, then their sums in order.
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(const float* __restrict__ partial,
                                                           const int strips, const int D,
                                                           const int W,
                                                           float* __restrict__ dweight,
                                                           float* __restrict__ dbias,
                                                           const int32_t* cu,
                                                           const StatusBlock* sb) {
  if (cu && !sb->seqlens_ok) return;
  __shared__ float red[8][32];
  const int64_t n = (int64_t)(W + 1) * D;
  const int64_t e = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (e < n)
    for (int p = threadIdx.y; p < strips; p += 8) s += partial[p * n + e];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || e >= n) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s += red[k][threadIdx.x];
  const int j = (int)(e / D), d = (int)(e % D);
  if (j < W) dweight[(int64_t)d * W + j] = s;
  else if (dbias) dbias[d] = s;
}

// Tokens per strip: long strips read fewer head rows again and leave fewer
// partial sums; strips are shortened (to `lo` at least) until the GPU has
// `want` threads.
int strip_len(int64_t total, int groups, int lo, int hi, int64_t want) {
  int64_t s = total * groups / want;
  s = s / 8 * 8;
  if (s < lo) s = lo;
  if (s > hi) s = hi;
  return (int)s;
}

constexpr int64_t kWantThreads = 148LL * 1024;

int bwd_strip(int64_t total, int D) {
  return strip_len(total, D / kBV, 16, 1 << 20, kWantThreads);
}

template <typename Tin>
cudaError_t dispatch_fwd(const ConvArgs& a, int W, cudaStream_t st) {
  constexpr int V = 16 / sizeof(Tin);
  const int64_t blocks = ((int64_t)a.strips * (a.D / V) + kConvThreads - 1) / kConvThreads;
  int64_t fin = 0;
  if (a.final_state)
    fin = ((int64_t)a.num_seqs * (W - 1) * (a.D / V) + kConvThreads - 1) / kConvThreads;
  const unsigned grid = (unsigned)(blocks + fin);
  switch (W) {
    case 2: conv_fwd_kernel<Tin, 2><<<grid, kConvThreads, 0, st>>>(a, (unsigned)blocks); break;
    case 3: conv_fwd_kernel<Tin, 3><<<grid, kConvThreads, 0, st>>>(a, (unsigned)blocks); break;
    default: conv_fwd_kernel<Tin, 4><<<grid, kConvThreads, 0, st>>>(a, (unsigned)blocks); break;
  }
  return cudaGetLastError();
}

template <typename Tin>
cudaError_t dispatch_step(const void* x, int64_t xs, const float* w, const float* b, void* state,
                          int N, int D, int W, bool silu, void* out, cudaStream_t st) {
  constexpr int V = 16 / sizeof(Tin);
  const unsigned grid = (unsigned)(((int64_t)N * (D / V) + kConvThreads - 1) / kConvThreads);
  const Tin* xp = static_cast<const Tin*>(x);
  Tin* sp = static_cast<Tin*>(state);
  Tin* op = static_cast<Tin*>(out);
  switch (W) {
    case 2: conv_step_kernel<Tin, 2><<<grid, kConvThreads, 0, st>>>(xp, xs, w, b, sp, N, D, silu, op); break;
    case 3: conv_step_kernel<Tin, 3><<<grid, kConvThreads, 0, st>>>(xp, xs, w, b, sp, N, D, silu, op); break;
    default: conv_step_kernel<Tin, 4><<<grid, kConvThreads, 0, st>>>(xp, xs, w, b, sp, N, D, silu, op); break;
  }
  return cudaGetLastError();
}

template <typename Tin>
cudaError_t dispatch_bwd(const ConvArgs& a, int W, cudaStream_t st) {
  const int64_t blocks = ((int64_t)a.strips * (a.D / kBV) + kConvThreads - 1) / kConvThreads;
  int64_t empty = 0;
  if (a.cu && a.d_init)
    empty = ((int64_t)a.num_seqs * (W - 1) * (a.D / kBV) + kConvThreads - 1) / kConvThreads;
  const unsigned grid = (unsigned)(blocks + empty);
  switch (W) {
    case 2: conv_bwd_kernel<Tin, 2><<<grid, kConvThreads, 0, st>>>(a, (unsigned)blocks); break;
    case 3: conv_bwd_kernel<Tin, 3><<<grid, kConvThreads, 0, st>>>(a, (unsigned)blocks); break;
    default: conv_bwd_kernel<Tin, 4><<<grid, kConvThreads, 0, st>>>(a, (unsigned)blocks); break;
  }
  return cudaGetLastError();
}

// argument checks that the three entries share (after the null checks)
kda_status check_conv(kda_dtype dt, int D, int W, kda_activation act, int64_t x_stride) {
  if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return KDA_ERR_INVALID_ARG;
  if (D <= 0 || W <= 0) return KDA_ERR_INVALID_ARG;
  if (D % 8 != 0 || W < 2 || W > 4 || D > (1 << 24)) return KDA_ERR_UNSUPPORTED;
  if (!stride_ok(x_stride, D, elem_bytes(dt))) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

// the launch grids are 32-bit
bool grid_fits(int64_t items) { return items / kConvThreads < 0x7ffffff0LL / 2; }

}  // namespace

cudaError_t launch_seqlens_plan(const int32_t* cu, int N, int T, StatusBlock* sb, int seg_len,
                                int32_t* seg_off, cudaStream_t stream) {
  seqlens_plan_kernel<<<1, 1024, 0, stream>>>(cu, N, T, sb, seg_len, seg_off);
  return cudaGetLastError();
}

}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_short_conv_fwd(const void* x, int64_t x_stride, const float* weight,
                              const float* bias, kda_dtype in_dtype, const void* init_state,
                              const int32_t* cu_seqlens, int num_seqs, int B, int T, int D,
                              int W, kda_activation activation, void* out, void* final_state,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !weight || !out || !workspace) return KDA_ERR_INVALID_ARG;
  if (kda_status s = check_conv(in_dtype, D, W, activation, x_stride)) return s;
  if (kda_status s = check_batch(cu_seqlens, num_seqs, B, T)) return s;
  const int64_t total = (int64_t)B * T, es = elem_bytes(in_dtype);
  const int64_t N = cu_seqlens ? num_seqs : B;
  const int64_t state_bytes = N * (W - 1) * D * es;
  const Span ins[] = {{x, row_bytes(total, x_stride, D, es)},
                      {weight, (int64_t)D * W * 4},
                      {bias, (int64_t)D * 4},
                      {init_state, state_bytes},
                      {cu_seqlens, (N + 1) * 4}};
  const Span outs[] = {{out, total * D * es}, {final_state, state_bytes},
                       {workspace, (int64_t)kStatusBytes}};
  if (kda_status s = check_spans(ins, outs)) return s;
  if (workspace_bytes < kStatusBytes) return KDA_ERR_WORKSPACE;
  const int V = (int)(16 / es);
  ConvArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.weight = weight;
  a.bias = bias;
  a.init = init_state;
  a.cu = cu_seqlens;
  a.num_seqs = (int)N;
  a.total = total;
  a.T = T;
  a.D = D;
  a.silu = activation == KDA_ACT_SILU;
  a.out = out;
  a.final_state = final_state;
  a.strip = strip_len(total, D / V, kUnroll, 32, kWantThreads);
  a.strips = (int)((total + a.strip - 1) / a.strip);
  a.sb = static_cast<StatusBlock*>(workspace);
  if (!grid_fits((int64_t)a.strips * (D / V)) || !grid_fits(N * (W - 1) * (D / V)))
    return KDA_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  if (cu_seqlens)
    if (cudaError_t e = launch_seqlens_plan(cu_seqlens, num_seqs, T, a.sb, 1, nullptr, st))
      return cuda_failure(e);
  const cudaError_t e = in_dtype == KDA_BF16 ? dispatch_fwd<__nv_bfloat16>(a, W, st)
                                             : dispatch_fwd<float>(a, W, st);
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

kda_status kda_short_conv_step(const void* x, int64_t x_stride, const float* weight,
                               const float* bias, kda_dtype in_dtype, void* state, int N, int D,
                               int W, kda_activation activation, void* out, void* stream) {
  if (!x || !weight || !state || !out) return KDA_ERR_INVALID_ARG;
  if (N <= 0) return KDA_ERR_INVALID_ARG;
  if (kda_status s = check_conv(in_dtype, D, W, activation, x_stride)) return s;
  const int64_t es = elem_bytes(in_dtype);
  const Span ins[] = {{x, row_bytes(N, x_stride, D, es)},
                      {weight, (int64_t)D * W * 4},
                      {bias, (int64_t)D * 4}};
  const Span outs[] = {{out, (int64_t)N * D * es}, {state, (int64_t)N * (W - 1) * D * es}};
  if (kda_status s = check_spans(ins, outs)) return s;
  if (!grid_fits((int64_t)N * (D / (16 / es)))) return KDA_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  const bool silu = activation == KDA_ACT_SILU;
  const cudaError_t e =
      in_dtype == KDA_BF16
          ? dispatch_step<__nv_bfloat16>(x, x_stride, weight, bias, state, N, D, W, silu, out, st)
          : dispatch_step<float>(x, x_stride, weight, bias, state, N, D, W, silu, out, st);
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

size_t kda_short_conv_bwd_workspace_size(int B, int T, int D, int W, int num_seqs) {
  (void)num_seqs;
  if (B <= 0 || T <= 0 || D <= 0 || D % 8 != 0 || D > (1 << 24) || W < 2 || W > 4 ||
      (int64_t)B * T > 0x7fffffffLL)
    return 0;
  const int64_t total = (int64_t)B * T;
  const int64_t strips = (total + bwd_strip(total, D) - 1) / bwd_strip(total, D);
  return kStatusBytes + sizeof(float) * (size_t)strips * (W + 1) * D;
}

kda_status kda_short_conv_bwd(const void* x, int64_t x_stride, const float* weight,
                              const float* bias, kda_dtype in_dtype, const void* init_state,
                              const float* dout, const float* d_final,
                              const int32_t* cu_seqlens, int num_seqs, int B, int T, int D,
                              int W, kda_activation activation, float* dx, float* dweight,
                              float* dbias, float* d_init, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!x || !weight || !dout || !dx || !dweight || !workspace) return KDA_ERR_INVALID_ARG;
  if (kda_status s = check_conv(in_dtype, D, W, activation, x_stride)) return s;
  if (kda_status s = check_batch(cu_seqlens, num_seqs, B, T)) return s;
  const int64_t total = (int64_t)B * T, es = elem_bytes(in_dtype);
  const int64_t N = cu_seqlens ? num_seqs : B;
  const int64_t rows = N * (W - 1) * D;
  const size_t need = kda_short_conv_bwd_workspace_size(B, T, D, W, num_seqs);
  const Span ins[] = {{x, row_bytes(total, x_stride, D, es)},
                      {weight, (int64_t)D * W * 4},
                      {bias, (int64_t)D * 4},
                      {init_state, rows * es},
                      {dout, total * D * 4},
                      {d_final, rows * 4},
                      {cu_seqlens, (N + 1) * 4}};
  const Span outs[] = {{dx, total * D * 4},
                       {dweight, (int64_t)D * W * 4},
                       {dbias, (int64_t)D * 4},
                       {d_init, rows * 4},
                       {workspace, (int64_t)need}};
  if (kda_status s = check_spans(ins, outs)) return s;
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
  ConvArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.weight = weight;
  a.bias = bias;
  a.init = init_state;
  a.cu = cu_seqlens;
  a.num_seqs = (int)N;
  a.total = total;
  a.T = T;
  a.D = D;
  a.silu = activation == KDA_ACT_SILU;
  a.dout = dout;
  a.d_final = d_final;
  a.dx = dx;
  a.d_init = d_init;
  a.strip = bwd_strip(total, D);
  a.strips = (int)((total + a.strip - 1) / a.strip);
  a.sb = static_cast<StatusBlock*>(workspace);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kStatusBytes);
  if (!grid_fits((int64_t)a.strips * (D / kBV)) || !grid_fits(N * (W - 1) * (D / kBV)))
    return KDA_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  if (cu_seqlens)
    if (cudaError_t e = launch_seqlens_plan(cu_seqlens, num_seqs, T, a.sb, 1, nullptr, st))
      return cuda_failure(e);
  cudaError_t e = in_dtype == KDA_BF16 ? dispatch_bwd<__nv_bfloat16>(a, W, st)
                                       : dispatch_bwd<float>(a, W, st);
  if (e != cudaSuccess) return cuda_failure(e);
  const int64_t n = (int64_t)(W + 1) * D;
  conv_bwd_sum_kernel<<<(unsigned)((n + 31) / 32), dim3(32, 8), 0, st>>>(
      a.partial, a.strips, D, W, dweight, dbias, cu_seqlens, a.sb);
  e = cudaGetLastError();
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

}  // extern "C"
