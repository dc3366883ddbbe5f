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
constexpr int kUnroll = 4;  // rows per step; the next step's are in flight
constexpr int kFV = 4;      // channels per thread of the prompt kernel

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
  int n, start, end;
};

__device__ __forceinline__ Run run_at(const ConvArgs& a, int t) {
  Run r;
  if (a.cu) {
    r.n = find_range(a.cu, a.num_seqs, t);
    r.start = __ldg(a.cu + r.n);
    r.end = __ldg(a.cu + r.n + 1);
  } else {
    r.n = t / a.T;
    r.start = r.n * a.T;
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
__device__ __forceinline__ void fill_window(const ConvArgs& a, const Run& r, int t, int c,
                                            float (&win)[W - 1][V]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int s = t - (W - 1) + j;
    if (s >= r.start)
      load_vec<Tin, V>(static_cast<const Tin*>(a.x) + (int64_t)s * a.x_stride + c, win[j]);
    else
      kept_row<Tin, W, V>(a, r.n, r.start - s, c, win[j]);
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
  // V * W consecutive floats; c is a multiple of V, so V * W floats are a whole
  // number of 8- or 16-byte pieces
  float flat[V * W];
  constexpr int P = V * W % 4 == 0 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < V * W; i += P) {
    float f[P];
    load_vec<float, P>(a.weight + (int64_t)c * W + i, f);
#pragma unroll
    for (int j = 0; j < P; ++j) flat[i + j] = f[j];
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
// blocks behind them write the final state.  Four channels a thread: eight
// would double the window and tap registers and halve the warps in flight
// (bf16 at W = 4: 506 us instead of KERNEL_US at 65,000 x 4096).
template <typename Tin, int W>
__global__ void __launch_bounds__(kConvThreads, sizeof(Tin) == 4 ? 2 : 3) conv_fwd_kernel(const ConvArgs a,
                                                                   unsigned strip_blocks) {
  constexpr int V = kFV;
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
  const int strip = (int)(idx / CG);
  if (strip >= a.strips) return;
  const int c = (int)(idx - (int64_t)strip * CG) * V;
  const int t0 = strip * a.strip;
  const int t1 = (int)min((int64_t)t0 + a.strip, a.total);
  const Tin* x = static_cast<const Tin*>(a.x) + (int64_t)t0 * a.x_stride + c;
  Tin* out = static_cast<Tin*>(a.out) + (int64_t)t0 * a.D + c;

  float w[V][W], b[V], win[W - 1][V];
  load_taps<W, V>(a, c, w, b);
  Run r = run_at(a, t0);
  fill_window<Tin, W, V>(a, r, t0, c, win);
  // one token whose row is given
  auto token = [&](const float (&row)[V], Tin* to) {
    float p[V];
    taps_dot<W, V>(w, b, win, row, p);
    if (a.silu) {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= sigmoid_fast(p[i]);
    }
    store_vec<V>(to, p);
    push_row<W, V>(win, row);
  };
  Raw<Tin, V> next[kUnroll];
  auto fetch = [&](int t) {  // the kUnroll rows from t on
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (t + u < t1) next[u].load(x + (int64_t)(t + u - t0) * a.x_stride);
  };
  fetch(t0);
  for (int t = t0; t < t1; t += kUnroll) {
    Raw<Tin, V> cur[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) cur[u] = next[u];
    fetch(t + kUnroll);  // in flight while these are worked on
    float row[V];
    if (t + kUnroll <= t1 && t + kUnroll <= r.end) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        cur[u].get(row);
        token(row, out + (int64_t)u * a.D);
      }
    } else {
      for (int u = 0; u < kUnroll && t + u < t1; ++u) {
        if (t + u >= r.end) {  // the next sequence that has tokens
          r = run_at(a, t + u);
          fill_window<Tin, W, V>(a, r, t + u, c, win);
        }
        load_vec<Tin, V>(x + (int64_t)(t + u - t0) * a.x_stride, row);
        token(row, out + (int64_t)u * a.D);
      }
    }
    out += (int64_t)kUnroll * a.D;
  }
}

// One token of NS sequences per thread and channel group; the state's rows move
// one place up.  The taps (16 bytes a channel) weigh as much as the rows, so
// with enough sequences a thread keeps them for four.
template <typename Tin, int W, int NS>
__global__ void __launch_bounds__(kConvThreads)
    conv_step_kernel(const ConvArgs a, Tin* __restrict__ state, int N) {
  constexpr int V = kFV;
  const int CG = a.D / V;
  const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  const int64_t n0 = idx / CG * NS;
  if (n0 >= N) return;
  const int c = (int)(idx % CG) * V;
  float w[V][W], b[V];
  float win[NS][W - 1][V], row[NS][V];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    if (n0 + s >= N) break;
    load_vec<Tin, V>(static_cast<const Tin*>(a.x) + (n0 + s) * a.x_stride + c, row[s]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      load_vec<Tin, V>(state + ((n0 + s) * (W - 1) + j) * a.D + c, win[s][j]);
  }
  load_taps<W, V>(a, c, w, b);
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    if (n0 + s >= N) break;
    float p[V];
    taps_dot<W, V>(w, b, win[s], row[s], p);
    if (a.silu) {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= sigmoid_fast(p[i]);
    }
    store_vec<V>(static_cast<Tin*>(a.out) + (n0 + s) * a.D + c, p);
    push_row<W, V>(win[s], row[s]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      store_vec<V>(state + ((n0 + s) * (W - 1) + j) * a.D + c, win[s][j]);
  }
}

// --------------------------------------------------------------- gradients
// A strip [t0, t1) is walked forward, run by run.  Token t gives ds[t]; the
// gradient of row s is complete once ds[s .. s + W - 1] are known, so the walk
// goes W - 1 tokens past the run (into the next strip's tokens, whose ds it
// forms again, or past the sequence's end, where ds is 0), and a window of
// the last W - 1 values of ds stays in registers.  dweight and dbias are
// summed in registers over the strip's own tokens and leave as one partial
// row per strip, added in strip order by conv_bwd_sum_kernel.
constexpr int kBV = 2;  // channels per thread
constexpr int kBU = 4;  // tokens whose rows are in flight

template <typename Tin, int W>
__global__ void __launch_bounds__(kConvThreads, sizeof(Tin) == 4 ? 2 : 3) conv_bwd_kernel(const ConvArgs a,
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
  const int strip = (int)(idx / CG);
  if (strip >= a.strips) return;
  const int c = (int)(idx - (int64_t)strip * CG) * V;
  const int t0 = strip * a.strip;
  const int t1 = (int)min((int64_t)t0 + a.strip, a.total);

  float w[V][W], b[V], win[W - 1][V], dsw[W - 1][V], dw[V][W], db[V];
  load_taps<W, V>(a, c, w, b);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[i][j] = 0.f;
  }
  for (int ta = t0; ta < t1;) {
    const Run r = run_at(a, ta);
    const int tb = min(t1, r.end);
    fill_window<Tin, W, V>(a, r, ta, c, win);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) dsw[j][i] = 0.f;
    const bool head = ta == r.start && a.d_init;
    // token t's ds from its rows, its sums; then the gradient of row t - (W-1)
    auto token = [&](int t, const float (&row)[V], const float (&dout)[V], bool own, bool give) {
      float ds[V];
#pragma unroll
      for (int i = 0; i < V; ++i) ds[i] = dout[i];
      if (a.silu) {
        float p[V];
        taps_dot<W, V>(w, b, win, row, p);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float sg = sigmoid_fast(p[i]);
          ds[i] *= sg * fmaf(p[i], 1.f - sg, 1.f);
        }
      }
      if (own) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          db[i] += ds[i];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) dw[i][j] = fmaf(ds[i], win[j][i], dw[i][j]);
          dw[i][W - 1] = fmaf(ds[i], row[i], dw[i][W - 1]);
        }
      }
      push_row<W, V>(win, row);
      if (give) {
        float g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          g[i] = w[i][0] * ds[i];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) g[i] = fmaf(w[i][W - 1 - j], dsw[j][i], g[i]);
        }
        const int s = t - (W - 1);
        const int f = s - (r.end - (W - 1));  // its row of the final state
        if (f >= 0 && a.d_final) {
          float d[V];
          load_vec<float, V>(a.d_final + ((int64_t)r.n * (W - 1) + f) * a.D + c, d);
#pragma unroll
          for (int i = 0; i < V; ++i) g[i] += d[i];
        }
        float* to = s >= ta ? a.dx + (int64_t)s * a.D
                            : a.d_init + ((int64_t)r.n * (W - 1) + (s - ta + W - 1)) * a.D;
        store_vec<V>(to + c, g);
      }
      push_row<W, V>(dsw, ds);
    };
    const Tin* xp = static_cast<const Tin*>(a.x) + (int64_t)ta * a.x_stride + c;
    const float* dp = a.dout + (int64_t)ta * a.D + c;
    Raw<Tin, V> nx[kBU];
    Raw<float, V> nd[kBU];
    auto fetch = [&](int t) {
#pragma unroll
      for (int u = 0; u < kBU; ++u)
        if (t + u < tb) {
          nx[u].load(xp + (int64_t)(t + u - ta) * a.x_stride);
          nd[u].load(dp + (int64_t)(t + u - ta) * a.D);
        }
    };
    fetch(ta);
    // the run's tokens, then the W - 1 behind them
    for (int t = ta; t < tb; t += kBU) {
      Raw<Tin, V> cx[kBU];
      Raw<float, V> cd[kBU];
#pragma unroll
      for (int u = 0; u < kBU; ++u) {
        cx[u] = nx[u];
        cd[u] = nd[u];
      }
      fetch(t + kBU);  // in flight while these are worked on
      float row[V], dout[V];
      if (t >= ta + W - 1 && t + kBU <= tb) {
#pragma unroll
        for (int u = 0; u < kBU; ++u) {
          cx[u].get(row);
          cd[u].get(dout);
          token(t + u, row, dout, true, true);
        }
      } else {
        for (int u = 0; u < kBU && t + u < tb; ++u) {
          load_vec<Tin, V>(xp + (int64_t)(t + u - ta) * a.x_stride, row);
          load_vec<float, V>(dp + (int64_t)(t + u - ta) * a.D, dout);
          token(t + u, row, dout, true, head || t + u - (W - 1) >= ta);
        }
      }
    }
    for (int t = tb; t < tb + W - 1; ++t) {
      float row[V] = {}, dout[V] = {};
      if (t < r.end) {
        load_vec<Tin, V>(static_cast<const Tin*>(a.x) + (int64_t)t * a.x_stride + c, row);
        load_vec<float, V>(a.dout + (int64_t)t * a.D + c, dout);
      }
      token(t, row, dout, false, head || t - (W - 1) >= ta);
    }
    ta = tb;
  }
  // [strip][W + 1][D]: tap j of all channels, then the bias
  float* part = a.partial + (int64_t)strip * (W + 1) * a.D + c;
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
  constexpr int V = kFV;
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

template <typename Tin, int W>
cudaError_t launch_step(const ConvArgs& a, void* state, int N, cudaStream_t st) {
  const int CG = a.D / kFV;
  Tin* sp = static_cast<Tin*>(state);
  constexpr int NS = 4;
  const int64_t few = ((int64_t)N + NS - 1) / NS * CG;  // threads with four sequences each
  if (few >= kWantThreads / 2) {
    conv_step_kernel<Tin, W, NS>
        <<<(unsigned)((few + kConvThreads - 1) / kConvThreads), kConvThreads, 0, st>>>(a, sp, N);
  } else {
    const int64_t all = (int64_t)N * CG;
    conv_step_kernel<Tin, W, 1>
        <<<(unsigned)((all + kConvThreads - 1) / kConvThreads), kConvThreads, 0, st>>>(a, sp, N);
  }
  return cudaGetLastError();
}

template <typename Tin>
cudaError_t dispatch_step(const ConvArgs& a, void* state, int N, int W, cudaStream_t st) {
  switch (W) {
    case 2: return launch_step<Tin, 2>(a, state, N, st);
    case 3: return launch_step<Tin, 3>(a, state, N, st);
    default: return launch_step<Tin, 4>(a, state, N, st);
  }
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
  const int V = kFV;
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
  if (!grid_fits((int64_t)N * (D / kFV))) return KDA_ERR_UNSUPPORTED;
  ConvArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.weight = weight;
  a.bias = bias;
  a.D = D;
  a.silu = activation == KDA_ACT_SILU;
  a.out = out;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = in_dtype == KDA_BF16
                            ? dispatch_step<__nv_bfloat16>(a, state, N, W, st)
                            : dispatch_step<float>(a, state, N, W, st);
  return e == cudaSuccess ? KDA_OK : cuda_failure(e);
}

size_t kda_short_conv_bwd_workspace_size(int B, int T, int D, int W, int num_seqs) {
  (void)num_seqs;
  if (B <= 0 || T <= 0 || D <= 0 || D % 8 != 0 || D > (1 << 24) || W < 2 || W > 4 ||
      (int64_t)B * T > kMaxRows)
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
