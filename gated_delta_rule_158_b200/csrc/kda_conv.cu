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
//
// Measured on a B200 (6455 GB/s copy): 65,000 packed tokens x 4096 bf16 with
// SiLU, 193 to 207 us = 5.2 to 5.5 TB/s.  Before the ring, with loads as they were needed, it
// took 507 us at eight channels a thread and 231 us at four; with the next rows
// prefetched to registers 239 us; with the ring 213 us, and 193 us once the
// strips filled whole waves.  One token of 256 sequences x 12,288: 11.2 us, 4.5
// TB/s.
// Gradients of 16,384 x 4096 (x bf16; dout, dx fp32): 114 us = 5.9 TB/s.
#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int kConvThreads = 256;
constexpr int kUnroll = 4;   // rows per step
constexpr int kRing = 16;    // rows of a thread's ring
constexpr int kFV = 4;       // channels per thread of the step kernel

// ------------------------------------------------------------ packed batch
// The status word: KDA_OK or KDA_ERR_BAD_SEQLENS.
__global__ void __launch_bounds__(1024) seqlens_plan_kernel(const int32_t* __restrict__ cu, int N,
                                                            int T, StatusBlock* sb) {
  int bad = threadIdx.x == 0 && (cu[0] != 0 || cu[N] != T);
  for (int n = threadIdx.x; n < N; n += 1024) bad |= cu[n + 1] < cu[n];
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    sb->status = bad ? KDA_ERR_BAD_SEQLENS : KDA_OK;
    sb->detail = 0;
    sb->never_set = 0;
    sb->seqlens_ok = bad ? 0 : 1;
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
    // (debug builds) a run outside the batch ends at its token: nothing beyond
    // is read
    if (!in_bounds(a.sb, r.end, a.total + 1, kSiteConvRun) ||
        !in_bounds(a.sb, t, r.end, kSiteConvRun)) {
      r.start = t;
      r.end = t + 1;
    }
  } else {
    r.n = t / a.T;
    r.start = r.n * a.T;
    r.end = r.start + a.T;
  }
  return r;
}

// Rows of V channels as V / 2 pairs.
template <typename Tin, int V>
__device__ __forceinline__ void load_row(const Tin* p, f2 (&v)[V / 2]) {
  float f[V];
  load_vec<Tin, V>(p, f);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
}
template <int V, typename T>
__device__ __forceinline__ void store_row(T* p, const f2 (&v)[V / 2]) {
  float f[V];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
  store_vec<V>(p, f);
}
template <typename T, int V>
__device__ __forceinline__ void raw_row(const Raw<T, V>& r, f2 (&v)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) v[i] = pack2(r.at(2 * i), r.at(2 * i + 1));
}

// the row `back` places before the run's start (1 = the newest kept row)
template <typename Tin, int W, int V>
__device__ __forceinline__ void kept_row(const ConvArgs& a, int n, int back, int c,
                                         f2 (&v)[V / 2]) {
  if (a.init) {
    load_row<Tin, V>(static_cast<const Tin*>(a.init) +
                         ((int64_t)n * (W - 1) + (W - 1 - back)) * a.D + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = zero2();
  }
}

// win = the W - 1 rows before token t of run r, oldest first
template <typename Tin, int W, int V>
__device__ __forceinline__ void fill_window(const ConvArgs& a, const Run& r, int t, int c,
                                            f2 (*win)[V / 2]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int s = t - (W - 1) + j;
    if (s >= r.start)
      load_row<Tin, V>(static_cast<const Tin*>(a.x) + (int64_t)s * a.x_stride + c, win[j]);
    else
      kept_row<Tin, W, V>(a, r.n, r.start - s, c, win[j]);
  }
}

template <int W, int P>
__device__ __forceinline__ void push_row(f2 (*win)[P], const f2 (&row)[P]) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) win[j][i] = win[j + 1][i];
#pragma unroll
  for (int i = 0; i < P; ++i) win[W - 2][i] = row[i];
}

template <int W, int V>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int c, f2 (&w)[W][V / 2],
                                          f2 (&b)[V / 2]) {
  // V * W consecutive floats; c is a multiple of V, and V of 4: whole 16-byte pieces
  float flat[V * W], bias[V] = {};
#pragma unroll
  for (int i = 0; i < V * W; i += 4) {
    float f[4];
    load_vec<float, 4>(a.weight + (int64_t)c * W + i, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) flat[i + j] = f[j];
  }
  if (a.bias) load_vec<float, V>(a.bias + c, bias);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    b[i] = pack2(bias[2 * i], bias[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = pack2(flat[2 * i * W + j], flat[(2 * i + 1) * W + j]);
  }
}

// p = b + sum_j w[j] rows[j], rows[0] the oldest
template <int W, int P, int N>
__device__ __forceinline__ void taps_dot(const f2 (&w)[W][P], const f2 (&b)[P],
                                         const f2 (&rows)[N][P], int first, f2 (&p)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    p[i] = b[i];
#pragma unroll
    for (int j = 0; j < W; ++j) p[i] = fma2(w[j][i], rows[first + j][i], p[i]);
  }
}

template <int P>
__device__ __forceinline__ void silu_row(f2 (&p)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) p[i] = mul2(p[i], sigmoid2(p[i]));
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
  f2 v[V / 2];
  if (s >= 0)
    load_row<Tin, V>(static_cast<const Tin*>(a.x) + (start + s) * a.x_stride + c, v);
  else
    kept_row<Tin, W, V>(a, n, (int)-s, c, v);
  store_row<V>(static_cast<Tin*>(a.final_state) + r * a.D + c, v);  // exact: the type is the same
}

// Threads [0, strips * D / V) take a strip each, channel groups fastest; the
// blocks behind them write the final state.  A thread's rows come through a
// ring of kRing rows in shared memory that it alone copies to and reads
// (cp.async): 16 bytes x 12 to 16 rows in flight a thread, without a register.
template <typename Tin, int W>
__global__ void __launch_bounds__(kConvThreads, 2) conv_fwd_kernel(const ConvArgs a,
                                                                   unsigned strip_blocks) {
  constexpr int V = 16 / (int)sizeof(Tin), P = V / 2, U = kUnroll, GROUPS = kRing / U;
  extern __shared__ __align__(16) char ring[];
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
  char* const own = ring + threadIdx.x * 16;
  auto copy_group = [&](int g) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = g * U + u;
      if (t0 + k < t1)
        copy_in<16>(own + (g % GROUPS * U + u) * kConvThreads * 16, x + (int64_t)k * a.x_stride,
                    true);
    }
    copies_issued();
  };
#pragma unroll
  for (int g = 0; g < GROUPS - 1; ++g) copy_group(g);

  f2 w[W][P], b[P];
  f2 rows[W - 1 + U][P];  // the W - 1 rows before the step's tokens, then theirs
  load_taps<W, V>(a, c, w, b);
  Run r = run_at(a, t0);
  fill_window<Tin, W, V>(a, r, t0, c, rows);
  for (int t = t0, g = 0; t < t1; t += U, ++g) {
    copy_group(g + GROUPS - 1);  // over the group that has been read
    copies_landed_but<GROUPS - 1>();
    const char* at = own + g % GROUPS * U * kConvThreads * 16;
    if (t + U <= t1 && t + U <= r.end) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        load_row<Tin, V>(reinterpret_cast<const Tin*>(at + u * kConvThreads * 16),
                         rows[W - 1 + u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f2 p[P];
        taps_dot<W, P>(w, b, rows, u, p);
        if (a.silu) silu_row(p);
        store_row<V>(out + (int64_t)u * a.D, p);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) rows[j][i] = rows[U + j][i];
    } else {
      for (int u = 0; u < U && t + u < t1; ++u) {
        if (t + u >= r.end) {  // the next sequence that has tokens
          r = run_at(a, t + u);
          fill_window<Tin, W, V>(a, r, t + u, c, rows);
        }
        f2 p[P];
        load_row<Tin, V>(reinterpret_cast<const Tin*>(at + u * kConvThreads * 16), rows[W - 1]);
        taps_dot<W, P>(w, b, rows, 0, p);
        if (a.silu) silu_row(p);
        store_row<V>(out + (int64_t)u * a.D, p);
        push_row<W, P>(rows, rows[W - 1]);
      }
    }
    out += (int64_t)U * a.D;
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
  constexpr int P = V / 2;
  f2 w[W][P], b[P], rows[NS][W][P];
  Raw<Tin, V> raw[NS][W];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    if (n0 + s >= N) break;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[s][j].load(state + ((n0 + s) * (W - 1) + j) * a.D + c);
    raw[s][W - 1].load(static_cast<const Tin*>(a.x) + (n0 + s) * a.x_stride + c);
  }
  load_taps<W, V>(a, c, w, b);
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    if (n0 + s >= N) break;
#pragma unroll
    for (int j = 0; j < W; ++j) raw_row(raw[s][j], rows[s][j]);
    f2 p[P];
    taps_dot<W, P>(w, b, rows[s], 0, p);
    if (a.silu) silu_row(p);
    store_row<V>(static_cast<Tin*>(a.out) + (n0 + s) * a.D + c, p);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[s][j + 1].store(state + ((n0 + s) * (W - 1) + j) * a.D + c);
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
constexpr int kBV = 4;     // channels per thread
constexpr int kBRing = 12; // rows of a thread's ring

template <typename Tin, int W>
__global__ void __launch_bounds__(kConvThreads, 2) conv_bwd_kernel(const ConvArgs a,
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

  constexpr int P = V / 2, U = kUnroll, GROUPS = kBRing / U;
  // the thread's ring: of each row x, then dout
  constexpr int XB = V * (int)sizeof(Tin), DB = V * 4;
  extern __shared__ __align__(16) char ring[];
  char* const own_x = ring + threadIdx.x * XB;
  char* const own_d = ring + kBRing * kConvThreads * XB + threadIdx.x * DB;
  const Tin* xs = static_cast<const Tin*>(a.x) + (int64_t)t0 * a.x_stride + c;
  const float* dsrc = a.dout + (int64_t)t0 * a.D + c;
  auto copy_group = [&](int g) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = g * U + u, at = (g % GROUPS * U + u) * kConvThreads;
      if (t0 + k < t1) {
        copy_in<XB>(own_x + at * XB, xs + (int64_t)k * a.x_stride, true);
        copy_in<DB>(own_d + at * DB, dsrc + (int64_t)k * a.D, true);
      }
    }
    copies_issued();
  };
#pragma unroll
  for (int g = 0; g < GROUPS - 1; ++g) copy_group(g);
  f2 w[W][P], b[P], dw[W][P], db[P];
  // the W - 1 rows (and values of ds) before the step's tokens, then theirs
  f2 rows[W - 1 + U][P], dss[W - 1 + U][P];
  load_taps<W, V>(a, c, w, b);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    db[i] = zero2();
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = zero2();
  }
  // ds of the token whose row is rows[u + W - 1], over its dout in dss[u + W - 1]
  auto ds_of = [&](int u) {
    if (!a.silu) return;
    f2 p[P];
    taps_dot<W, P>(w, b, rows, u, p);
#pragma unroll
    for (int i = 0; i < P; ++i) {  // silu'(p) = s + p s (1 - s)
      const f2 s = sigmoid2(p[i]), ps = mul2(p[i], s);
      dss[u + W - 1][i] = mul2(
          dss[u + W - 1][i], fma2(ps, fma2(s, pack2(-1.f, -1.f), pack2(1.f, 1.f)), s));
    }
  };
  auto sums_of = [&](int u) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      db[i] = add2(db[i], dss[u + W - 1][i]);
#pragma unroll
      for (int j = 0; j < W; ++j) dw[j][i] = fma2(dss[u + W - 1][i], rows[u + j][i], dw[j][i]);
    }
  };
  // the gradient of the row W - 1 places before the token
  auto row_gradient = [&](int u, f2 (&g)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      g[i] = mul2(w[0][i], dss[u + W - 1][i]);
#pragma unroll
      for (int j = 1; j < W; ++j) g[i] = fma2(w[j][i], dss[u + W - 1 - j][i], g[i]);
    }
  };
  Run r;
  int ta, tb;  // the run's tokens within the strip
  bool head;
  auto start_run = [&](int t) {
    r = run_at(a, t);
    ta = t;
    tb = min(t1, r.end);
    head = ta == r.start && a.d_init;
    fill_window<Tin, W, V>(a, r, ta, c, rows);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) dss[j][i] = zero2();
  };
  // token t alone, its row and dout in rows[W - 1] and dss[W - 1]
  auto token = [&](int t, bool own) {
    if (t < r.end) ds_of(0);
    if (own) sums_of(0);
    const int s = t - (W - 1);
    if (s >= ta || head) {
      f2 g[P];
      row_gradient(0, g);
      const int f = t - r.end;  // the row's place in the final state
      if (f >= 0 && a.d_final) {
        f2 d[P];
        load_row<float, V>(a.d_final + ((int64_t)r.n * (W - 1) + f) * a.D + c, d);
#pragma unroll
        for (int i = 0; i < P; ++i) g[i] = add2(g[i], d[i]);
      }
      float* to = s >= ta ? a.dx + (int64_t)s * a.D
                          : a.d_init + ((int64_t)r.n * (W - 1) + (s - ta + W - 1)) * a.D;
      store_row<V>(to + c, g);
    }
    push_row<W, P>(rows, rows[W - 1]);
    push_row<W, P>(dss, dss[W - 1]);
  };
  // the W - 1 tokens behind a run: the sequence's next ones (whose sums belong
  // to the next strip), or none
  auto end_run = [&]() {
    for (int t = tb; t < tb + W - 1; ++t) {
#pragma unroll
      for (int i = 0; i < P; ++i) rows[W - 1][i] = dss[W - 1][i] = zero2();
      if (t < r.end) {
        load_row<Tin, V>(static_cast<const Tin*>(a.x) + (int64_t)t * a.x_stride + c, rows[W - 1]);
        load_row<float, V>(a.dout + (int64_t)t * a.D + c, dss[W - 1]);
      }
      token(t, false);
    }
  };
  start_run(t0);
  float* gp = a.dx + (int64_t)t0 * a.D + c;
  for (int t = t0, g = 0; t < t1; t += U, ++g) {
    copy_group(g + GROUPS - 1);  // over the group that has been read
    copies_landed_but<GROUPS - 1>();
    const int at = g % GROUPS * U * kConvThreads;
    if (t >= ta + W - 1 && t + U <= tb) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        load_row<Tin, V>(reinterpret_cast<const Tin*>(own_x + (at + u * kConvThreads) * XB),
                         rows[W - 1 + u]);
        load_row<float, V>(reinterpret_cast<const float*>(own_d + (at + u * kConvThreads) * DB),
                           dss[W - 1 + u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f2 gr[P];
        ds_of(u);
        sums_of(u);
        row_gradient(u, gr);
        store_row<V>(gp + (int64_t)(u - (W - 1)) * a.D, gr);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          rows[j][i] = rows[U + j][i];
          dss[j][i] = dss[U + j][i];
        }
    } else {
      for (int u = 0; u < U && t + u < t1; ++u) {
        if (t + u >= tb) {
          end_run();
          start_run(t + u);
        }
        load_row<Tin, V>(reinterpret_cast<const Tin*>(own_x + (at + u * kConvThreads) * XB),
                         rows[W - 1]);
        load_row<float, V>(reinterpret_cast<const float*>(own_d + (at + u * kConvThreads) * DB),
                           dss[W - 1]);
        token(t + u, true);
      }
    }
    gp += (int64_t)U * a.D;
  }
  end_run();
  // [strip][W + 1][D]: tap j of all channels, then the bias
  float* part = a.partial + (int64_t)strip * (W + 1) * a.D + c;
#pragma unroll
  for (int j = 0; j < W; ++j) store_row<V>(part + (int64_t)j * a.D, dw[j]);
  store_row<V>(part + (int64_t)W * a.D, db);
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

// Tokens per strip.  Long strips read fewer head rows again and leave fewer
// partial sums, but the strips have to fill the GPU evenly: 148 SMs hold two
// blocks each, so the batch is cut into as many strips as fill one, two, ..
// such waves, the fewest waves that keep a strip within `hi` tokens.
int strip_len(int64_t total, int groups, int lo, int hi) {
  int64_t per_wave = 148LL * 2 * kConvThreads / groups;
  if (per_wave < 1) per_wave = 1;
  int64_t waves = (total + per_wave * hi - 1) / (per_wave * hi);
  int64_t s = (total + per_wave * waves - 1) / (per_wave * waves);
  s = (s + 3) / 4 * 4;
  return (int)(s < lo ? lo : s);
}

int bwd_strip(int64_t total, int D) { return strip_len(total, D / kBV, 16, 512); }

// shared memory above the default needs the kernel's permission
template <typename K>
cudaError_t launch_ring(K kernel, const ConvArgs& a, int64_t blocks, int64_t more, size_t bytes,
                        cudaStream_t st) {
  if (bytes > 48 * 1024)
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)bytes))
      return e;
  kernel<<<(unsigned)(blocks + more), kConvThreads, bytes, st>>>(a, (unsigned)blocks);
  return cudaGetLastError();
}

template <typename Tin>
cudaError_t dispatch_fwd(const ConvArgs& a, int W, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(Tin);
  constexpr size_t bytes = (size_t)kRing * kConvThreads * 16;
  const int64_t blocks = ((int64_t)a.strips * (a.D / V) + kConvThreads - 1) / kConvThreads;
  int64_t fin = 0;
  if (a.final_state)
    fin = ((int64_t)a.num_seqs * (W - 1) * (a.D / V) + kConvThreads - 1) / kConvThreads;
  switch (W) {
    case 2: return launch_ring(conv_fwd_kernel<Tin, 2>, a, blocks, fin, bytes, st);
    case 3: return launch_ring(conv_fwd_kernel<Tin, 3>, a, blocks, fin, bytes, st);
    default: return launch_ring(conv_fwd_kernel<Tin, 4>, a, blocks, fin, bytes, st);
  }
}

template <typename Tin, int W>
cudaError_t launch_step(const ConvArgs& a, void* state, int N, cudaStream_t st) {
  const int CG = a.D / kFV;
  Tin* sp = static_cast<Tin*>(state);
  constexpr int NS = 4;
  const int64_t few = ((int64_t)N + NS - 1) / NS * CG;  // threads with four sequences each
  // From 256 such threads an SM on; one sequence a thread against four, W = 4,
  // bf16: 2.4 and 3.1 us at 55 threads an SM (32 sequences x 4096), 3.2 both at
  // 166, 5.9 and 5.3 at 332, 6.7 and 5.1 at 443, 15.0 and 11.5 at 1328 (256 x
  // 12,288).
  if (few >= 148 * 256) {
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
  constexpr size_t bytes = (size_t)kBRing * kConvThreads * kBV * (sizeof(Tin) + 4);
  const int64_t blocks = ((int64_t)a.strips * (a.D / kBV) + kConvThreads - 1) / kConvThreads;
  int64_t empty = 0;
  if (a.cu && a.d_init)
    empty = ((int64_t)a.num_seqs * (W - 1) * (a.D / kBV) + kConvThreads - 1) / kConvThreads;
  switch (W) {
    case 2: return launch_ring(conv_bwd_kernel<Tin, 2>, a, blocks, empty, bytes, st);
    case 3: return launch_ring(conv_bwd_kernel<Tin, 3>, a, blocks, empty, bytes, st);
    default: return launch_ring(conv_bwd_kernel<Tin, 4>, a, blocks, empty, bytes, st);
  }
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

cudaError_t launch_plan(const ConvArgs& a, cudaStream_t stream) {
  seqlens_plan_kernel<<<1, 1024, 0, stream>>>(a.cu, a.num_seqs, a.T, a.sb);
  return cudaGetLastError();
}

}  // namespace
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
  a.strip = strip_len(total, D / V, 8, 128);
  a.strips = (int)((total + a.strip - 1) / a.strip);
  a.sb = static_cast<StatusBlock*>(workspace);
  if (!grid_fits((int64_t)a.strips * (D / V)) || !grid_fits(N * (W - 1) * (D / V)))
    return KDA_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  if (cu_seqlens)
    if (cudaError_t e = launch_plan(a, st))
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
  if (B <= 0 || T <= 0 || D <= 0 || D % 8 != 0 || D > (1 << 24) || W < 2 || W > 4 ||
      (int64_t)B * T > kMaxRows || num_seqs < 0 || num_seqs > kMaxRows)
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
    if (cudaError_t e = launch_plan(a, st))
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
