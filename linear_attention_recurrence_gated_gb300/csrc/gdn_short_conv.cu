// Short causal depthwise convolution with a bias and an activation: prompts (dense rows
// or packed sequences), gradients, and single tokens on the pages of a pool.
//
//   z_t = bias + sum_{k < K} w[ch, k] x[t - (K - 1) + k],   y_t = silu(z_t) (or z_t)
//   dz = dy silu'(z),   dx_t = sum_k w[ch, k] dz[t + (K - 1) - k],
//   dw[ch, k] = sum_t dz_t x[t - (K - 1) + k],   dbias = sum_t dz_t
//
// with x before a sequence's start taken from its prefix (else zero).  A thread walks over
// some tens or hundreds of tokens of four channels, in packed fp32 arithmetic, and keeps
// the last K - 1 inputs (backward: and the K - 1 unfinished rows of dx) in registers, so
// that a row is read once but at the segments' seams.  Its rows come through a ring in
// shared memory that asynchronous copies fill some batches ahead (each thread its own
// part: no barriers).  Forward, 32 packed sequences of 120k tokens together, 1280 channels,
// bf16: 106 us, 5.8 TB/s, bound by HBM (with rows asked for a batch ahead in registers 155).
// Backward, [4, 4096, 1280]: 33 us, 3.8 TB/s, 5 of them the second launch; its multiply-adds'
// pipe is busy for half of the rest (in registers 50).
#include "gdn_launch.cuh"
#include "gdn_layers.cuh"

namespace gdn {
namespace conv {
namespace {

using namespace layer;

constexpr int kThreads = 256;
constexpr int kBatch = 4;   // rows copied, and gone over, together
constexpr int kFar = 1 << 30;   // tokens counted from a thread's first: farther ones do not matter

// A thread's part of the ring: `stages` batches of kBatch rows, four elements each.
template <typename T, int STAGES>
struct Ring {
  Raw4<T> *at;   // [stage][row][thread]
  __device__ __forceinline__ void copy(int batch, const T *row, int64_t stride, int rows) const {
    Raw4<T> *to = at + batch % STAGES * kBatch * kThreads;
#pragma unroll
    for (int i = 0; i < kBatch; ++i, to += kThreads, row += stride)
      if (i < rows) {
        const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
        if constexpr (sizeof(T) == 2)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(s), "l"(row) : "memory");
        else
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(row) : "memory");
      }
  }
  __device__ __forceinline__ Raw4<T> row(int batch, int i) const {
    return at[(batch % STAGES * kBatch + i) * kThreads];
  }
};
__device__ __forceinline__ void close_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {   // all but the last N have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// (fp32: 48 KB a CTA of the forward pass, three an SM; 85 KB of the backward pass, two.  bf16,
// backward, [4, 4096, 1280]: two stages 33 us, three and four 35, six 43; forward, packed,
// three or four 106 to 108)
template <typename T, bool BACK> constexpr int kStages = BACK ? 2 : sizeof(T) == 2 ? 4 : 3;

struct Params {
  Sequences seq;
  const void *x, *x_prev, *dy, *d_tail;
  const float *w, *bias;
  void *y, *x_tail, *dx, *dx_prev;
  float *dw, *dbias;
  float *part;          // [parts][C][K + 1]
  int64_t sx;           // elements from token to token of x
  int32_t C, lanes;     // lanes: threads side by side along the channels (a power of two)
  int32_t walks_y;      // forward: grid rows that take tokens; the rest take the sequences' ends
  int64_t segment;
  int32_t parts;
  bool silu;
};

// The sequence of a token, walking forward.
struct At {
  int n;
  int64_t start, end;
  bool good;
  __device__ __forceinline__ void look(const Sequences &q) {
    int64_t len = 0;
    good = q.bounds(n, start, len);
    end = start + len;
  }
  // the sequence of token t (first: a token at or before it, the same in the whole warp)
  __device__ __forceinline__ void find(const Sequences &q, int64_t first, int64_t t) {
    if (q.cu == nullptr) {
      n = (int)(t / q.seq_len);
      start = n * q.seq_len;
      end = start + q.seq_len;
      good = true;
      return;
    }
    n = q.find(first);
    next_to(q, t);
  }
  // on to the sequence of token t, past empty ones
  __device__ __forceinline__ void next_to(const Sequences &q, int64_t t) {
    if (q.cu == nullptr) {
      ++n;
      start = end;
      end += q.seq_len;
      return;
    }
    while (n + 1 < q.num_seqs && q.cu[n + 1] <= t) ++n;
    look(q);
    good = good && t >= start && t < end;
    if (!good) {   // token by token until a sequence holds one
      start = t;
      end = t + 1;
    }
  }
};

// Row i (0 .. K - 2) of a sequence's prefix.
template <int K, typename T, typename R>
__device__ __forceinline__ void load_prev(const Params &p, int n, int i, int ch, R &r) {
  r.zero();
  if (p.x_prev)
    r.load(static_cast<const T *>(p.x_prev) + ((int64_t)n * (K - 1) + i) * p.C + ch);
}

// w[k] and the bias of four channels, in pairs (their 4 K weights lie together).
template <int K>
__device__ __forceinline__ void load_weights(const float *w_all, const float *bias_all, int ch, bool on,
                                             uint64_t (&w)[K][2], uint64_t (&bias)[2]) {
  float v[4 * K];   // [channel][tap]
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float4 f = on ? reinterpret_cast<const float4 *>(w_all + (int64_t)ch * K)[k]
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    v[4 * k] = f.x; v[4 * k + 1] = f.y; v[4 * k + 2] = f.z; v[4 * k + 3] = f.w;
  }
  const float4 b = on && bias_all ? *reinterpret_cast<const float4 *>(bias_all + ch)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][i] = pk(v[2 * i * K + k], v[(2 * i + 1) * K + k]);
  bias[0] = pk(b.x, b.y);
  bias[1] = pk(b.z, b.w);
}

// A thread's segment of tokens, counted from its first in 32 bits, and the sequence that it
// is in.
struct Segment {
  int64_t a;             // its first token
  int mine, last;        // tokens; those and the next ones that it has to look at
  int n, start, end;     // the sequence, its bounds (cut off at +-kFar)
  bool good;
  // All lanes of the warp together; false where the thread has no tokens.
  __device__ __forceinline__ bool begin(const Params &p, int64_t row, int64_t warp_row, int64_t total,
                                        int beyond, bool on) {
    const int64_t first = warp_row * p.segment;
    if (first >= total) return false;
    a = row * p.segment;
    At s;
    s.find(p.seq, first, a < total ? a : total - 1);
    if (!on || a >= total) return false;
    const int64_t b = a + p.segment < total ? a + p.segment : total;
    mine = (int)(b - a);
    last = (int)((b + beyond < total ? b + beyond : total) - a);
    set(s);
    return true;
  }
  __device__ __forceinline__ void next(const Params &p, int t) {
    At s{n, a + start, a + end, good};
    s.next_to(p.seq, a + t);
    set(s);
  }
  __device__ __forceinline__ void set(const At &s) {
    n = s.n;
    start = near(s.start);
    end = near(s.end);
    good = s.good;
  }
  __device__ __forceinline__ int near(int64_t t) const {
    t -= a;
    return (int)(t < -kFar ? -kFar : t > kFar ? kFar : t);
  }
};
// The K - 1 inputs before the segment's first token.
template <typename T, int K>
__device__ __forceinline__ void first_window(const Params &p, const Segment &s, const T *xa, int ch,
                                             uint64_t (&win)[K > 1 ? K - 1 : 1][2]) {
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int t = i - (K - 1);
    Raw4<T> r;
    r.zero();
    if (s.good && t >= s.start) r.load(xa + t * p.sx);
    else if (s.good) load_prev<K, T>(p, s.n, t - s.start + K - 1, ch, r);
    r.get(win[i]);
  }
}
// ... and those before a sequence's.
template <typename T, int K>
__device__ __forceinline__ void prefix_window(const Params &p, const Segment &s, int ch,
                                              uint64_t (&win)[K > 1 ? K - 1 : 1][2]) {
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    Raw4<T> r;
    r.zero();
    if (s.good) load_prev<K, T>(p, s.n, i, ch, r);
    r.get(win[i]);
  }
}
// z of a token, whose input then moves into the window.  Backward in scalar arithmetic, whose
// operands need not lie in pairs: 33 us where packed sums took 37, [4, 4096, 1280], bf16 (dw
// and dx in scalar arithmetic too, 35); forward 106 us packed, 108 scalar.
template <int K, bool PACKED>
__device__ __forceinline__ uint64_t sum_taps(const uint64_t (&w)[K][2], const uint64_t (&bias)[2],
                                             uint64_t (&win)[K > 1 ? K - 1 : 1][2], uint64_t v, int j) {
  if constexpr (PACKED) {
    uint64_t z = bias[j];
#pragma unroll
    for (int k = 0; k < K; ++k) z = fma2(w[k][j], k < K - 1 ? win[k][j] : v, z);
    return z;
  }
  float lo, hi, w0, w1, x0, x1;
  unpk(bias[j], lo, hi);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    unpk(w[k][j], w0, w1);
    unpk(k < K - 1 ? win[k][j] : v, x0, x1);
    lo = fmaf(w0, x0, lo);
    hi = fmaf(w1, x1, hi);
  }
  return pk(lo, hi);
}
template <int K>
__device__ __forceinline__ void move_on(uint64_t (&win)[K > 1 ? K - 1 : 1][2], uint64_t v, int j) {
#pragma unroll
  for (int k = 0; k + 1 < K - 1; ++k) win[k][j] = win[k + 1][j];
  if constexpr (K > 1) win[K - 2][j] = v;
}

template <typename T> constexpr int kFwdCtas = sizeof(T) == 2 ? 4 : 3;   // an SM

template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(kThreads, kFwdCtas<T>)
gdn_conv_fwd_kernel(const Params p) {
  constexpr int P = K - 1, PA = P ? P : 1, ST = kStages<T, false>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, tx = tid % p.lanes, ty = tid / p.lanes, per = kThreads / p.lanes;
  const int ch = (blockIdx.x * p.lanes + tx) * 4;
  const bool on = ch < p.C;
  const int64_t total = p.seq.tokens();
  const T *x = static_cast<const T *>(p.x) + ch;

  if ((int)blockIdx.y >= p.walks_y) {   // the last inputs of the sequences
    const int64_t rows = p.seq.num_seqs, step = (int64_t)(gridDim.y - p.walks_y) * per;
    for (int64_t n = (int64_t)(blockIdx.y - p.walks_y) * per + ty; n < rows; n += step) {
      int64_t start, len;
      if (!p.seq.bounds((int)n, start, len) || !p.x_tail || !on) continue;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int64_t t = len - P + i;   // in the sequence; before it: the prefix
        Raw4<T> r;
        if (t >= 0) r.load(x + (start + t) * p.sx);
        else load_prev<K, T>(p, (int)n, (int)(t + P), ch, r);
        r.store(static_cast<T *>(p.x_tail) + (n * P + i) * p.C + ch);
      }
    }
    return;
  }

  const int64_t row = (int64_t)blockIdx.y * per + ty;
  Segment s;
  if (!s.begin(p, row, row - ty + (tid & ~31) / p.lanes, total, 0, on)) return;
  const Ring<T, ST> ring{reinterpret_cast<Raw4<T> *>(smem) + tid};
  const T *xa = x + s.a * p.sx;
#pragma unroll
  for (int b = 0; b < ST - 1; ++b) {
    ring.copy(b, xa + b * kBatch * p.sx, p.sx, s.mine - b * kBatch);
    close_group();
  }
  uint64_t w[K][2], bias[2], win[PA][2];
  load_weights<K>(p.w, p.bias, ch, on, w, bias);
  first_window<T, K>(p, s, xa, ch, win);
  T *y = static_cast<T *>(p.y) + s.a * p.C + ch;
  const auto token = [&](const Raw4<T> &r) {
    uint64_t v[2], z[2];
    r.get(v);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      z[j] = sum_taps<K, true>(w, bias, win, v[j], j);
      if constexpr (SILU) z[j] = mul2(z[j], sigmoid2(z[j]));
      move_on<K>(win, v[j], j);
    }
    Raw4<T> out;
    out.set(z);
    return out;
  };
  const T *ahead = xa + (ST - 1) * kBatch * p.sx;
  for (int t0 = 0, b = 0; t0 < s.mine; t0 += kBatch, ++b) {
    ring.copy(b + ST - 1, ahead, p.sx, s.mine - t0 - (ST - 1) * kBatch);
    close_group();
    ahead += kBatch * p.sx;
    wait_groups<ST - 1>();
    if (s.good && t0 + kBatch <= s.mine && t0 + kBatch <= s.end) {   // one sequence
#pragma unroll
      for (int i = 0; i < kBatch; ++i, y += p.C) token(ring.row(b, i)).store(y);
      continue;
    }
    for (int i = 0; i < kBatch && t0 + i < s.mine; ++i, y += p.C) {
      if (t0 + i == s.end) {
        s.next(p, t0 + i);
        prefix_window<T, K>(p, s, ch, win);
      }
      const Raw4<T> out = token(ring.row(b, i));
      if (s.good) out.store(y);
    }
  }
}

// dy silu'(z), or dy; silu'(z) = s (1 + z (1 - s))
template <bool SILU>
__device__ __forceinline__ uint64_t through(uint64_t dy, uint64_t z) {
  if constexpr (!SILU) return dy;
  const uint64_t s = sigmoid2(z), one = pk(1.f, 1.f);
  return mul2(dy, mul2(s, fma2(z, fma2(s, pk(-1.f, -1.f), one), one)));
}

constexpr int kSum = 64;   // tokens that one plain sum of dw, dbias runs over

template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(kThreads, 2)
gdn_conv_bwd_kernel(const Params p) {
  constexpr int P = K - 1, PA = P ? P : 1, ST = kStages<T, true>;
  extern __shared__ __align__(16) uint8_t smem[];
  float4 *sums = reinterpret_cast<float4 *>(smem);   // [K + 1][thread]: over blocks of kSum tokens
  const int tid = threadIdx.x, tx = tid % p.lanes, ty = tid / p.lanes, per = kThreads / p.lanes;
  const int ch = (blockIdx.x * p.lanes + tx) * 4;
  const bool on = ch < p.C;
  const int64_t total = p.seq.tokens();
  const T *x = static_cast<const T *>(p.x) + ch, *dy = static_cast<const T *>(p.dy) + ch;
  let_second();
#pragma unroll
  for (int k = 0; k <= K; ++k) sums[k * kThreads + tid] = make_float4(0.f, 0.f, 0.f, 0.f);

  const int64_t row = (int64_t)blockIdx.y * per + ty;
  Segment s;
  if (s.begin(p, row, row - ty + (tid & ~31) / p.lanes, total, P, on)) {
    const Ring<T, ST> rx{reinterpret_cast<Raw4<T> *>(sums + (K + 1) * kThreads) + tid};
    const Ring<T, ST> ry{rx.at + ST * kBatch * kThreads};
    const T *xa = x + s.a * p.sx, *ya = dy + s.a * p.C;
    T *da = static_cast<T *>(p.dx) + ch + s.a * p.C;
#pragma unroll
    for (int b = 0; b < ST - 1; ++b) {
      rx.copy(b, xa + b * kBatch * p.sx, p.sx, s.last - b * kBatch);
      ry.copy(b, ya + b * kBatch * (int64_t)p.C, p.C, s.last - b * kBatch);
      close_group();
    }
    uint64_t w[K][2], bias[2], win[PA][2], acc[PA][2], own[K + 1][2];   // acc[j]: row t - 1 - j, unfinished
    load_weights<K>(p.w, p.bias, ch, on, w, bias);
    first_window<T, K>(p, s, xa, ch, win);
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i][0] = acc[i][1] = 0ull;
#pragma unroll
    for (int k = 0; k <= K; ++k) own[k][0] = own[k][1] = 0ull;
    const auto flush = [&] {
#pragma unroll
      for (int k = 0; k <= K; ++k) {
        float4 &at = sums[k * kThreads + tid];
        float v[4];
        unpk(own[k][0], v[0], v[1]);
        unpk(own[k][1], v[2], v[3]);
        at = make_float4(at.x + v[0], at.y + v[1], at.z + v[2], at.w + v[3]);
        own[k][0] = own[k][1] = 0ull;
      }
    };
    // rows t - 1 .. t - P of the sequence that ends before token t
    const auto finish = [&](int t) {
      if (!s.good) return;
#pragma unroll
      for (int m = 0; m < P; ++m) {
        const int r = t - 1 - m;
        if (r < 0 || r < s.start || r >= s.mine) continue;
        Raw4<T> out;
        if (p.d_tail) {
          uint64_t v[2];
          out.load(static_cast<const T *>(p.d_tail) + ((int64_t)s.n * P + P - 1 - m) * p.C + ch);
          out.get(v);
          acc[m][0] = add2(acc[m][0], v[0]);
          acc[m][1] = add2(acc[m][1], v[1]);
        }
        out.set(acc[m]);
        out.store(da + (int64_t)r * p.C);
      }
    };
    // the next token; returns row t - P of dx, which it finishes
    const auto token = [&](const Raw4<T> &xt, const Raw4<T> &yt, bool counts) {
      uint64_t v[2], d[2], done[2];
      xt.get(v);
      yt.get(d);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        d[j] = through<SILU>(d[j], sum_taps<K, false>(w, bias, win, v[j], j));
        if (counts) {
#pragma unroll
          for (int k = 0; k < P; ++k) own[k][j] = fma2(d[j], win[k][j], own[k][j]);
          own[P][j] = fma2(d[j], v[j], own[P][j]);
          own[K][j] = add2(own[K][j], d[j]);
        }
        done[j] = P ? fma2(w[0][j], d[j], acc[PA - 1][j]) : mul2(w[0][j], d[j]);
#pragma unroll
        for (int m = P - 1; m > 0; --m) acc[m][j] = fma2(w[P - m][j], d[j], acc[m - 1][j]);
        if (P) acc[0][j] = mul2(w[P][j], d[j]);
        move_on<K>(win, v[j], j);
      }
      Raw4<T> out;
      out.set(done);
      return out;
    };
    bool over = false;
    const T *xn = xa + (ST - 1) * kBatch * p.sx, *yn = ya + (ST - 1) * kBatch * (int64_t)p.C;
    for (int t0 = 0, b = 0; t0 < s.last && !over; t0 += kBatch, ++b) {
      const int left = s.last - t0 - (ST - 1) * kBatch;
      rx.copy(b + ST - 1, xn, p.sx, left);
      ry.copy(b + ST - 1, yn, p.C, left);
      close_group();
      xn += kBatch * p.sx;
      yn += kBatch * p.C;
      wait_groups<ST - 1>();
      if (t0 && t0 % kSum == 0) flush();
      T *to = da + (int64_t)(t0 - P) * p.C;
      if (s.good && t0 + kBatch <= s.mine && t0 + kBatch <= s.end) {   // one sequence, own tokens
        const int skip = (s.start > 0 ? s.start : 0) - (t0 - P);   // rows before that are not its own
#pragma unroll
        for (int i = 0; i < kBatch; ++i, to += p.C) {
          const Raw4<T> out = token(rx.row(b, i), ry.row(b, i), true);
          if (i >= skip) out.store(to);
        }
        continue;
      }
      for (int i = 0; i < kBatch; ++i, to += p.C) {
        const int t = t0 + i;
        if (t >= s.last) break;
        if (t == s.end) {
          finish(t);
          if (t >= s.mine) {   // what follows is another sequence's, and not this thread's
            over = true;
            break;
          }
          s.next(p, t);
          prefix_window<T, K>(p, s, ch, win);
#pragma unroll
          for (int m = 0; m < P; ++m) acc[m][0] = acc[m][1] = 0ull;
        }
        const Raw4<T> out = token(rx.row(b, i), ry.row(b, i), t < s.mine && s.good);
        if (s.good && t - P >= 0 && t - P >= s.start) out.store(to);
      }
    }
    if (!over && s.a + s.last == total && s.end == s.last) finish(s.last);
    flush();
    wait_groups<0>();
  }
  // the CTA's sums, in the order of its rows of threads
  __syncthreads();
  for (int i = tid; i < (K + 1) * p.lanes; i += kThreads) {
    const int k = i / p.lanes, l = i % p.lanes, c = (blockIdx.x * p.lanes + l) * 4;
    if (c >= p.C) continue;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < per; ++j) {
      const float4 v = sums[k * kThreads + j * p.lanes + l];
      r = make_float4(r.x + v.x, r.y + v.y, r.z + v.z, r.w + v.w);
    }
    float *at = p.part + ((int64_t)blockIdx.y * p.C + c) * (K + 1) + k;
    at[0] = r.x;
    at[K + 1] = r.y;
    at[2 * (K + 1)] = r.z;
    at[3 * (K + 1)] = r.w;
  }
}

// The sums over the CTAs (32 of the C (K + 1) a CTA), and behind them the gradient of the
// prefixes (four channels of a sequence a thread).
template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
gdn_conv_ends_kernel(const Params p, int sum_blocks) {
  constexpr int P = K - 1, PA = P ? P : 1;
  wait_first();
  if ((int)blockIdx.x < sum_blocks) {   // its eight warps share the partial sums
    __shared__ float red[kThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane, n = (int64_t)p.C * (K + 1);
    float r = 0.f;
    if (i < n)
#pragma unroll 4
      for (int k = warp; k < p.parts; k += kThreads / 32) r += p.part[k * n + i];
    red[warp][lane] = r;
    __syncthreads();
    if (warp || i >= n) return;
    r = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) r += red[w][lane];
    const int64_t c = i / (K + 1);
    const int k = (int)(i % (K + 1));
    if (k == K) {
      if (p.dbias) p.dbias[c] = r;
    } else if (p.dw) {
      p.dw[c * K + k] = r;
    }
    return;
  }
  const int64_t i = (int64_t)(blockIdx.x - sum_blocks) * kThreads + threadIdx.x, vecs = p.C / 4;
  if (i >= vecs * p.seq.num_seqs) return;
  const int n = (int)(i / vecs), ch = (int)(i % vecs) * 4;
  int64_t start, len;
  if (!p.seq.bounds(n, start, len) || !p.dx_prev) return;
  uint64_t w[K][2], bias[2], win[PA][2], g[PA][2];   // g: of the prefix's rows
  load_weights<K>(p.w, p.bias, ch, true, w, bias);
#pragma unroll
  for (int m = 0; m < P; ++m) {
    Raw4<T> r;
    load_prev<K, T>(p, n, m, ch, r);
    r.get(win[m]);
    g[m][0] = g[m][1] = 0ull;
    if (p.d_tail && m >= len) {   // with fewer tokens than that the tail begins in the prefix
      r.load(static_cast<const T *>(p.d_tail) + ((int64_t)n * P + m - len) * p.C + ch);
      r.get(g[m]);
    }
  }
#pragma unroll
  for (int t = 0; t < P; ++t) {
    if (t >= len) break;
    uint64_t v[2], e[2];
    Raw4<T> r;
    r.load(static_cast<const T *>(p.x) + (start + t) * p.sx + ch);
    r.get(v);
    r.load(static_cast<const T *>(p.dy) + (start + t) * p.C + ch);
    r.get(e);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint64_t z = bias[j];
#pragma unroll
      for (int k = 0; k < P; ++k) z = fma2(w[k][j], win[k][j], z);
      z = fma2(w[P][j], v[j], z);
      e[j] = p.silu ? through<true>(e[j], z) : e[j];
#pragma unroll
      for (int m = t; m < P; ++m) g[m][j] = fma2(w[m - t][j], e[j], g[m][j]);
#pragma unroll
      for (int k = 0; k + 1 < P; ++k) win[k][j] = win[k + 1][j];
      win[PA - 1][j] = v[j];
    }
  }
#pragma unroll
  for (int m = 0; m < P; ++m) {
    Raw4<T> r;
    r.set(g[m]);
    r.store(static_cast<T *>(p.dx_prev) + ((int64_t)n * P + m) * p.C + ch);
  }
}

// One token per sequence: a page holds the last K - 1 inputs, the oldest first.
struct StepParams {
  const void *x;
  const float *w, *bias;
  void *pool, *y;
  const int32_t *pages;
  DeviceStatus *status;
  int64_t page_stride;   // elements
  int32_t num_seqs, C, num_pages;
  bool silu;
};
template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
gdn_conv_step_kernel(const StepParams p) {
  constexpr int P = K - 1;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, vecs = p.C / 4;
  if (i >= vecs * p.num_seqs) return;
  const int n = (int)(i / vecs), ch = (int)(i % vecs) * 4;
  const int page = p.pages ? p.pages[n] : n;
  T *y = static_cast<T *>(p.y) + (int64_t)n * p.C + ch;
  if (page < 0 || page >= p.num_pages) {
    if (page != -1 && ch == 0 && p.status)
      report(p.status, GDN_ERR_DEVICE_CHECK, (uint32_t)n, 0u, 0u);
    Raw4<T> zero;
    zero.zero();
    zero.store(y);
    return;
  }
  T *at = static_cast<T *>(p.pool) + page * p.page_stride + ch;
  Raw4<T> r[K];
#pragma unroll
  for (int k = 0; k < P; ++k) r[k].load(at + (int64_t)k * p.C);
  r[P].load(static_cast<const T *>(p.x) + (int64_t)n * p.C + ch);
  uint64_t w[K][2], z[2];
  load_weights<K>(p.w, p.bias, ch, true, w, z);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    uint64_t v[2];
    r[k].get(v);
#pragma unroll
    for (int j = 0; j < 2; ++j) z[j] = fma2(w[k][j], v[j], z[j]);
  }
  if (p.silu)
#pragma unroll
    for (int j = 0; j < 2; ++j) z[j] = mul2(z[j], sigmoid2(z[j]));
  Raw4<T> out;
  out.set(z);
  out.store(y);
#pragma unroll
  for (int k = 0; k < P; ++k) r[k + 1].store(at + (int64_t)k * p.C);
}

int lanes_of(int vecs) {
  int n = 1;
  while (n < 32 && n < vecs) n *= 2;
  return n;
}
int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

// A launch over the tokens: every thread that fits on the GPU (`ctas` CTAs an SM) walks
// over one segment of at least `least_` tokens.
struct Walk {
  int64_t segment;
  int lanes, gx;
  int64_t gy;
};
Walk walk(int C, int64_t total, int ctas, int64_t least_) {
  Walk k;
  const int vecs = C / 4;
  k.lanes = lanes_of(vecs);
  k.gx = (vecs + k.lanes - 1) / k.lanes;
  const int per = kThreads / k.lanes;
  const int64_t y = ctas * kSMs / k.gx;
  const int64_t rows = (y > 1 ? y : 1) * per;   // of threads
  k.segment = ((total + rows - 1) / rows + kBatch - 1) / kBatch * kBatch;
  if (k.segment < least_) k.segment = least_;
  k.gy = ((total + k.segment - 1) / k.segment + per - 1) / per;
  return k;
}
// (Backward: a segment goes over K - 1 tokens of the next one too, and leaves a partial sum.)
Walk walk_bwd(int C, int64_t total) { return walk(C, total, 2, 16); }

template <typename T, int K, bool SILU>
cudaError_t launch_fwd_s(const Params &p, dim3 grid, cudaStream_t stream) {
  constexpr size_t kBytes = sizeof(Raw4<T>) * kStages<T, false> * kBatch * kThreads;
  const cudaError_t err = allow_smem<gdn_conv_fwd_kernel<T, K, SILU>>(kBytes);
  if (err != cudaSuccess) return err;
  gdn_conv_fwd_kernel<T, K, SILU><<<grid, kThreads, kBytes, stream>>>(p);
  return taken(cudaGetLastError());
}
template <typename T, int K>
cudaError_t launch_fwd(Params p, int64_t total, cudaStream_t stream) {
  const Walk k = walk(p.C, total, kFwdCtas<T>, 8);
  p.lanes = k.lanes;
  p.segment = k.segment;
  p.walks_y = (int32_t)k.gy;
  const int per = kThreads / k.lanes;
  const int64_t ends = p.seq.cu || (p.x_tail && K > 1)
                           ? least((p.seq.num_seqs + per - 1) / per, 64) : 0;
  const dim3 grid(k.gx, (unsigned)(k.gy + ends));
  return p.silu ? launch_fwd_s<T, K, true>(p, grid, stream) : launch_fwd_s<T, K, false>(p, grid, stream);
}
template <typename T, int K, bool SILU>
cudaError_t launch_bwd_s(const Params &p, dim3 grid, cudaStream_t stream) {
  constexpr size_t kBytes = 16 * (K + 1) * kThreads + 2 * sizeof(Raw4<T>) * kStages<T, true> * kBatch * kThreads;
  const cudaError_t err = allow_smem<gdn_conv_bwd_kernel<T, K, SILU>>(kBytes);
  if (err != cudaSuccess) return err;
  gdn_conv_bwd_kernel<T, K, SILU><<<grid, kThreads, kBytes, stream>>>(p);
  return taken(cudaGetLastError());
}
template <typename T, int K>
cudaError_t launch_bwd(Params p, int64_t total, cudaStream_t stream) {
  const Walk k = walk_bwd(p.C, total);
  p.lanes = k.lanes;
  p.segment = k.segment;
  p.parts = (int32_t)k.gy;
  const dim3 grid(k.gx, (unsigned)k.gy);
  const cudaError_t err = p.silu ? launch_bwd_s<T, K, true>(p, grid, stream)
                                 : launch_bwd_s<T, K, false>(p, grid, stream);
  if (err != cudaSuccess) return err;
  const int sums = (int)(((int64_t)p.C * (K + 1) + 31) / 32);
  const int64_t ends = p.seq.cu || (p.dx_prev && K > 1)
                           ? ((int64_t)p.C / 4 * p.seq.num_seqs + kThreads - 1) / kThreads : 0;
  return launch_beside(gdn_conv_ends_kernel<T, K>, dim3((unsigned)(sums + ends)), kThreads, 0, stream, p,
                       sums);
}
template <typename T, int K>
cudaError_t launch_step(const StepParams &p, cudaStream_t stream) {
  const int64_t n = (int64_t)p.C / 4 * p.num_seqs;
  gdn_conv_step_kernel<T, K><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(p);
  return taken(cudaGetLastError());
}

#define GDN_TAPS(call)                                    \
  (taps == 1   ? call(1)                                  \
   : taps == 2 ? call(2)                                  \
   : taps == 3 ? call(3)                                  \
               : call(4))

gdn_status check_sizes(int32_t batch, int32_t seq_len, int32_t channels, int32_t taps,
                       int32_t num_seqs, const void *cu, gdn_dtype dtype, uint32_t flags) {
  if (batch <= 0 || seq_len < 0 || channels <= 0 || taps <= 0 || num_seqs <= 0)
    return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)GDN_CONV_SILU) return GDN_ERR_INVALID_ARG;
  if (cu ? batch != 1 : num_seqs != batch) return GDN_ERR_INVALID_ARG;
  if (taps > 4 || channels % 8 || channels > (1 << 20) || num_seqs > 16384)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
cudaError_t fill(void *p, size_t n, cudaStream_t s) {
  return p && n ? taken(cudaMemsetAsync(p, 0, n, s)) : cudaSuccess;
}
// No tokens: `to` gets what `from` holds (zeros without it).
cudaError_t pass(const void *from, void *to, size_t n, cudaStream_t s) {
  if (!to || n == 0) return cudaSuccess;
  if (!from) return fill(to, n, s);
  return taken(cudaMemcpyAsync(to, from, n, cudaMemcpyDeviceToDevice, s));
}

}  // namespace
}  // namespace conv
}  // namespace gdn

extern "C" {

gdn_status gdn_conv_fwd(const void *x, const float *w, const float *bias, const void *x_prev,
                        const int32_t *cu_seqlens, void *y, void *x_tail, int32_t batch,
                        int32_t seq_len, int32_t channels, int32_t taps, int32_t num_seqs,
                        int64_t x_stride, gdn_dtype dtype, uint32_t flags, void *workspace,
                        size_t workspace_bytes, void *stream) {
  using namespace gdn;
  using namespace gdn::conv;
  const gdn_status st = check_sizes(batch, seq_len, channels, taps, num_seqs, cu_seqlens, dtype,
                                    flags);
  if (st != GDN_OK) return st;
  const size_t e = dtype == GDN_F32 ? 4 : 2, rows = (size_t)batch * seq_len;
  const size_t ends = (size_t)num_seqs * (taps - 1) * channels * e;
  const int64_t sx = row_stride(x_stride, channels, e);
  if (!sx) return GDN_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const void *ptrs[] = {x, w, bias, x_prev, cu_seqlens, y, x_tail, workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_INVALID_ARG;
  const Range outs[] = {{y, rows * channels * e}, {x_tail, ends}};
  const Range ins[] = {{x, span_bytes(rows, sx, channels, e)}, {w, (size_t)channels * taps * 4},
                       {bias, (size_t)channels * 4}, {x_prev, ends},
                       {cu_seqlens, (size_t)(num_seqs + 1) * 4}, {workspace, workspace_bytes}};
  if (seq_len == 0) {
    if (overlaps(outs[1], ins[3])) return GDN_ERR_INVALID_ARG;
    return pass(x_prev, x_tail, ends, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
  }
  if (!x || !w || !y) return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kStatusBytes) return GDN_ERR_WORKSPACE;
  if (!apart(outs, ins)) return GDN_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i)
    if (overlaps(ins[5], ins[i])) return GDN_ERR_INVALID_ARG;

  Params p{};
  p.seq = {cu_seqlens, static_cast<DeviceStatus *>(workspace), seq_len, num_seqs};
  p.x = x; p.w = w; p.bias = bias; p.x_prev = x_prev; p.y = y; p.x_tail = x_tail;
  p.sx = sx;
  p.C = channels;
  p.silu = flags & GDN_CONV_SILU;
  cudaError_t err;
#define GDN_CALL(k) \
  (dtype == GDN_F32 ? launch_fwd<float, k>(p, rows, s) : launch_fwd<__nv_bfloat16, k>(p, rows, s))
  err = GDN_TAPS(GDN_CALL);
#undef GDN_CALL
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_conv_workspace_size(int32_t num_seqs, int32_t seq_len, int32_t channels, int32_t taps) {
  using namespace gdn::conv;
  if (num_seqs <= 0 || seq_len < 0 || channels <= 0 || channels % 4 || taps <= 0) return 0;
  const int64_t dense = walk_bwd(channels, (int64_t)num_seqs * seq_len).gy;
  const int64_t packed = walk_bwd(channels, seq_len).gy, most = dense > packed ? dense : packed;
  return gdn::kStatusBytes + (size_t)most * channels * (taps + 1) * 4;
}

gdn_status gdn_conv_bwd(const void *x, const float *w, const float *bias, const void *x_prev,
                        const int32_t *cu_seqlens, const void *d_y, const void *d_x_tail, void *dx,
                        float *dw, float *dbias, void *dx_prev, int32_t batch, int32_t seq_len,
                        int32_t channels, int32_t taps, int32_t num_seqs, int64_t x_stride,
                        gdn_dtype dtype, uint32_t flags, void *workspace, size_t workspace_bytes,
                        void *stream) {
  using namespace gdn;
  using namespace gdn::conv;
  const gdn_status st = check_sizes(batch, seq_len, channels, taps, num_seqs, cu_seqlens, dtype,
                                    flags);
  if (st != GDN_OK) return st;
  const size_t e = dtype == GDN_F32 ? 4 : 2, rows = (size_t)batch * seq_len;
  const size_t ends = (size_t)num_seqs * (taps - 1) * channels * e, wide = rows * channels * e;
  const int64_t sx = row_stride(x_stride, channels, e);
  if (!sx) return GDN_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const void *ptrs[] = {x, w, bias, x_prev, cu_seqlens, d_y, d_x_tail, dx, dw, dbias, dx_prev,
                        workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_INVALID_ARG;
  const Range outs[] = {{dx, wide}, {dw, (size_t)channels * taps * 4},
                        {dbias, (size_t)channels * 4}, {dx_prev, ends}};
  const Range ins[] = {{x, span_bytes(rows, sx, channels, e)}, {w, (size_t)channels * taps * 4},
                       {bias, (size_t)channels * 4}, {x_prev, ends},
                       {cu_seqlens, (size_t)(num_seqs + 1) * 4}, {d_y, wide}, {d_x_tail, ends},
                       {workspace, workspace_bytes}};
  if (!apart(outs, ins)) return GDN_ERR_INVALID_ARG;
  if (seq_len == 0) {
    if (fill(dw, outs[1].n, s) != cudaSuccess || fill(dbias, outs[2].n, s) != cudaSuccess ||
        pass(d_x_tail, dx_prev, ends, s) != cudaSuccess)
      return GDN_ERR_CUDA;
    return GDN_OK;
  }
  if (!x || !w || !d_y || !dx) return GDN_ERR_INVALID_ARG;
  const Walk k = walk_bwd(channels, (int64_t)rows);
  if (!workspace || workspace_bytes < kStatusBytes + (size_t)k.gy * channels * (taps + 1) * 4)
    return GDN_ERR_WORKSPACE;
  for (int i = 0; i < 7; ++i)
    if (overlaps(ins[7], ins[i])) return GDN_ERR_INVALID_ARG;

  Params p{};
  p.seq = {cu_seqlens, static_cast<DeviceStatus *>(workspace), seq_len, num_seqs};
  p.x = x; p.w = w; p.bias = bias; p.x_prev = x_prev; p.dy = d_y; p.d_tail = d_x_tail;
  p.dx = dx; p.dw = dw; p.dbias = dbias; p.dx_prev = dx_prev;
  p.sx = sx;
  p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kStatusBytes);
  p.C = channels;
  p.silu = flags & GDN_CONV_SILU;
  cudaError_t err;
#define GDN_CALL(n) \
  (dtype == GDN_F32 ? launch_bwd<float, n>(p, rows, s) : launch_bwd<__nv_bfloat16, n>(p, rows, s))
  err = GDN_TAPS(GDN_CALL);
#undef GDN_CALL
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_conv_step(const void *x, const float *w, const float *bias, void *state,
                         const int32_t *pages, void *y, int32_t num_seqs, int32_t channels,
                         int32_t taps, int32_t num_pages, int64_t page_stride, gdn_dtype dtype,
                         uint32_t flags, void *workspace, size_t workspace_bytes, void *stream) {
  using namespace gdn;
  using namespace gdn::conv;
  const gdn_status st = check_sizes(num_seqs, 1, channels, taps, num_seqs, nullptr, dtype, flags);
  if (st != GDN_OK) return st;
  if (num_pages <= 0 || (!pages && num_pages < num_seqs)) return GDN_ERR_INVALID_ARG;
  const size_t e = dtype == GDN_F32 ? 4 : 2, wide = (size_t)num_seqs * channels * e;
  const int64_t page = (int64_t)(taps - 1) * channels;
  if (page_stride == 0) page_stride = page;
  if (page_stride < page || page_stride * (int64_t)e % 16) return GDN_ERR_INVALID_ARG;
  if (!x || !w || !y || (!state && taps > 1)) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {x, w, bias, state, pages, y, workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_INVALID_ARG;
  if (workspace && workspace_bytes < kStatusBytes) return GDN_ERR_WORKSPACE;
  const Range outs[] = {{y, wide},
                        {state, page ? ((size_t)(num_pages - 1) * page_stride + page) * e : 0}};
  const Range ins[] = {{x, wide}, {w, (size_t)channels * taps * 4}, {bias, (size_t)channels * 4},
                       {pages, (size_t)num_seqs * 4}, {workspace, kStatusBytes}};
  if (!apart(outs, ins)) return GDN_ERR_INVALID_ARG;
  const StepParams p{x, w, bias, state, y, pages, static_cast<DeviceStatus *>(workspace),
                     page_stride, num_seqs, channels, num_pages, (flags & GDN_CONV_SILU) != 0};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t err;
#define GDN_CALL(k) (dtype == GDN_F32 ? launch_step<float, k>(p, s) : launch_step<__nv_bfloat16, k>(p, s))
  err = GDN_TAPS(GDN_CALL);
#undef GDN_CALL
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
