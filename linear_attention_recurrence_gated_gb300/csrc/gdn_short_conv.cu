// Short causal depthwise convolution with a bias and an activation: prompts (dense rows
// or packed sequences), gradients, and single tokens on the pages of a pool.
//
//   z_t = bias + sum_{k < K} w[ch, k] x[t - (K - 1) + k],   y_t = silu(z_t) (or z_t)
//   dz = dy silu'(z),   dx_t = sum_k w[ch, k] dz[t + (K - 1) - k],
//   dw[ch, k] = sum_t dz_t x[t - (K - 1) + k],   dbias = sum_t dz_t
//
// with x before a sequence's start taken from its prefix (else zero).  Forward: a thread
// takes eight channels of a run of eight tokens, all of whose loads are under way
// together; backward: four channels of some tens of tokens, which it walks over once,
// keeping the last K - 1 inputs and the K - 1 unfinished rows of dx in registers.  Both
// are bound by HBM bandwidth.
#include "gdn_launch.cuh"
#include "gdn_layers.cuh"

namespace gdn {
namespace conv {
namespace {

using namespace layer;

constexpr int kThreads = 256;
constexpr int kRun = 8;

// Four consecutive elements: 8 bytes of bf16, 16 of fp32.
template <typename T> struct Raw4;
template <> struct Raw4<__nv_bfloat16> {
  uint2 a;
  __device__ __forceinline__ void zero() { a = make_uint2(0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint2 *>(p); }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = __uint_as_float(a.x << 16);
    v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16);
    v[3] = __uint_as_float(a.y & 0xffff0000u);
  }
};
template <> struct Raw4<float> {
  float4 a;
  __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float *p) { a = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
};
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                             *reinterpret_cast<const uint32_t *>(&b));
}

struct Params {
  Sequences seq;
  const void *x, *x_prev, *dy, *d_tail;
  const float *w, *bias;
  void *y, *x_tail, *dx, *dx_prev;
  float *dw, *dbias;
  float *part;          // [parts][C][K + 1]
  int64_t sx;           // elements from token to token of x
  int32_t C, lanes;     // lanes: threads side by side along the channels (a power of two)
  int32_t runs_y;       // grid rows that take tokens; the rest take the sequences' ends
  int32_t segment, parts;
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

template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
gdn_conv_fwd_kernel(const Params p) {
  constexpr int P = K - 1, PA = P ? P : 1;
  const int tid = threadIdx.x, tx = tid % p.lanes, ty = tid / p.lanes, per = kThreads / p.lanes;
  const int ch = (blockIdx.x * p.lanes + tx) * 8;
  const bool on = ch < p.C;
  const int64_t total = p.seq.tokens();
  const T *x = static_cast<const T *>(p.x) + ch;

  if ((int)blockIdx.y >= p.runs_y) {   // the last inputs of the sequences
    const int64_t rows = p.seq.num_seqs, step = (int64_t)(gridDim.y - p.runs_y) * per;
    for (int64_t n = (int64_t)(blockIdx.y - p.runs_y) * per + ty; n < rows; n += step) {
      int64_t start, len;
      if (!p.seq.bounds((int)n, start, len) || !p.x_tail || !on) continue;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int64_t t = len - P + i;   // in the sequence; before it: the prefix
        Raw8<T> r;
        if (t >= 0) r.load(x + (start + t) * p.sx);
        else load_prev<K, T>(p, (int)n, (int)(t + P), ch, r);
        r.store(static_cast<T *>(p.x_tail) + (n * P + i) * p.C + ch);
      }
    }
    return;
  }

  float w[K][8], bias[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][j] = on ? p.w[(int64_t)(ch + j) * K + k] : 0.f;
    bias[j] = on && p.bias ? p.bias[ch + j] : 0.f;
  }
  const int64_t runs = (total + kRun - 1) / kRun, step = (int64_t)p.runs_y * per;
  const int wrow = (tid & ~31) / p.lanes;   // the warp's first run of the CTA's
  for (int64_t base = (int64_t)blockIdx.y * per; base + wrow < runs; base += step) {
    const int64_t run = base + ty, t0 = run * kRun;
    const bool mine = on && run < runs;
    At s;
    s.find(p.seq, (base + wrow) * kRun, t0 < total ? t0 : total - 1);
    if (!mine) continue;
    Raw8<T> r[kRun + P];
#pragma unroll
    for (int i = 0; i < kRun + P; ++i) {
      const int64_t t = t0 - P + i;
      r[i].zero();
      if (t < total && (i >= P || (s.good && t >= s.start))) r[i].load(x + t * p.sx);
      else if (i < P && s.good) load_prev<K, T>(p, s.n, (int)(t - s.start) + P, ch, r[i]);
    }
    float win[PA][8];
#pragma unroll
    for (int i = 0; i < P; ++i) r[i].get(win[i]);
    T *y = static_cast<T *>(p.y) + t0 * p.C + ch;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int64_t t = t0 + i;
      if (t >= total) break;
      if (t == s.end) {
        s.next_to(p.seq, t);
#pragma unroll
        for (int m = 0; m < P; ++m) {
          Raw8<T> q;
          q.zero();
          if (s.good) load_prev<K, T>(p, s.n, m, ch, q);
          q.get(win[m]);
        }
      }
      float v[8], z[8];
      r[i + P].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[j] = bias[j];
#pragma unroll
        for (int k = 0; k < P; ++k) z[j] = fmaf(w[k][j], win[k][j], z[j]);
        z[j] = fmaf(w[P][j], v[j], z[j]);
        if (p.silu) z[j] *= sigmoid(z[j]);
      }
#pragma unroll
      for (int k = 0; k + 1 < P; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) win[k][j] = win[k + 1][j];
      if (P)
#pragma unroll
        for (int j = 0; j < 8; ++j) win[PA - 1][j] = v[j];
      if (s.good) {
        Raw8<T> out;
        out.set(z);
        out.store(y + (int64_t)i * p.C);
      }
    }
  }
}

// silu'(z) (or 1)
__device__ __forceinline__ float slope(float z, bool silu) {
  if (!silu) return 1.f;
  const float s = sigmoid(z);
  return s * fmaf(z, 1.f - s, 1.f);
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
gdn_conv_bwd_kernel(const Params p) {
  constexpr int P = K - 1, PA = P ? P : 1;
  __shared__ float red[kThreads][4];
  const int tid = threadIdx.x, tx = tid % p.lanes, ty = tid / p.lanes, per = kThreads / p.lanes;
  const int ch = (blockIdx.x * p.lanes + tx) * 4;
  const bool on = ch < p.C;
  const int64_t total = p.seq.tokens();
  const T *x = static_cast<const T *>(p.x) + ch, *dy = static_cast<const T *>(p.dy) + ch;
  T *dx = static_cast<T *>(p.dx) + ch;
  float w[K][4], bias[4], sum[K + 1][4] = {};   // sums: over all of the thread's segments
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][j] = on ? p.w[(int64_t)(ch + j) * K + k] : 0.f;
    bias[j] = on && p.bias ? p.bias[ch + j] : 0.f;
  }
  const int64_t segs = (total + p.segment - 1) / p.segment, step = (int64_t)gridDim.y * per;
  const int wrow = (tid & ~31) / p.lanes;
  for (int64_t base = (int64_t)blockIdx.y * per; base + wrow < segs; base += step) {
    const int64_t seg = base + ty, a = seg * p.segment;
    const int64_t b = a + p.segment < total ? a + p.segment : total;
    const int64_t stop = b + P < total ? b + P : total;   // tokens that reach back into a .. b - 1
    At s;
    s.find(p.seq, (base + wrow) * p.segment, a < total ? a : total - 1);
    if (!on || seg >= segs) continue;
    float win[PA][4], acc[PA][4], own[K + 1][4];   // acc[j]: row t - 1 - j, unfinished
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int64_t t = a - P + i;
      Raw4<T> r;
      r.zero();
      if (s.good && t >= s.start) r.load(x + t * p.sx);
      else if (s.good) load_prev<K, T>(p, s.n, (int)(t - s.start) + P, ch, r);
      r.get(win[i]);
    }
#pragma unroll
    for (int i = 0; i < PA; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) own[k][j] = 0.f;
    // rows t - 1 .. t - P of the sequence that ends before token t
    const auto finish = [&](int64_t t) {
      if (!s.good) return;
#pragma unroll
      for (int m = 0; m < P; ++m) {
        const int64_t row = t - 1 - m;
        if (row < a || row < s.start || row >= b) continue;
        if (p.d_tail) {
          Raw4<T> r;
          float v[4];
          r.load(static_cast<const T *>(p.d_tail) + ((int64_t)s.n * P + P - 1 - m) * p.C + ch);
          r.get(v);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][j] += v[j];
        }
        store4(dx + row * p.C, acc[m]);
      }
    };
    Raw4<T> rx[kRun], ry[kRun];
    const auto fetch = [&](int64_t t0) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        rx[i].zero();
        ry[i].zero();
        if (t0 + i < stop) {
          rx[i].load(x + (t0 + i) * p.sx);
          ry[i].load(dy + (t0 + i) * p.C);
        }
      }
    };
    fetch(a);
    bool over = false;
    for (int64_t t0 = a; t0 < stop && !over; t0 += kRun) {
      Raw4<T> cx[kRun], cy[kRun];
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        cx[i] = rx[i];
        cy[i] = ry[i];
      }
      fetch(t0 + kRun);
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int64_t t = t0 + i;
        if (t >= stop || over) break;
        if (t == s.end) {
          finish(t);
          if (t >= b) {   // what follows is another sequence's, and not this thread's
            over = true;
            break;
          }
          s.next_to(p.seq, t);
#pragma unroll
          for (int m = 0; m < P; ++m) {
            Raw4<T> q;
            q.zero();
            if (s.good) load_prev<K, T>(p, s.n, m, ch, q);
            q.get(win[m]);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][j] = 0.f;
          }
        }
        float v[4], d[4], row[4];
        cx[i].get(v);
        cy[i].get(d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float z = bias[j];
#pragma unroll
          for (int k = 0; k < P; ++k) z = fmaf(w[k][j], win[k][j], z);
          z = fmaf(w[P][j], v[j], z);
          d[j] *= slope(z, p.silu);
          if (t < b && s.good) {
#pragma unroll
            for (int k = 0; k < P; ++k) own[k][j] = fmaf(d[j], win[k][j], own[k][j]);
            own[P][j] = fmaf(d[j], v[j], own[P][j]);
            own[K][j] += d[j];
          }
          // row t - P is finished; the others move on by one
          row[j] = P ? fmaf(w[0][j], d[j], acc[PA - 1][j]) : w[0][j] * d[j];
#pragma unroll
          for (int m = P - 1; m > 0; --m) acc[m][j] = fmaf(w[P - m][j], d[j], acc[m - 1][j]);
          if (P) acc[0][j] = w[P][j] * d[j];
#pragma unroll
          for (int k = 0; k + 1 < P; ++k) win[k][j] = win[k + 1][j];
          if (P) win[PA - 1][j] = v[j];
        }
        if (s.good && t - P >= a && t - P >= s.start) store4(dx + (t - P) * p.C, row);
      }
    }
    if (!over && stop == total && s.end == total) finish(total);
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[k][j] += own[k][j];
  }
  // the CTA's sums, in the order of its rows of threads
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) red[tid][j] = sum[k][j];
    __syncthreads();
    if (ty == 0 && on)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float r = 0.f;
        for (int i = 0; i < per; ++i) r += red[i * p.lanes + tx][j];
        p.part[((int64_t)blockIdx.y * p.C + ch + j) * (K + 1) + k] = r;
      }
  }
}

// The sums over the CTAs (a thread for each of C (K + 1)), and behind them the gradient of
// the prefixes (four channels of a sequence a thread).
template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
gdn_conv_ends_kernel(const Params p, int sum_blocks) {
  constexpr int P = K - 1, PA = P ? P : 1;
  if ((int)blockIdx.x < sum_blocks) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, n = (int64_t)p.C * (K + 1);
    if (i >= n) return;
    float r = 0.f;
    for (int k = 0; k < p.parts; ++k) r += p.part[k * n + i];
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
  float win[PA][4], d[PA][4], g[PA][4];   // g: of the prefix's rows
#pragma unroll
  for (int m = 0; m < P; ++m) {
    Raw4<T> r;
    load_prev<K, T>(p, n, m, ch, r);
    r.get(win[m]);
#pragma unroll
    for (int j = 0; j < 4; ++j) g[m][j] = 0.f;
    if (p.d_tail && m >= len) {   // with fewer tokens than that the tail begins in the prefix
      r.load(static_cast<const T *>(p.d_tail) + ((int64_t)n * P + m - len) * p.C + ch);
      r.get(g[m]);
    }
  }
#pragma unroll
  for (int t = 0; t < P; ++t) {
    float v[4] = {}, e[4] = {};
    if (t < len) {
      Raw4<T> r;
      r.load(static_cast<const T *>(p.x) + (start + t) * p.sx + ch);
      r.get(v);
      r.load(static_cast<const T *>(p.dy) + (start + t) * p.C + ch);
      r.get(e);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float *w = p.w + (int64_t)(ch + j) * K;
      float z = p.bias ? p.bias[ch + j] : 0.f;
#pragma unroll
      for (int k = 0; k < P; ++k) z = fmaf(w[k], win[k][j], z);
      z = fmaf(w[P], v[j], z);
      d[t][j] = t < len ? e[j] * slope(z, p.silu) : 0.f;
#pragma unroll
      for (int m = 0; m < P; ++m)
        if (m >= t) g[m][j] = fmaf(w[m - t], d[t][j], g[m][j]);
#pragma unroll
      for (int k = 0; k + 1 < P; ++k) win[k][j] = win[k + 1][j];
      win[PA - 1][j] = v[j];
    }
  }
#pragma unroll
  for (int m = 0; m < P; ++m)
    store4(static_cast<T *>(p.dx_prev) + ((int64_t)n * P + m) * p.C + ch, g[m]);
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
    const float zero[4] = {};
    store4(y, zero);
    return;
  }
  T *at = static_cast<T *>(p.pool) + page * p.page_stride + ch;
  float win[K][4];
  Raw4<T> r[K];
#pragma unroll
  for (int k = 0; k < P; ++k) r[k].load(at + (int64_t)k * p.C);
  r[P].load(static_cast<const T *>(p.x) + (int64_t)n * p.C + ch);
#pragma unroll
  for (int k = 0; k < K; ++k) r[k].get(win[k]);
  float z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float *w = p.w + (int64_t)(ch + j) * K;
    z[j] = p.bias ? p.bias[ch + j] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) z[j] = fmaf(w[k], win[k][j], z[j]);
    if (p.silu) z[j] *= sigmoid(z[j]);
  }
  store4(y, z);
#pragma unroll
  for (int k = 0; k < P; ++k) store4(at + (int64_t)k * p.C, win[k + 1]);
}

int lanes_of(int vecs) {
  int n = 1;
  while (n < 32 && n < vecs) n *= 2;
  return n;
}
int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

template <typename T, int K>
cudaError_t launch_fwd(Params p, int64_t total, cudaStream_t stream) {
  const int vecs = p.C / 8;
  p.lanes = lanes_of(vecs);
  const int per = kThreads / p.lanes, gx = (vecs + p.lanes - 1) / p.lanes;
  const int64_t runs = (total + kRun - 1) / kRun;
  // CTAs that fit at a time (registers), each going over several runs of tokens
  const int64_t most = (3 * kSMs + gx - 1) / gx;
  p.runs_y = (int32_t)least((runs + per - 1) / per, most);
  const int64_t ends = p.seq.cu || (p.x_tail && K > 1)
                           ? least((p.seq.num_seqs + per - 1) / per, 64) : 0;
  gdn_conv_fwd_kernel<T, K><<<dim3(gx, (unsigned)(p.runs_y + ends)), kThreads, 0, stream>>>(p);
  return taken(cudaGetLastError());
}
// Tokens that a thread of the backward pass walks over, and the CTAs along them: long
// segments read few rows twice, short ones fill the GPU.
struct Walk {
  int segment, lanes, gx;
  int64_t gy;
};
Walk walk(int C, int64_t total) {
  Walk k;
  const int vecs = C / 4;
  k.lanes = lanes_of(vecs);
  k.gx = (vecs + k.lanes - 1) / k.lanes;
  const int per = kThreads / k.lanes;
  k.segment = 64;
  const int64_t want = 2 * kSMs;
  while (k.segment > 8 && k.gx * ((total + k.segment * per - 1) / (k.segment * per)) < want)
    k.segment /= 2;
  const int64_t segs = (total + k.segment - 1) / k.segment;
  k.gy = least((segs + per - 1) / per, (4 * kSMs + k.gx - 1) / k.gx);
  return k;
}
template <typename T, int K>
cudaError_t launch_bwd(Params p, int64_t total, cudaStream_t stream) {
  const Walk k = walk(p.C, total);
  p.lanes = k.lanes;
  p.segment = k.segment;
  p.parts = (int32_t)k.gy;
  gdn_conv_bwd_kernel<T, K><<<dim3(k.gx, (unsigned)k.gy), kThreads, 0, stream>>>(p);
  const cudaError_t err = taken(cudaGetLastError());
  if (err != cudaSuccess) return err;
  const int sums = (int)(((int64_t)p.C * (K + 1) + kThreads - 1) / kThreads);
  const int64_t ends = p.seq.cu || (p.dx_prev && K > 1)
                           ? ((int64_t)p.C / 4 * p.seq.num_seqs + kThreads - 1) / kThreads : 0;
  gdn_conv_ends_kernel<T, K><<<(unsigned)(sums + ends), kThreads, 0, stream>>>(p, sums);
  return taken(cudaGetLastError());
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
  const int64_t dense = walk(channels, (int64_t)num_seqs * seq_len).gy;
  const int64_t packed = walk(channels, seq_len).gy, most = dense > packed ? dense : packed;
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
  const Walk k = walk(channels, (int64_t)rows);
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
