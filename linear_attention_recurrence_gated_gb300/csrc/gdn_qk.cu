// Norm of each head of q and k, then the rotation of its first R elements by the token's
// position, and the gradients.  With x one head of a token (D elements), s = q_scale for
// q and 1 for k:
//
//   r = 1 / sqrt(mean(x^2) + eps)  (l2: sum in place of mean),   u = s r x w
//   out = u, pairs (a, b) of its first R elements turned by phi = position inv_freq[i]:
//         (a cos phi - b sin phi, a sin phi + b cos phi)
//   backward: du = s (pairs turned back), dw = sum du x r, g = du w,
//             dx = r (g - x r^2 mean(x g))
//
// Bound by HBM bandwidth: every element is read and written once.  A head takes D / 16
// lanes with sixteen elements each: two runs of eight columns, whose pairs of the rotation
// are both in the thread (columns 8 v and R / 2 + 8 v for pairs R / 2 apart), so that
// packed arithmetic turns them without exchanges between lanes; where R / 2 is not a
// multiple of eight a row goes through shared memory.  The cosines and sines of a token
// are computed once, in shared memory, for all of its heads: forward of q and k in turn
// ([8, 4096, 16 + 16, 64], bf16: 49 us, 5.5 TB/s; with CTAs of their own for q and for k, 55:
// the table was a third of their instructions), backward, where a thread's sums for the
// weight are of one of the two, of q or of k.  An angle's whole turns are taken off exactly:
// inv_freq / 2 pi is held as a fraction of 2^64, whose product with the position drops them
// by overflowing.
#include "gdn_launch.cuh"
#include "gdn_layers.cuh"

namespace gdn {
namespace qk {
namespace {

using namespace layer;

constexpr int kThreads = 256;
// CTAs an SM.  (bf16 forward, [8, 4096, 16 + 16, 64]: 49 us, 53 with three, 59 with six.)
template <typename T, bool BACK> constexpr int kCtas = BACK ? 2 : sizeof(T) == 2 ? 4 : 3;
// Most tokens of a CTA at a time.  (Forward as above, with 4, 6, 12: 51, 59, 49 us; backward,
// [4, 8192, 16 + 16, 128], 151, with them 168, 158, 149, and fp32, [4, 4096, 32 + 8, 64], 104,
// with them 142, 115, 109.)
constexpr int kTokens = 8;
constexpr int kMaxHalf = 128;  // most pairs of a head

// q, or k.
struct Side {
  const void *x, *g;      // rows; gradients of the outputs (densely packed)
  void *out;              // densely packed
  const float *w;
  float *dw;
  int64_t stride;
  int32_t heads, ctas;    // backward: CTAs that take this side; forward: all, of the first
  float scale;
  uint32_t magic;         // 2^32 / heads, rounded up: rows of a tile < 2^16
};
struct Params {
  Side side[2];
  const float *inv_freq;
  const int32_t *positions;
  float *part;
  int64_t tokens, seq_len;
  int32_t D, R, pitch, tile;   // pitch: R / 2 rounded up to 4
  float eps;
  bool l2, interleaved;
};

// cos and sin of r, |r| <= pi / 4, by the polynomials that minimise the largest error
// (2e-9 and 4e-10 there, far below the rounding of an fp32 result).
__device__ __forceinline__ void cos_sin(float r, float &c, float &s) {
  const float q = r * r;
  s = fmaf(fmaf(fmaf(-0.00019495601009111851f, q, 0.00833197869360447f), q, -0.16666650772094727f), q * r, r);
  c = fmaf(fmaf(fmaf(fmaf(2.4390410544583574e-05f, q, -0.0013886763481423259f), q, 0.04166662320494652f), q, -0.5f), q, 1.f);
}
// Cosines and sines of positions x inv_freq for the tile's tokens: [token][2][pitch].
__device__ __forceinline__ void turn_table(const Params &p, int64_t tok0, int cnt, int lanes,
                                           const uint64_t *freq, const float *unit,
                                           float *table) {
  const int half = p.R / 2;   // lanes: the power of two that holds it, at most 256
  for (int t = threadIdx.x / lanes; t < cnt; t += kThreads / lanes) {
    const int f = threadIdx.x & (lanes - 1);
    if (f >= half) break;
    const int64_t tok = tok0 + t;
    const int64_t pos = p.positions ? (int64_t)p.positions[tok] : tok % p.seq_len;
    // of 2^32; whole turns overflow
    const uint32_t turns = (uint32_t)(((uint64_t)pos * freq[f]) >> 32);
    // to the nearest quarter turn, whose cosine and sine are exact, and the rest
    const uint32_t quarter = (turns + (1u << 29)) >> 30;   // (0 .. 4, 4 being none)
    const int32_t rest = (int32_t)(turns - (quarter << 30));
    float c, s;
    cos_sin((float)rest * unit[f], c, s);
    const float a = quarter & 1 ? -s : c, b = quarter & 1 ? c : s;
    float *at = table + t * 2 * p.pitch + f;
    at[0] = quarter & 2 ? -a : a;
    at[p.pitch] = quarter & 2 ? -b : b;
  }
}
// The frequencies as fractions of a turn, whole turns left out, and the angle of 2^-32 of
// one: NaN for a frequency that is not finite, so that its cosines and sines are.
__device__ __forceinline__ void load_freq(const Params &p, uint64_t *freq, float *unit) {
  for (int i = threadIdx.x; i < p.R / 2; i += kThreads) {
    const double t = (double)p.inv_freq[i] * 0.15915494309189533577;   // / (2 pi)
    const double f = t - floor(t);
    freq[i] = f < 1.0 ? (uint64_t)(f * 0x1p53) << 11 : 0ull;
    unit[i] = f == f ? 1.4629180792671596e-9f : __int_as_float(0x7fffffff);   // 2 pi / 2^32
  }
}

template <int LR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < LR; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// How the pairs lie: R / 2 apart with R / 2 a multiple of eight, neighbours, or otherwise
// (no rotation at all, too).
enum Mode { kApart, kNext, kOther };

// A thread's columns: c[0] .. c[0] + 7 and c[1] .. c[1] + 7, where on[].
struct Cols {
  int c[2];
  bool on[2];
  bool split;    // pairs (c[0] + i, c[1] + i)
};
template <Mode M>
__device__ __forceinline__ Cols cols_of(const Params &p, int v) {
  if (M == kApart && 16 * v < p.R) return {{8 * v, p.R / 2 + 8 * v}, {true, true}, true};
  return {{16 * v, 16 * v + 8}, {16 * v < p.D, 16 * v + 8 < p.D}, false};
}
__device__ __forceinline__ void load_pairs(const float *at, uint64_t (&v)[4]) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(at)[0];
  const ulonglong2 b = reinterpret_cast<const ulonglong2 *>(at)[1];
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
// The thread's pairs turned by the token's angles cs (BACK: the other way).  All lanes of
// the warp together.
template <Mode M, bool BACK>
__device__ __forceinline__ void turn(const Params &p, const Cols &col, const float *cs, float *row,
                                     uint64_t (&u)[2][4]) {
  constexpr float sign = BACK ? -1.f : 1.f;
  const int half = p.R / 2;
  if constexpr (M == kNext) {   // a column and its neighbour
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (col.c[g] >= p.R) continue;
      const float4 x = *reinterpret_cast<const float4 *>(cs + col.c[g] / 2);
      const float4 y = *reinterpret_cast<const float4 *>(cs + p.pitch + col.c[g] / 2);
      const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (col.c[g] + 2 * m >= p.R) continue;
        float a, b;
        unpk(u[g][m], a, b);
        const float s = sign * ys[m];
        u[g][m] = pk(fmaf(a, xs[m], -(b * s)), fmaf(a, s, b * xs[m]));
      }
    }
  } else if constexpr (M == kApart) {
    if (!col.split) return;
    uint64_t x[4], y[4];
    load_pairs(cs + col.c[0], x);
    load_pairs(cs + p.pitch + col.c[0], y);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint64_t a = u[0][m], b = u[1][m], neg = mul2(y[m], pk(-1.f, -1.f));
      u[0][m] = fma2(b, BACK ? y[m] : neg, mul2(a, x[m]));
      u[1][m] = fma2(a, BACK ? neg : y[m], mul2(b, x[m]));
    }
  } else {
    if (p.R == 0) return;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      ulonglong2 *at = reinterpret_cast<ulonglong2 *>(row + col.c[g]);
      at[0] = make_ulonglong2(u[g][0], u[g][1]);
      at[1] = make_ulonglong2(u[g][2], u[g][3]);
    }
    __syncwarp();
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float w[2];
        unpk(u[g][m], w[0], w[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = col.c[g] + 2 * m + j;
          if (i >= p.R) continue;
          const bool low = i < half;
          const float o = row[low ? i + half : i - half];
          const float x = cs[low ? i : i - half], s = sign * cs[p.pitch + (low ? i : i - half)];
          w[j] = low ? fmaf(w[j], x, -(o * s)) : fmaf(o, s, w[j] * x);
        }
        u[g][m] = pk(w[0], w[1]);
      }
    __syncwarp();
  }
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw8<T> &r, uint64_t (&u)[4]) {
  float v[8];
  r.get(v);
#pragma unroll
  for (int m = 0; m < 4; ++m) u[m] = pk(v[2 * m], v[2 * m + 1]);
}

template <typename T, int LR, Mode M, bool BACK>
__global__ void __launch_bounds__(kThreads, kCtas<T, BACK>)
gdn_qk_norm_kernel(const Params p) {
  constexpr int RG = kThreads / LR;   // rows side by side
  __shared__ __align__(16) float tables[2][kTokens * 2 * kMaxHalf];   // of a tile and the next
  __shared__ __align__(16) float rows_buf[RG * LR * 16];
  __shared__ uint64_t freq[kMaxHalf];
  __shared__ float unit[kMaxHalf];
  __shared__ __align__(16) float weights[BACK ? 1 : 2][LR * 16];   // times q's scale
  const int tid = threadIdx.x, rg = tid / LR;
  // the sides that this CTA takes
  const int side0 = BACK && (int)blockIdx.x >= p.side[0].ctas, side1 = BACK ? side0 : 1;
  const Cols col = cols_of<M>(p, tid % LR);
  // (lanes without columns read the first ones, and store nothing)
  const int c0 = col.on[0] ? col.c[0] : 0, c1 = col.on[1] ? col.c[1] : 0;
  float *buf = rows_buf + rg * LR * 16;
  if (BACK) let_second();
  uint64_t w[2][4], own[2][4] = {}, all[2][4] = {};   // own, all: sums for the weight
  if constexpr (BACK) {
    const Side &s = p.side[side0];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int c = (g ? c1 : c0) + 2 * m;
        w[g][m] = s.w ? pk(s.w[c], s.w[c + 1]) : pk(1.f, 1.f);
        w[g][m] = mul2(w[g][m], pk(s.scale, s.scale));
      }
  } else {
    for (int i = tid; i < 2 * LR * 16; i += kThreads) {
      const Side &s = p.side[i / (LR * 16)];
      const int c = i % (LR * 16);
      weights[i / (LR * 16)][c] = s.w && c < p.D ? s.w[c] * s.scale : s.scale;
    }
  }
  int lanes = 32;
  if (p.R) {
    load_freq(p, freq, unit);
    while (lanes < p.R / 2) lanes *= 2;
  }
  const float over = p.l2 ? 1.f : 1.f / (float)p.D;
  const int64_t tiles = (p.tokens + p.tile - 1) / p.tile;
  const int ctas = p.side[side0].ctas;
  int summed = 0, which_table = 0;
  __syncthreads();
  for (int64_t tile = blockIdx.x - (side0 ? p.side[0].ctas : 0); tile < tiles; tile += ctas) {
    const int64_t tok0 = tile * p.tile;
    const int cnt = (int)(p.tokens - tok0 < p.tile ? p.tokens - tok0 : p.tile);
    Raw8<T> x[2], d[BACK ? 2 : 1];
    int tok, at, rows;
    const auto fetch = [&](int side, int r) {   // (rows behind the last: the last)
      const Side &s = p.side[side];
      rows = cnt * s.heads;
      r = r < rows ? r : rows - 1;
      tok = s.heads == 1 ? r : (int)__umulhi((uint32_t)r, s.magic);
      const int head = (r - tok * s.heads) * p.D;
      at = tok * s.heads * p.D + head;
      const T *from = static_cast<const T *>(s.x) + tok0 * s.stride + tok * s.stride + head;
      x[0].load(from + c0);
      x[1].load(from + c1);
      if constexpr (BACK) {
        const T *g = static_cast<const T *>(s.g) + tok0 * (s.heads * p.D) + at;
        d[0].load(g + c0);
        d[1].load(g + c1);
      }
    };
    fetch(side0, rg);   // on its way while the table is made
    // (a table is made again two tiles later: every thread has passed a barrier after reading it)
    which_table ^= 1;
    float *table = tables[which_table];
    if (p.R) {
      turn_table(p, tok0, cnt, lanes, freq, unit, table);
      __syncthreads();
    }
    int side = side0, base = 0;
    while (side <= side1) {
      const Side &s = p.side[side];
      const bool on = base + rg < rows;
      const float *cs = table + tok * 2 * p.pitch;
      T *to = static_cast<T *>(s.out) + tok0 * (s.heads * p.D) + at;
      const float *ws = weights[BACK ? 0 : side];
      uint64_t xv[2][4], u[2][4], ss = 0ull;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        unpack(x[g], xv[g]);
        if (LR * 16 != p.D && !col.on[g]) xv[g][0] = xv[g][1] = xv[g][2] = xv[g][3] = 0ull;
#pragma unroll
        for (int m = 0; m < 4; ++m) ss = fma2(xv[g][m], xv[g][m], ss);
        if constexpr (BACK) unpack(d[g], u[g]);
      }
      base += RG;
      if (base >= rows) {
        base = 0;
        ++side;
      }
      if (side <= side1) fetch(side, base + rg);
      float lo, hi;
      unpk(ss, lo, hi);
      const float r = rsqrtf(fmaf(row_sum<LR>(lo + hi), over, p.eps));
      const uint64_t rr = pk(r, r);
      if constexpr (!BACK) {
        load_pairs(ws + c0, w[0]);
        load_pairs(ws + c1, w[1]);
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int m = 0; m < 4; ++m) u[g][m] = mul2(mul2(xv[g][m], rr), w[g][m]);
        turn<M, BACK>(p, col, cs, buf, u);
      } else {
        turn<M, BACK>(p, col, cs, buf, u);
        uint64_t m2 = 0ull;
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint64_t t = mul2(u[g][m], xv[g][m]);
            if (on) own[g][m] = fma2(t, rr, own[g][m]);
            m2 = fma2(t, w[g][m], m2);
          }
        unpk(m2, lo, hi);
        const float f = -(row_sum<LR>(lo + hi) * over * r * r);
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int m = 0; m < 4; ++m)
            u[g][m] = mul2(rr, fma2(xv[g][m], pk(f, f), mul2(u[g][m], w[g][m])));
      }
      if (on)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float v[8];
#pragma unroll
          for (int m = 0; m < 4; ++m) unpk(u[g][m], v[2 * m], v[2 * m + 1]);
          Raw8<T> o;
          o.set(v);
          if (col.on[g]) o.store(to + (g ? c1 : c0));
        }
      if (BACK && ++summed == 64) {   // at most 64 rows in one run of an accumulator
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            all[g][m] = add2(all[g][m], own[g][m]);
            own[g][m] = 0ull;
          }
        summed = 0;
      }
    }
  }
  if constexpr (BACK) {   // the CTA's sums, in the order of its rows of threads
    __syncthreads();
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int m = 0; m < 4; ++m)   // (du carries q's scale)
        *reinterpret_cast<uint64_t *>(buf + col.c[g] + 2 * m) =
            mul2(add2(all[g][m], own[g][m]), pk(p.side[side0].scale, p.side[side0].scale));
    __syncthreads();
    for (int c = tid; c < p.D; c += kThreads) {
      float sum = 0.f;
      for (int i = 0; i < RG; ++i) sum += rows_buf[i * LR * 16 + c];
      p.part[(int64_t)blockIdx.x * p.D + c] = sum;
    }
  }
}

// The weights' gradients: 32 columns of q's or k's a CTA, its 32 warps over the partial sums.
__global__ void __launch_bounds__(1024) gdn_qk_weights_kernel(const Params p) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const Side &s = p.side[blockIdx.y];
  wait_first();
  float sum = 0.f;
  if (c < p.D) {
    const float *part = p.part + (blockIdx.y ? (int64_t)p.side[0].ctas * p.D : 0) + c;
#pragma unroll 4
    for (int i = warp; i < s.ctas; i += 32) sum += part[(int64_t)i * p.D];
  }
  red[warp][lane] = sum;
  __syncthreads();
  if (warp) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += red[i][lane];
  if (c < p.D && s.dw) s.dw[c] = sum;
}

// Tokens of a tile (one where there are few) and CTAs, those that fit on the GPU; backward in
// proportion to the heads.
struct Grid {
  int tile;
  int64_t ctas[2];
};
Grid grid_of(int64_t tokens, int64_t Hq, int64_t Hk, int ctas, bool back) {
  Grid g;
  const int64_t fit = ctas * kSMs;
  g.tile = tokens >= 2 * kTokens * kSMs ? kTokens : 1;
  const int64_t tiles = (tokens + g.tile - 1) / g.tile;
  int64_t q = fit * Hq / (Hq + Hk);
  q = !back ? fit : q < 1 ? 1 : q > fit - 1 ? fit - 1 : q;
  const int64_t k = fit - q;
  g.ctas[0] = q < tiles ? q : tiles;
  g.ctas[1] = k < tiles ? k : tiles;
  return g;
}

template <typename T, Mode M, bool BACK>
cudaError_t launch_m(const Params &p, cudaStream_t stream) {
  const unsigned n = (unsigned)(p.side[0].ctas + p.side[1].ctas);
  if (p.D <= 64) gdn_qk_norm_kernel<T, 4, M, BACK><<<n, kThreads, 0, stream>>>(p);
  else if (p.D <= 128) gdn_qk_norm_kernel<T, 8, M, BACK><<<n, kThreads, 0, stream>>>(p);
  else gdn_qk_norm_kernel<T, 16, M, BACK><<<n, kThreads, 0, stream>>>(p);
  return taken(cudaGetLastError());
}
template <typename T, bool BACK>
cudaError_t launch_t(const Params &p, cudaStream_t stream) {
  if (p.R && p.interleaved) return launch_m<T, kNext, BACK>(p, stream);
  if (p.R && p.R % 16 == 0) return launch_m<T, kApart, BACK>(p, stream);
  return launch_m<T, kOther, BACK>(p, stream);
}

gdn_status check_sizes(int32_t batch, int32_t seq_len, int32_t Hq, int32_t Hk, int32_t D, int32_t R,
                       gdn_dtype dtype, uint32_t flags) {
  if (batch <= 0 || seq_len < 0 || Hq <= 0 || Hk <= 0 || D <= 0 || R < 0 || R > D || R % 2)
    return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)(GDN_QK_L2NORM | GDN_ROPE_INTERLEAVED)) return GDN_ERR_INVALID_ARG;
  if (D > 256 || D % 8 || Hq > 4096 || Hk > 4096) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

}  // namespace
}  // namespace qk
}  // namespace gdn

extern "C" {

gdn_status gdn_qk_norm(const void *q, const void *k, const float *q_weight, const float *k_weight,
                       const int32_t *positions, const float *inv_freq, void *q_out, void *k_out,
                       int32_t batch, int32_t seq_len, int32_t q_heads, int32_t k_heads,
                       int32_t head_dim, int32_t rotary_dim, int64_t q_stride, int64_t k_stride,
                       float q_scale, float eps, gdn_dtype dtype, uint32_t flags, void *stream) {
  using namespace gdn;
  using namespace gdn::qk;
  const gdn_status st = check_sizes(batch, seq_len, q_heads, k_heads, head_dim, rotary_dim, dtype,
                                    flags);
  if (st != GDN_OK) return st;
  if (seq_len == 0) return GDN_OK;
  const size_t e = dtype == GDN_F32 ? 4 : 2, rows = (size_t)batch * seq_len;
  const int64_t wq = (int64_t)q_heads * head_dim, wk = (int64_t)k_heads * head_dim;
  const int64_t sq = row_stride(q_stride, wq, e), sk = row_stride(k_stride, wk, e);
  if (!sq || !sk) return GDN_ERR_INVALID_ARG;
  if (!q || !k || !q_out || !k_out || (rotary_dim && !inv_freq)) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out};
  if (!all_aligned(ptrs)) return GDN_ERR_INVALID_ARG;
  const Range outs[] = {{q_out, rows * wq * e}, {k_out, rows * wk * e}};
  const Range ins[] = {{q, span_bytes(rows, sq, wq, e)}, {k, span_bytes(rows, sk, wk, e)},
                       {q_weight, (size_t)head_dim * 4}, {k_weight, (size_t)head_dim * 4},
                       {positions, rows * 4}, {inv_freq, (size_t)rotary_dim * 2}};
  if (!apart(outs, ins)) return GDN_ERR_INVALID_ARG;
  Params p{};
  const Grid g = grid_of((int64_t)rows, q_heads, k_heads,
                         dtype == GDN_F32 ? kCtas<float, false> : kCtas<__nv_bfloat16, false>, false);
  p.side[0] = {q, nullptr, q_out, q_weight, nullptr, sq, q_heads, (int32_t)g.ctas[0], q_scale,
               0xffffffffu / q_heads + 1};
  p.side[1] = {k, nullptr, k_out, k_weight, nullptr, sk, k_heads, (int32_t)g.ctas[1], 1.f,
               0xffffffffu / k_heads + 1};
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.tokens = (int64_t)rows;
  p.seq_len = seq_len;
  p.D = head_dim; p.R = rotary_dim;
  p.pitch = (rotary_dim / 2 + 3) / 4 * 4;
  p.eps = eps;
  p.l2 = flags & GDN_QK_L2NORM;
  p.interleaved = flags & GDN_ROPE_INTERLEAVED;
  p.tile = g.tile;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t err = dtype == GDN_F32 ? launch_t<float, false>(p, s)
                                           : launch_t<__nv_bfloat16, false>(p, s);
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_qk_norm_workspace_size(int32_t batch, int32_t seq_len, int32_t head_dim) {
  if (batch <= 0 || seq_len < 0 || head_dim <= 0) return 0;
  // (of every number of heads; calls without tokens need none)
  const int64_t tokens = (int64_t)batch * seq_len, most = gdn::qk::kCtas<float, true> * gdn::layer::kSMs;
  return (size_t)(tokens < most ? 2 * tokens < most ? 2 * tokens : most : most) * head_dim * 4;
}

gdn_status gdn_qk_norm_bwd(const void *q, const void *k, const float *q_weight,
                           const float *k_weight, const int32_t *positions, const float *inv_freq,
                           const void *d_q_out, const void *d_k_out, void *dq, void *dk,
                           float *dq_weight, float *dk_weight, int32_t batch, int32_t seq_len,
                           int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t rotary_dim,
                           int64_t q_stride, int64_t k_stride, float q_scale, float eps,
                           gdn_dtype dtype, uint32_t flags, void *workspace,
                           size_t workspace_bytes, void *stream) {
  using namespace gdn;
  using namespace gdn::qk;
  const gdn_status st = check_sizes(batch, seq_len, q_heads, k_heads, head_dim, rotary_dim, dtype,
                                    flags);
  if (st != GDN_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const size_t w_bytes = (size_t)head_dim * 4;
  if (seq_len == 0) {
    for (float *w : {dq_weight, dk_weight})
      if (w && taken(cudaMemsetAsync(w, 0, w_bytes, s)) != cudaSuccess) return GDN_ERR_CUDA;
    return GDN_OK;
  }
  const size_t e = dtype == GDN_F32 ? 4 : 2, rows = (size_t)batch * seq_len;
  const int64_t wq = (int64_t)q_heads * head_dim, wk = (int64_t)k_heads * head_dim;
  const int64_t sq = row_stride(q_stride, wq, e), sk = row_stride(k_stride, wk, e);
  if (!sq || !sk) return GDN_ERR_INVALID_ARG;
  if (!q || !k || !d_q_out || !d_k_out || !dq || !dk || (rotary_dim && !inv_freq))
    return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {q, k, q_weight, k_weight, positions, inv_freq, d_q_out, d_k_out, dq, dk,
                        dq_weight, dk_weight, workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_INVALID_ARG;
  const Grid g = grid_of((int64_t)rows, q_heads, k_heads, kCtas<float, true>, true);
  const bool sums = dq_weight || dk_weight;
  if (!workspace || workspace_bytes < (size_t)(g.ctas[0] + g.ctas[1]) * w_bytes) return GDN_ERR_WORKSPACE;
  const Range outs[] = {{dq, rows * wq * e}, {dk, rows * wk * e}, {dq_weight, w_bytes},
                        {dk_weight, w_bytes}};
  const Range ins[] = {{workspace, workspace_bytes},
                       {q, span_bytes(rows, sq, wq, e)}, {k, span_bytes(rows, sk, wk, e)},
                       {q_weight, w_bytes}, {k_weight, w_bytes}, {positions, rows * 4},
                       {inv_freq, (size_t)rotary_dim * 2}, {d_q_out, rows * wq * e},
                       {d_k_out, rows * wk * e}};
  if (!apart(outs, ins)) return GDN_ERR_INVALID_ARG;
  for (int i = 1; i < 9; ++i)
    if (overlaps(ins[0], ins[i])) return GDN_ERR_INVALID_ARG;
  Params p{};
  p.side[0] = {q, d_q_out, dq, q_weight, dq_weight, sq, q_heads, (int32_t)g.ctas[0], q_scale,
               0xffffffffu / q_heads + 1};
  p.side[1] = {k, d_k_out, dk, k_weight, dk_weight, sk, k_heads, (int32_t)g.ctas[1], 1.f,
               0xffffffffu / k_heads + 1};
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.part = static_cast<float *>(workspace);
  p.tokens = (int64_t)rows;
  p.seq_len = seq_len;
  p.D = head_dim; p.R = rotary_dim;
  p.pitch = (rotary_dim / 2 + 3) / 4 * 4;
  p.eps = eps;
  p.l2 = flags & GDN_QK_L2NORM;
  p.interleaved = flags & GDN_ROPE_INTERLEAVED;
  p.tile = g.tile;
  cudaError_t err = dtype == GDN_F32 ? launch_t<float, true>(p, s) : launch_t<__nv_bfloat16, true>(p, s);
  if (err == cudaSuccess && sums)
    err = launch_beside(gdn_qk_weights_kernel, dim3((head_dim + 31) / 32, 2), 1024, 0, s, p);
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
