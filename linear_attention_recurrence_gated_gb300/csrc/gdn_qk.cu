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
// Bound by HBM bandwidth: every element is read and written once.  A head takes D / 8
// lanes with eight elements each, four rows of a thread are on their way together; the
// cosines and sines of a token are computed once, in shared memory, for all of its heads.
// An angle's whole turns are taken off exactly: inv_freq / 2 pi is held as a fraction of
// 2^64, whose product with the position drops them by overflowing.
#include "gdn_launch.cuh"
#include "gdn_layers.cuh"

namespace gdn {
namespace qk {
namespace {

using namespace layer;

constexpr int kThreads = 256;
constexpr int kRows = 4;       // rows of a thread that are loaded together
constexpr int kTokens = 8;     // most tokens of a CTA at a time
constexpr int kMaxHalf = 128;  // most pairs of a head

struct Params {
  const void *q, *k, *dq_in, *dk_in;
  const float *wq, *wk, *inv_freq;
  const int32_t *positions;
  void *oq, *ok;          // outputs, or dq and dk
  float *part, *dwq, *dwk;
  int64_t sq, sk, tokens, seq_len;
  int32_t Hq, Hk, D, R, tile, parts;
  float eps, scale;
  bool l2, interleaved;
};

// cos and sin of positions x inv_freq for the tile's tokens, [token][R / 2].
__device__ __forceinline__ void turn_table(const Params &p, int64_t tok0, int cnt,
                                           const uint64_t *freq, float2 *table) {
  const int half = p.R / 2;
  for (int i = threadIdx.x; i < cnt * half; i += kThreads) {
    const int64_t tok = tok0 + i / half;
    const int64_t pos = p.positions ? (int64_t)p.positions[tok] : tok % p.seq_len;
    const uint64_t turns = (uint64_t)pos * freq[i % half];   // of 2^64; whole turns overflow
    // to the nearest quarter turn, whose cosine and sine are exact, and the rest
    const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62) & 3u;
    const int64_t rest = (int64_t)(turns - ((uint64_t)quarter << 62));
    float c, s;
    sincospif((float)rest * 0x1p-63f, &s, &c);   // half turns
    const float a = quarter & 1 ? -s : c, b = quarter & 1 ? c : s;
    table[i] = quarter & 2 ? make_float2(-a, -b) : make_float2(a, b);
  }
}
// The frequencies as fractions of a turn, whole turns left out.
__device__ __forceinline__ void load_freq(const Params &p, uint64_t *freq) {
  for (int i = threadIdx.x; i < p.R / 2; i += kThreads) {
    const double t = (double)p.inv_freq[i] * 0.15915494309189533577;   // / (2 pi)
    const double f = t - floor(t);
    freq[i] = f < 1.0 ? (uint64_t)(f * 0x1p53) << 11 : 0ull;
  }
}

template <int LR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < LR; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// The pairs of eight elements u from column 8 v turned by the table's angles (back: the
// other way).  All lanes of the warp together.
template <int LR>
__device__ __forceinline__ void turn(const Params &p, const float2 *cs, float *row, int v, bool back,
                                     float (&u)[8]) {
  const int half = p.R / 2;
  const float sign = back ? -1.f : 1.f;
  if (p.interleaved) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int i = 4 * v + m;
      if (i >= half) continue;
      const float2 t = cs[i];
      const float a = u[2 * m], b = u[2 * m + 1], s = sign * t.y;
      u[2 * m] = fmaf(a, t.x, -(b * s));
      u[2 * m + 1] = fmaf(a, s, b * t.x);
    }
  } else if (half % 8 == 0) {   // the partners of a lane's elements are all in one other lane
    const int w = half / 8, lane = threadIdx.x & 31, first = lane - v;
    const bool low = v < w, on = v < 2 * w;
    const int from = on ? first + (low ? v + w : v - w) : lane;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float o = __shfl_sync(0xffffffffu, u[j], from);
      if (!on) continue;
      const float2 t = cs[8 * (low ? v : v - w) + j];
      const float s = sign * t.y;
      u[j] = low ? fmaf(u[j], t.x, -(o * s)) : fmaf(o, s, u[j] * t.x);
    }
  } else {
    float4 *at = reinterpret_cast<float4 *>(row + 8 * v);
    at[0] = make_float4(u[0], u[1], u[2], u[3]);
    at[1] = make_float4(u[4], u[5], u[6], u[7]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = 8 * v + j;
      if (i >= p.R) continue;
      const bool low = i < half;
      const float o = row[low ? i + half : i - half];
      const float2 t = cs[low ? i : i - half];
      const float s = sign * t.y;
      u[j] = low ? fmaf(u[j], t.x, -(o * s)) : fmaf(o, s, u[j] * t.x);
    }
    __syncwarp();
  }
}

// Rows of a tile: token by token, its heads of q, then of k.
struct Row {
  bool on, key;
  int tok, head;
};
__device__ __forceinline__ Row row_of(const Params &p, int r, int rows) {
  const int H = p.Hq + p.Hk, tok = r / H, h = r - tok * H;
  return {r < rows, h >= p.Hq, tok, h >= p.Hq ? h - p.Hq : h};
}

template <typename T, int LR, bool BACK>
__global__ void __launch_bounds__(kThreads)
gdn_qk_norm_kernel(const Params p) {
  constexpr int RG = kThreads / LR;   // rows side by side
  __shared__ float2 table[kTokens * kMaxHalf];
  __shared__ __align__(16) float rows_buf[RG * LR * 8];
  __shared__ uint64_t freq[kMaxHalf];
  const int tid = threadIdx.x, v = tid % LR, rg = tid / LR;
  const bool von = 8 * v < p.D;
  float *buf = rows_buf + rg * LR * 8;
  float w[2][8];
  float own[BACK ? 2 : 1][8] = {}, all[BACK ? 2 : 1][8] = {};   // sums for the weights
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w[0][j] = von && p.wq ? p.wq[8 * v + j] : 1.f;
    w[1][j] = von && p.wk ? p.wk[8 * v + j] : 1.f;
  }
  if (p.R) load_freq(p, freq);
  const float over = p.l2 ? 1.f : 1.f / (float)p.D;
  const int64_t tiles = (p.tokens + p.tile - 1) / p.tile;
  int summed = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t tok0 = tile * p.tile;
    const int cnt = (int)(p.tokens - tok0 < p.tile ? p.tokens - tok0 : p.tile);
    const int rows = cnt * (p.Hq + p.Hk);
    __syncthreads();   // the last tile's table has been read
    if (p.R) turn_table(p, tok0, cnt, freq, table);
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += kRows * RG) {
      Raw8<T> x[kRows], d[BACK ? kRows : 1];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const Row row = row_of(p, r0 + i * RG + rg, rows);
        x[i].zero();
        if (BACK) d[i].zero();
        if (!row.on || !von) continue;
        const int64_t tok = tok0 + row.tok;
        x[i].load(row.key ? static_cast<const T *>(p.k) + tok * p.sk + row.head * p.D + 8 * v
                          : static_cast<const T *>(p.q) + tok * p.sq + row.head * p.D + 8 * v);
        if (BACK)
          d[i].load(row.key
                        ? static_cast<const T *>(p.dk_in) + (tok * p.Hk + row.head) * p.D + 8 * v
                        : static_cast<const T *>(p.dq_in) + (tok * p.Hq + row.head) * p.D + 8 * v);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (r0 + i * RG >= rows) break;   // the same for the whole CTA
        const Row row = row_of(p, r0 + i * RG + rg, rows);
        const float2 *cs = table + (row.on ? row.tok : 0) * (p.R / 2);
        float xv[8], u[8], ss = 0.f;
        x[i].get(xv);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(xv[j], xv[j], ss);
        const float sq = row_sum<LR>(ss);
        const float r = row.on ? rsqrtf(fmaf(sq, over, p.eps)) : 0.f;
        const float scale = row.key ? 1.f : p.scale;
        if constexpr (!BACK) {
          const float f = r * scale;
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = xv[j] * f * (row.key ? w[1][j] : w[0][j]);
          if (p.R) turn<LR>(p, cs, buf, v, false, u);
        } else {
          d[i].get(u);
          if (p.R) turn<LR>(p, cs, buf, v, true, u);
          float m = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            u[j] *= scale;
            const float t = u[j] * xv[j] * r;
            if (row.key) own[1][j] += t;
            else own[0][j] += t;
            u[j] *= row.key ? w[1][j] : w[0][j];
            m = fmaf(xv[j], u[j], m);
          }
          m = row_sum<LR>(m) * over * r * r;
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = r * fmaf(-xv[j], m, u[j]);
        }
        if (row.on && von) {
          const int64_t tok = tok0 + row.tok;
          Raw8<T> out;
          out.set(u);
          out.store(row.key ? static_cast<T *>(p.ok) + (tok * p.Hk + row.head) * p.D + 8 * v
                            : static_cast<T *>(p.oq) + (tok * p.Hq + row.head) * p.D + 8 * v);
        }
      }
      if (BACK && ++summed == 16) {   // at most 64 rows in one run of an accumulator
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          all[0][j] += own[0][j];
          all[BACK][j] += own[BACK][j];
          own[0][j] = own[BACK][j] = 0.f;
        }
        summed = 0;
      }
    }
  }
  if constexpr (BACK) {   // the CTA's sums, in the order of its rows of threads
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) buf[8 * v + j] = all[s][j] + own[s][j];
      __syncthreads();
      for (int c = tid; c < p.D; c += kThreads) {
        float sum = 0.f;
        for (int i = 0; i < RG; ++i) sum += rows_buf[i * LR * 8 + c];
        p.part[((int64_t)blockIdx.x * 2 + s) * p.D + c] = sum;
      }
    }
  }
}

// The weights' gradients: 32 columns a CTA, its 32 warps over the partial sums.
__global__ void __launch_bounds__(1024) gdn_qk_weights_kernel(const Params p) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const int n = 2 * p.D;
  float sum = 0.f;
  if (c < n)
    for (int i = warp; i < p.parts; i += 32) sum += p.part[(int64_t)i * n + c];
  red[warp][lane] = sum;
  __syncthreads();
  if (warp) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += red[i][lane];
  if (c >= n) return;
  float *out = c < p.D ? p.dwq : p.dwk;
  if (out) out[c < p.D ? c : c - p.D] = sum;
}

// Tokens of a tile and CTAs: one token where there are few.
struct Grid {
  int tile;
  int64_t ctas;
};
Grid grid_of(int64_t tokens, bool back) {
  Grid g;
  g.tile = tokens >= 2 * kTokens * kSMs ? kTokens : 1;
  const int64_t tiles = (tokens + g.tile - 1) / g.tile, most = (back ? 3 : 5) * kSMs;
  g.ctas = tiles < most ? tiles : most;
  return g;
}

template <typename T, bool BACK>
cudaError_t launch_t(const Params &p, int64_t ctas, cudaStream_t stream) {
  const unsigned n = (unsigned)ctas;
  if (p.D <= 32) gdn_qk_norm_kernel<T, 4, BACK><<<n, kThreads, 0, stream>>>(p);
  else if (p.D <= 64) gdn_qk_norm_kernel<T, 8, BACK><<<n, kThreads, 0, stream>>>(p);
  else if (p.D <= 128) gdn_qk_norm_kernel<T, 16, BACK><<<n, kThreads, 0, stream>>>(p);
  else gdn_qk_norm_kernel<T, 32, BACK><<<n, kThreads, 0, stream>>>(p);
  return taken(cudaGetLastError());
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
  p.q = q; p.k = k; p.wq = q_weight; p.wk = k_weight;
  p.positions = positions; p.inv_freq = inv_freq;
  p.oq = q_out; p.ok = k_out;
  p.sq = sq; p.sk = sk;
  p.tokens = (int64_t)rows;
  p.seq_len = seq_len;
  p.Hq = q_heads; p.Hk = k_heads; p.D = head_dim; p.R = rotary_dim;
  p.eps = eps;
  p.scale = q_scale;
  p.l2 = flags & GDN_QK_L2NORM;
  p.interleaved = flags & GDN_ROPE_INTERLEAVED;
  const Grid g = grid_of(p.tokens, false);
  p.tile = g.tile;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t err = dtype == GDN_F32 ? launch_t<float, false>(p, g.ctas, s)
                                           : launch_t<__nv_bfloat16, false>(p, g.ctas, s);
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_qk_norm_workspace_size(int32_t batch, int32_t seq_len, int32_t head_dim) {
  if (batch <= 0 || seq_len < 0 || head_dim <= 0) return 0;
  return (size_t)gdn::qk::grid_of((int64_t)batch * seq_len, true).ctas * 2 * head_dim * 4;
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
  const Grid g = grid_of((int64_t)rows, true);
  const bool sums = dq_weight || dk_weight;
  if (!workspace || workspace_bytes < (size_t)g.ctas * 2 * w_bytes) return GDN_ERR_WORKSPACE;
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
  p.q = q; p.k = k; p.wq = q_weight; p.wk = k_weight;
  p.positions = positions; p.inv_freq = inv_freq;
  p.dq_in = d_q_out; p.dk_in = d_k_out;
  p.oq = dq; p.ok = dk;
  p.dwq = dq_weight; p.dwk = dk_weight;
  p.part = static_cast<float *>(workspace);
  p.sq = sq; p.sk = sk;
  p.tokens = (int64_t)rows;
  p.seq_len = seq_len;
  p.Hq = q_heads; p.Hk = k_heads; p.D = head_dim; p.R = rotary_dim;
  p.eps = eps;
  p.scale = q_scale;
  p.l2 = flags & GDN_QK_L2NORM;
  p.interleaved = flags & GDN_ROPE_INTERLEAVED;
  p.tile = g.tile;
  p.parts = (int32_t)g.ctas;
  cudaError_t err = dtype == GDN_F32 ? launch_t<float, true>(p, g.ctas, s)
                                     : launch_t<__nv_bfloat16, true>(p, g.ctas, s);
  if (err == cudaSuccess && sums) {
    gdn_qk_weights_kernel<<<(2 * head_dim + 31) / 32, 1024, 0, s>>>(p);
    err = taken(cudaGetLastError());
  }
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
