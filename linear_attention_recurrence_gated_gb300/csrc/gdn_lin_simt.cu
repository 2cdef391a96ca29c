// Linear attention with a decay for each head on the CUDA cores: the scan of
// gdn_lin.cuh in fp32, for fp32 storage and for head sizes without a
// tensor-core form.
//
// One CTA owns 32 value columns of one (sequence, head) and walks its chunks
// of 64 tokens.  Per chunk, with rows i, j of the tile and e valid rows:
//   P_ij = lam^|i-j| (a_i.b_j) for j <= i (j >= i backward in time), else 0
//   o_i  = lam^(i+1) S^T a_i + sum_j P_ij c_j      (lam^(e-1-i) backward)
//   S   <- lam^e S + sum_j lam^(e-1-j) b_j c_j^T   (lam^(j+1)   backward)
// The state stays in shared memory in fp32; masked products are replaced by
// zeros and rows past the sequence's end are never loaded, so nothing that
// lies there (an infinity, a NaN of the next sequence) reaches a result.
#include "gdn_lin.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kThreads = 256;
constexpr int kC = 64;        // tokens per chunk
constexpr int kCols = 32;     // value columns per CTA
constexpr int kLd = kC + 4;   // row of the transposed tiles

__host__ __device__ constexpr size_t smem_floats(int da) {
  return (size_t)2 * da * kLd + kC * kCols + kC * (kC + 1) + (size_t)da * kCols + kC + 1;
}

// STATES: the first launch of a split along time (the state increments alone).
template <typename T, bool STATES>
__global__ void __launch_bounds__(kThreads)
gdn_lin_simt_kernel(const Params p) {
  extern __shared__ __align__(16) float sm[];
  const Scan &s = p.scan[blockIdx.z % p.num_scans];
  const int z = blockIdx.z / p.num_scans, h = blockIdx.y, col0 = blockIdx.x * kCols;
  if (col0 >= s.dc) return;  // (the scans of a launch may have fewer tiles)
  const int tid = threadIdx.x, H = p.num_heads, da = s.da, dc = s.dc;
  const bool rev = s.reverse != 0;
  float *At = sm, *Bt = At + (size_t)da * kLd, *V = Bt + (size_t)da * kLd, *P = V + kC * kCols,
        *S = P + kC * (kC + 1), *lam = S + (size_t)da * kCols;

  Span span;
  if (!span_of(p, z, h, span)) return;
  const int64_t start = span.start, len = span.len;
  const int64_t unit = (int64_t)span.n * H + h;
  // the segment whose end is the sequence's, in the scan's direction
  const bool last = span.seg == (rev ? 0 : span.count - 1);
  if (STATES && last) return;
  const int64_t x_unit = ((int64_t)(blockIdx.z % p.num_scans) * p.slots + z) * H + h;  // of seg_x
  float *const s_out = STATES ? p.seg_x + x_unit * da * dc
                              : s.s_out && last ? s.s_out + unit * da * dc : nullptr;
  const float ld = p.log_decay[h];
  for (int i = tid; i <= kC; i += kThreads) lam[i] = i ? expf(ld * (float)i) : 1.f;
  for (int i = tid; i < da * kCols; i += kThreads) {
    const int row = i / kCols, col = col0 + i % kCols;
    float v = STATES ? 0.f : state_in(s, unit, row, col);
    if (!STATES)  // the segments before this one, in order
      for (int k = rev ? span.count - 1 : 0; k != span.seg; k += rev ? -1 : 1) {
        const int64_t length = k == span.count - 1 ? span.total - k * p.seg_len : p.seg_len;
        v = fmaf(expf(ld * (float)length), v,
                 p.seg_x[(x_unit + (int64_t)(k - span.seg) * H) * da * dc + (int64_t)row * dc + col]);
      }
    S[i] = v;
  }
  const T *a = static_cast<const T *>(s.a) + (int64_t)h * da;
  const T *b = static_cast<const T *>(s.b) + (int64_t)h * da;
  const T *c = static_cast<const T *>(s.c) + (int64_t)h * dc + col0;
  T *o = static_cast<T *>(s.o) + (int64_t)h * dc + col0;

  const int64_t nc = (len + kC - 1) / kC;
  for (int64_t step = 0; step < nc; ++step) {
    const int64_t t0 = (rev ? nc - 1 - step : step) * kC, tok = start + t0;
    const int e = (int)(len - t0 < kC ? len - t0 : kC);
    __syncthreads();  // the last chunk's reads of the tiles are done
    for (int x = tid; x < kC * da; x += kThreads) {
      const int i = x / da, k = x % da;
      if (!STATES) At[k * kLd + i] = i < e ? to_f32(a[(tok + i) * s.sa + k]) : 0.f;
      Bt[k * kLd + i] = i < e ? to_f32(b[(tok + i) * s.sb + k]) : 0.f;
    }
    for (int x = tid; x < kC * kCols; x += kThreads) {
      const int i = x / kCols, j = x % kCols;
      V[x] = i < e ? to_f32(c[(tok + i) * s.sc + j]) : 0.f;
    }
    __syncthreads();
    if (!STATES) {  // P, 4 x 4 per thread
      const int i0 = (tid >> 4) * 4, j0 = (tid & 15) * 4;
      float acc[4][4] = {};
      for (int k = 0; k < da; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(At + k * kLd + i0);
        const float4 y = *reinterpret_cast<const float4 *>(Bt + k * kLd + j0);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int w = 0; w < 4; ++w) acc[u][w] = fmaf(xs[u], ys[w], acc[u][w]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int i = i0 + u, j = j0 + w, d = rev ? j - i : i - j;
          P[i * (kC + 1) + j] = d >= 0 ? acc[u][w] * lam[d] : 0.f;
        }
    }
    __syncthreads();
    if (!STATES) {  // o, 8 columns per thread
      const int i = tid >> 2, c0 = (tid & 3) * 8;
      float acc[8] = {};
      for (int k = 0; k < da; ++k) {
        const float x = At[k * kLd + i];
#pragma unroll
        for (int u = 0; u < 8; ++u) acc[u] = fmaf(x, S[k * kCols + c0 + u], acc[u]);
      }
      if (i < e) {
        const float f = lam[rev ? e - 1 - i : i + 1];
#pragma unroll
        for (int u = 0; u < 8; ++u) acc[u] *= f;
      }
      for (int j = 0; j < kC; ++j) {
        const float x = P[i * (kC + 1) + j];
#pragma unroll
        for (int u = 0; u < 8; ++u) acc[u] = fmaf(x, V[j * kCols + c0 + u], acc[u]);
      }
      if (i < e) {
        T *row = o + (tok + i) * ((int64_t)H * dc) + c0;
#pragma unroll
        for (int u = 0; u < 8; ++u) store_out(row + u, acc[u]);
      }
    }
    __syncthreads();
    for (int x = tid; x < kC * kCols; x += kThreads) {  // values times their weight
      const int j = x / kCols;
      if (j < e) V[x] *= lam[rev ? j + 1 : e - 1 - j];
    }
    __syncthreads();
    {  // the state, 4 columns per thread and step of 32 rows
      const int c0 = (tid & 7) * 4;
      const float le = lam[e];
      for (int k = tid >> 3; k < da; k += kThreads / 8) {
        float4 *st = reinterpret_cast<float4 *>(S + k * kCols + c0);
        float4 acc = *st;
        acc.x *= le;
        acc.y *= le;
        acc.z *= le;
        acc.w *= le;
        for (int j = 0; j < kC; ++j) {
          const float x = Bt[k * kLd + j];
          const float4 v = *reinterpret_cast<const float4 *>(V + j * kCols + c0);
          acc.x = fmaf(x, v.x, acc.x);
          acc.y = fmaf(x, v.y, acc.y);
          acc.z = fmaf(x, v.z, acc.z);
          acc.w = fmaf(x, v.w, acc.w);
        }
        *st = acc;
      }
    }
  }
  if (s_out == nullptr) return;
  __syncthreads();
  for (int i = tid; i < da * kCols; i += kThreads)
    s_out[(int64_t)(i / kCols) * dc + col0 + i % kCols] = S[i];
}

template <typename T, bool STATES>
cudaError_t run(const Params &p, int da, int dc, cudaStream_t stream) {
  const size_t bytes = smem_floats(da) * 4;
  const cudaError_t err = cudaFuncSetAttribute(
      gdn_lin_simt_kernel<T, STATES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (err != cudaSuccess) return err;
  const dim3 grid(dc / kCols, p.num_heads, p.slots * p.num_scans);
  gdn_lin_simt_kernel<T, STATES><<<grid, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const Params &p, cudaStream_t stream) {
  int da = 0, dc = 0;
  for (int i = 0; i < p.num_scans; ++i) {
    da = p.scan[i].da > da ? p.scan[i].da : da;
    dc = p.scan[i].dc > dc ? p.scan[i].dc : dc;
  }
  Params on = p;
  split(on, dc / kCols, kSimtWidth);
  if (on.seg_len) {
    const cudaError_t err = run<T, true>(on, da, dc, stream);
    if (err != cudaSuccess) return err;
  }
  return run<T, false>(on, da, dc, stream);
}

}  // namespace

cudaError_t launch_simt(const Params &p, gdn_dtype dtype, cudaStream_t stream) {
  return dtype == GDN_F32 ? launch_t<float>(p, stream) : launch_t<__nv_bfloat16>(p, stream);
}

}  // namespace lin
}  // namespace gdn
