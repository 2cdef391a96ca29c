// One token of linear attention with a decay for each head, on states that
// live in the pages of a pool: per (sequence, head), with S the fp32 state,
//
//   S' = lam S + k v^T,   o = S'^T q,   lam = exp(log_decay[h])
//
// The step reads and writes each state once and does 5 dk dv operations on
// it, so it is bound by HBM bandwidth (by latency for a few sequences).  One
// CTA of 256 threads owns COLS columns of one head's state: thread t holds
// columns 4 (t % (COLS/4)) .. +3 of rows t / (COLS/4) + m rows apart in
// registers.  64 columns where dv holds whole ones: the page number is one more
// latency ahead of the state, and twice the bytes on their way cover it (1024
// sequences of 16 heads, 64/64: 82 us, 97 % of the copy bandwidth, against 95 us with
// 32 columns; 128 sequences 7.7 against 9.3; 8 of them 2.3 either way).
#include "gdn_lin.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kThreads = 256;

struct DecodeParams {
  const void *q, *k, *v;
  const float *log_decay;
  const float *s_in;
  float *s_out;
  const int32_t *pages;
  void *o;
  DeviceStatus *status;
  int64_t page_stride;  // floats from page to page
  int32_t num_heads, dk, dv, num_pages;
};

template <typename T, int DKT, int COLS>
__global__ void __launch_bounds__(kThreads)
gdn_lin_decode_kernel(const DecodeParams p) {
  constexpr int kCols = COLS, LANES = COLS / 4, ROWS = kThreads / LANES, RPT = DKT / ROWS;
  __shared__ float sk[DKT], sq[DKT];
  __shared__ float part[8][kCols];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = blockIdx.x, h = blockIdx.y, n = blockIdx.z;
  const int dv = p.dv, cg = tid % LANES, rg = tid / LANES, col = tile * kCols + 4 * cg;
  const size_t head = (size_t)n * p.num_heads + h;
  T *o = static_cast<T *>(p.o) + head * dv + tile * kCols;

  const int page = p.pages ? p.pages[n] : n;
  if (page < 0 || page >= p.num_pages) {  // a padded row (-1), or a bad number
    if (page != -1 && tid == 0 && p.status)
      report(p.status, GDN_ERR_DEVICE_CHECK, (uint32_t)n, (uint32_t)h, 0u);
    if (tid < kCols) store_out(o + tid, 0.f);
    return;
  }
  const size_t base = (size_t)page * p.page_stride + (size_t)h * DKT * dv + col;
  float4 s[RPT];
#pragma unroll
  for (int m = 0; m < RPT; ++m)
    s[m] = p.s_in ? *reinterpret_cast<const float4 *>(p.s_in + base + (size_t)(rg + ROWS * m) * dv)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
  const T *v = static_cast<const T *>(p.v) + head * dv + col;
  const float v0 = to_f32(v[0]), v1 = to_f32(v[1]), v2 = to_f32(v[2]), v3 = to_f32(v[3]);
  for (int i = tid; i < DKT; i += kThreads) {
    sk[i] = to_f32(static_cast<const T *>(p.k)[head * DKT + i]);
    sq[i] = to_f32(static_cast<const T *>(p.q)[head * DKT + i]);
  }
  const float lam = expf(p.log_decay[h]);
  __syncthreads();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int m = 0; m < RPT; ++m) {
    const int i = rg + ROWS * m;
    const float ki = sk[i], qi = sq[i];
    float4 x = s[m];
    x.x = fmaf(lam, x.x, ki * v0);
    x.y = fmaf(lam, x.y, ki * v1);
    x.z = fmaf(lam, x.z, ki * v2);
    x.w = fmaf(lam, x.w, ki * v3);
    *reinterpret_cast<float4 *>(p.s_out + base + (size_t)i * dv) = x;
    a.x = fmaf(qi, x.x, a.x);
    a.y = fmaf(qi, x.y, a.y);
    a.z = fmaf(qi, x.z, a.z);
    a.w = fmaf(qi, x.w, a.w);
  }
  // lanes cg, cg + LANES, ... hold the same columns
#pragma unroll
  for (int off = LANES; off < 32; off <<= 1) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, off);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, off);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, off);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, off);
  }
  if (lane < LANES) *reinterpret_cast<float4 *>(&part[warp][4 * lane]) = a;
  __syncthreads();
  if (tid < kCols) {
    float r = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) r += part[w][tid];
    store_out(o + tid, r);
  }
}

template <typename T, int COLS>
cudaError_t launch_c(const DecodeParams &p, int num_seqs, cudaStream_t stream) {
  const dim3 grid(p.dv / COLS, p.num_heads, num_seqs);
  switch (p.dk) {
    case 32: gdn_lin_decode_kernel<T, 32, COLS><<<grid, kThreads, 0, stream>>>(p); break;
    case 64: gdn_lin_decode_kernel<T, 64, COLS><<<grid, kThreads, 0, stream>>>(p); break;
    case 96: gdn_lin_decode_kernel<T, 96, COLS><<<grid, kThreads, 0, stream>>>(p); break;
    case 128: gdn_lin_decode_kernel<T, 128, COLS><<<grid, kThreads, 0, stream>>>(p); break;
    case 160: gdn_lin_decode_kernel<T, 160, COLS><<<grid, kThreads, 0, stream>>>(p); break;
    case 192: gdn_lin_decode_kernel<T, 192, COLS><<<grid, kThreads, 0, stream>>>(p); break;
    case 224: gdn_lin_decode_kernel<T, 224, COLS><<<grid, kThreads, 0, stream>>>(p); break;
    case 256: gdn_lin_decode_kernel<T, 256, COLS><<<grid, kThreads, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}
// 64 columns a CTA wherever dv holds whole ones (measured at the top).
template <typename T>
cudaError_t launch_t(const DecodeParams &p, int num_seqs, cudaStream_t stream) {
  return p.dv % 64 == 0 ? launch_c<T, 64>(p, num_seqs, stream)
                        : launch_c<T, 32>(p, num_seqs, stream);
}

bool aligned16(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }
bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace lin
}  // namespace gdn

extern "C" gdn_status gdn_lin_decode(const void *q, const void *k, const void *v,
                                     const float *log_decay, const float *state_in,
                                     float *state_out, const int32_t *pages, void *o,
                                     int32_t num_seqs, int32_t num_heads, int32_t head_dim_k,
                                     int32_t head_dim_v, int32_t num_pages, int64_t page_stride,
                                     gdn_dtype dtype, uint32_t flags, void *workspace,
                                     size_t workspace_bytes, void *stream) {
  using namespace gdn;
  using namespace gdn::lin;
  if (num_seqs <= 0 || num_heads <= 0 || head_dim_k <= 0 || head_dim_v <= 0 || num_pages <= 0)
    return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (flags) return GDN_ERR_INVALID_ARG;
  if (head_dim_k > 256 || head_dim_k % 32 || head_dim_v > 256 || head_dim_v % 32)
    return GDN_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || num_heads > 65535) return GDN_ERR_UNSUPPORTED;
  const int64_t page = (int64_t)num_heads * head_dim_k * head_dim_v;
  if (page_stride == 0) page_stride = page;
  if (page_stride < page || page_stride % 4) return GDN_ERR_INVALID_ARG;
  if (!q || !k || !v || !log_decay || !state_out || !o) return GDN_ERR_INVALID_ARG;
  if (!pages && num_pages < num_seqs) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {q, k, v, log_decay, state_in, state_out, pages, o, workspace};
  for (const void *x : ptrs)
    if (x && !aligned16(x)) return GDN_ERR_INVALID_ARG;
  if (workspace && workspace_bytes < kStatusBytes) return GDN_ERR_WORKSPACE;

  const size_t e = dtype == GDN_F32 ? 4 : 2, rows = (size_t)num_seqs * num_heads;
  const size_t b_state = ((size_t)(num_pages - 1) * page_stride + page) * 4;
  const size_t b_o = rows * head_dim_v * e;
  struct Range { const void *p; size_t n; };
  const Range inputs[] = {{q, rows * head_dim_k * e}, {k, rows * head_dim_k * e},
                          {v, b_o}, {log_decay, (size_t)num_heads * 4},
                          {pages, pages ? (size_t)num_seqs * 4 : 0},
                          {workspace, workspace ? kStatusBytes : 0}};
  for (const Range &r : inputs)
    if (overlaps(o, b_o, r.p, r.n) || overlaps(state_out, b_state, r.p, r.n))
      return GDN_ERR_INVALID_ARG;
  if (overlaps(o, b_o, state_out, b_state) || overlaps(o, b_o, state_in, b_state))
    return GDN_ERR_INVALID_ARG;
  if (state_in && state_in != state_out && overlaps(state_in, b_state, state_out, b_state))
    return GDN_ERR_INVALID_ARG;

  DecodeParams p{q, k, v, log_decay, state_in, state_out, pages, o,
                 static_cast<DeviceStatus *>(workspace), page_stride, num_heads, head_dim_k,
                 head_dim_v, num_pages};
  const cudaError_t err = dtype == GDN_F32
                              ? launch_t<float>(p, num_seqs, (cudaStream_t)stream)
                              : launch_t<__nv_bfloat16>(p, num_seqs, (cudaStream_t)stream);
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
