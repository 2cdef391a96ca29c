// One token of the selective scan per sequence, on states in the pages of a pool:
//
//   h' = exp(delta A) h + delta x b,   y = (c . h' + D_skip x) silu(gate)
//
// A state is read and written once for five operations on an element, so the step is
// bound by HBM bandwidth (by latency for a few sequences).  S / 4 lanes share a channel,
// each with four states in one 16-byte load; a CTA owns 512 / S channels and goes over
// SEQS sequences with all of their loads on the way at once, its rates computed once.
#include "gdn_ssm.cuh"

namespace gdn {
namespace ssm {
namespace {

// Sequences of a CTA, its threads, CTAs an SM.  (1024 of [1280, 16], one call behind another:
// 35.4 us, 4.7 TB/s of the states alone; caches cold 39 us, 4.6 TB/s of all bytes.  As the
// first, with 3, 6 or 8 sequences 39, 51, 51; 256 threads in 4 or 5 CTAs 37 and 41, 128 in 7,
// 8 or 10 37, 36 and 39.  By CTAs that stay, the next states on their way to shared memory by
// asynchronous copies, 42; to registers, 70.)
constexpr int kSeqs = 4;
constexpr int kStepThreads = 128, kCtas = 9;

struct StepParams {
  const void *x, *dt, *b, *c, *gate;
  const float *A_log, *d_skip, *dt_bias, *s_in;
  float *s_out;
  const int32_t *pages;
  void *y;
  DeviceStatus *status;
  int64_t page_stride;   // floats from page to page
  int32_t num_seqs, D, Dg, G, num_pages;
  bool softplus;
};

__device__ __forceinline__ float4 four(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 four(const __nv_bfloat16 *p) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

template <typename T, int S, int SEQS>
__global__ void __launch_bounds__(kStepThreads, kCtas)
gdn_ssm_step_kernel(const StepParams p) {
  constexpr int LS = S / 4, CH = kStepThreads / LS, PER = (SEQS + LS - 1) / LS;
  constexpr uint32_t kAll = 0xffffffffu;
  const int tid = threadIdx.x, sl = tid % LS, ch = blockIdx.x * CH + tid / LS;
  const bool on = ch < p.D;
  const int n0 = blockIdx.y * SEQS, lane0 = (tid & 31) - sl;
  const int64_t at = (int64_t)ch * S + 4 * sl;

  float4 h[SEQS];
  int page[SEQS];
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    const int n = n0 + i;
    page[i] = n >= p.num_seqs ? -1 : p.pages ? p.pages[n] : n;
  }
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    const bool good = page[i] >= 0 && page[i] < p.num_pages;
    if (!good && page[i] != -1 && tid == 0 && p.status)
      report(p.status, GDN_ERR_DEVICE_CHECK, (uint32_t)(n0 + i), (uint32_t)blockIdx.x, 0u);
    if (!good) page[i] = -1;
    h[i] = on && good && p.s_in ? four(p.s_in + page[i] * p.page_stride + at)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // The steps of sequences n0 + sl, n0 + sl + LS, ...: the LS lanes of a channel share them.
  const float bias = on && p.dt_bias ? p.dt_bias[ch] : 0.f;
  const float skip = on && p.d_skip ? p.d_skip[ch] : 0.f;
  const int64_t tok = (int64_t)(n0 + sl) * p.D + ch;
  float x[PER], d[PER], gate[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const bool go = on && sl + k * LS < SEQS && n0 + sl + k * LS < p.num_seqs;
    const int64_t i = tok + (int64_t)k * LS * p.D;
    x[k] = go ? to_f32(static_cast<const T *>(p.x)[i]) : 0.f;
    d[k] = go ? to_f32(static_cast<const T *>(p.dt)[i]) + bias : 0.f;
    gate[k] = go && p.gate ? to_f32(static_cast<const T *>(p.gate)[i]) : 0.f;
  }
  const float4 al = on ? four(p.A_log + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 A = make_float4(rate(al.x), rate(al.y), rate(al.z), rate(al.w));
  const float slow = fmaxf(fmaxf(A.x, A.y), fmaxf(A.z, A.w));
  if (p.softplus) {
#pragma unroll
    for (int k = 0; k < PER; k += 2) {
      float a, b;
      unpk(softplus2<T>(pk(d[k], k + 1 < PER ? d[k + 1] : 0.f)), a, b);
      d[k] = a;
      if (k + 1 < PER) d[k + 1] = b;
    }
  }
  const int group = on && p.G > 1 ? ch / p.Dg : 0;
  const T *b = static_cast<const T *>(p.b) + ((int64_t)n0 * p.G + group) * S + 4 * sl;
  const T *c = static_cast<const T *>(p.c) + ((int64_t)n0 * p.G + group) * S + 4 * sl;
  const int next = p.G * S;
  float sum[SEQS];
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    const float di = __shfl_sync(kAll, d[i / LS], lane0 + i % LS);
    const float ui = di * __shfl_sync(kAll, x[i / LS], lane0 + i % LS);
    sum[i] = 0.f;
    if (!on || page[i] < 0) continue;
    const float4 bv = four(b + i * next), cv = four(c + i * next);
    float4 s = h[i];
    const float lift = lift_of(di, slow);
    s.x = fmaf(ex2(fmaf(di, A.x, lift)), s.x, ui * bv.x);
    s.y = fmaf(ex2(fmaf(di, A.y, lift)), s.y, ui * bv.y);
    s.z = fmaf(ex2(fmaf(di, A.z, lift)), s.z, ui * bv.z);
    s.w = fmaf(ex2(fmaf(di, A.w, lift)), s.w, ui * bv.w);
    *reinterpret_cast<float4 *>(p.s_out + page[i] * p.page_stride + at) = s;
    sum[i] = fmaf(cv.x, s.x, cv.y * s.y) + fmaf(cv.z, s.z, cv.w * s.w);
  }
  // c . h of a sequence to the lane that holds its step
#pragma unroll
  for (int i = 0; i < SEQS; ++i)
#pragma unroll
    for (int m = 1; m < LS; m *= 2) sum[i] += __shfl_xor_sync(kAll, sum[i], m);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    float y = 0.f;
    int mine = -1;
#pragma unroll
    for (int i = 0; i < SEQS; ++i)
      if (i == sl + k * LS) {
        y = sum[i];
        mine = page[i];
      }
    if (!on || sl + k * LS >= SEQS || n0 + sl + k * LS >= p.num_seqs) continue;
    if (mine >= 0) {
      if (p.d_skip) y = fmaf(skip, x[k], y);
      if (p.gate) y *= gate[k] * sigmoid(gate[k]);
    }
    store_out(static_cast<T *>(p.y) + tok + (int64_t)k * LS * p.D, y);
  }
}

template <typename T, int S>
cudaError_t launch_s(const StepParams &p, cudaStream_t stream) {
  constexpr int CH = 4 * kStepThreads / S;
  const int blocks = (p.D + CH - 1) / CH;
  if ((int64_t)blocks * p.num_seqs >= 32 * kSMs) {
    const dim3 grid(blocks, (p.num_seqs + kSeqs - 1) / kSeqs);
    gdn_ssm_step_kernel<T, S, kSeqs><<<grid, kStepThreads, 0, stream>>>(p);
  } else {
    gdn_ssm_step_kernel<T, S, 1><<<dim3(blocks, p.num_seqs), kStepThreads, 0, stream>>>(p);
  }
  return taken(cudaGetLastError());
}
template <typename T>
cudaError_t launch_t(const StepParams &p, int S, cudaStream_t stream) {
  switch (S) {
    case 8: return launch_s<T, 8>(p, stream);
    case 16: return launch_s<T, 16>(p, stream);
    case 32: return launch_s<T, 32>(p, stream);
    default: return launch_s<T, 64>(p, stream);
  }
}

}  // namespace
}  // namespace ssm
}  // namespace gdn

extern "C" gdn_status gdn_ssm_step(const void *x, const void *dt, const float *A_log, const void *b,
                                   const void *c, const float *D_skip, const void *gate,
                                   const float *dt_bias, const float *state_in, float *state_out,
                                   const int32_t *pages, void *y, int32_t num_seqs,
                                   int32_t channels, int32_t d_state, int32_t groups,
                                   int32_t num_pages, int64_t page_stride, gdn_dtype dtype,
                                   uint32_t flags, void *workspace, size_t workspace_bytes,
                                   void *stream) {
  using namespace gdn;
  using namespace gdn::ssm;
  const gdn_status st = check_sizes(num_seqs, 1, channels, d_state, groups, num_seqs, nullptr,
                                    dtype, flags);
  if (st != GDN_OK) return st;
  if (num_pages <= 0 || (!pages && num_pages < num_seqs)) return GDN_ERR_INVALID_ARG;
  const int64_t page = (int64_t)channels * d_state;
  if (page_stride == 0) page_stride = page;
  if (page_stride < page || page_stride % 4) return GDN_ERR_INVALID_ARG;
  if (!x || !dt || !A_log || !b || !c || !state_out || !y) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {x, dt, A_log, b, c, D_skip, gate, dt_bias, state_in, state_out, pages, y,
                        workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_INVALID_ARG;
  if (workspace && workspace_bytes < kStatusBytes) return GDN_ERR_WORKSPACE;
  const size_t e = dtype == GDN_F32 ? 4 : 2, wide = (size_t)num_seqs * channels * e;
  const size_t thin = (size_t)num_seqs * groups * d_state * e;
  const size_t pool = ((size_t)(num_pages - 1) * page_stride + page) * 4;
  const Range outs[] = {{y, wide}, {state_out, pool}};
  const Range ins[] = {{x, wide}, {dt, wide}, {gate, wide}, {b, thin}, {c, thin},
                       {A_log, (size_t)page * 4}, {D_skip, (size_t)channels * 4},
                       {dt_bias, (size_t)channels * 4}, {pages, (size_t)num_seqs * 4},
                       {workspace, kStatusBytes},
                       {state_in == state_out ? nullptr : state_in, pool}};
  if (!apart(outs, ins) || overlaps(outs[0], {state_in, pool})) return GDN_ERR_INVALID_ARG;

  const StepParams p{x, dt, b, c, gate, A_log, D_skip, dt_bias, state_in, state_out, pages, y,
                     static_cast<DeviceStatus *>(workspace), page_stride, num_seqs, channels,
                     channels / groups, groups, num_pages, (flags & GDN_DT_SOFTPLUS) != 0};
  const cudaError_t err = dtype == GDN_F32
                              ? launch_t<float>(p, d_state, (cudaStream_t)stream)
                              : launch_t<__nv_bfloat16>(p, d_state, (cudaStream_t)stream);
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
