// Group norm with an activation, channels last, forward and backward.
//
// x is [N][S][C]; sample n's group g holds channels g D .. (g + 1) D - 1 of
// its S rows (D = C / G).  With mean and var over those S D values
//   xh = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  u = xh w + b,
//   y  = act(u) silu(z)       (act: identity or silu; z the optional gate)
// and backward, with du = dy silu(z) act'(u) and dxh = du w,
//   dx = rstd (dxh - mean(dxh) - xh mean(dxh xh)),  dz = dy act(u) silu'(z),
//   dw = sum du xh,  db = sum du   (over every sample and row).
//
// Statistics are fp32: a thread sums x - c and (x - c)^2 over blocks of a few
// rows about the first value c of the block, and the partial (count, mean,
// squared deviation) triples are joined.  Their means are kept relative to the
// group's first value x0, and a value is normalised as ((x - x0) - mean) rstd:
// a mean far from zero cancels nothing and is rounded once, as it is stored.
// No sum runs over more than 128 values one after the other.
#include <stdint.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace norm {
namespace {

constexpr int kThreads = 256;
constexpr int kSMs = 152;
constexpr int kBlock = 16;   // rows summed by a thread before it joins them

struct Params {
  const void *x, *gate, *dy;
  const float *w, *b;
  void *y, *dx, *dgate;
  float *mean, *rstd;        // forward: written (may be NULL); backward: read
  float *dw, *db;
  float *part;               // backward: [CTAs][2][C] sums of du xh and du
  int64_t N, S;
  int32_t C, G, D;
  float eps;
  bool silu;
};

template <int V>
__device__ __forceinline__ void load(const float *p, float (&v)[V]) {
  if constexpr (V == 4) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[i];
  }
}
template <int V>
__device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[V]) {
  if constexpr (V == 8) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __bfloat162float(p[i]);
  }
}
template <int V>
__device__ __forceinline__ void store(float *p, const float (&v)[V]) {
  if constexpr (V == 4) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = v[i];
  }
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[V]) {
  if constexpr (V == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&t);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = __float2bfloat16_rn(v[i]);
  }
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// (count, mean, squared deviation) of two disjoint sets of values as one.
struct Stat {
  float n, mean, m2;
};
__device__ __forceinline__ Stat join(const Stat &a, const Stat &b) {
  const float n = a.n + b.n;
  if (n == 0.f) return a;
  const float f = b.n / n, d = b.mean - a.mean;
  return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}

// y of one value.
__device__ __forceinline__ float activate(float u, float z, bool silu, bool gated) {
  if (silu) u *= sigmoid(u);
  return gated ? u * z * sigmoid(z) : u;
}

// One CTA per sample: statistics in one pass over the sample's rows, the
// normalisation in a second (which finds a small sample in L1 or L2).  Threads
// are tiled over (row, vector of V channels).  Shared memory: a (count, mean,
// m2) triple per channel vector, then mean and rstd per group.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
gdn_norm_fwd_kernel(const Params p) {
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = CV < kThreads ? CV : kThreads, TY = kThreads / TX;
  const int tx = tid % TX, ty = tid / TX;
  Stat *st = reinterpret_cast<Stat *>(sm);             // [TY][CV]
  float *smean = sm + (size_t)3 * TY * CV, *srstd = smean + p.G;
  const T *xs = static_cast<const T *>(p.x), *zs = static_cast<const T *>(p.gate);
  for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
    const int64_t base = n * p.S * p.C;
    __syncthreads();
    for (int cv = tx; cv < CV && ty < TY; cv += TX) {
      const float x0 = to_f32(xs[base + (cv / DV) * p.D]);
      Stat all = {0.f, 0.f, 0.f};
      for (int64_t r0 = ty; r0 < p.S; r0 += kBlock * TY) {
        float c = 0.f, s1 = 0.f, s2 = 0.f, cnt = 0.f;
        for (int64_t r = r0; r < p.S && r < r0 + kBlock * TY; r += TY) {
          float v[V];
          load<V>(xs + base + r * p.C + cv * V, v);
          if (cnt == 0.f) c = v[0];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float d = v[i] - c;
            s1 += d;
            s2 = fmaf(d, d, s2);
          }
          cnt += V;
        }
        const float m = s1 / cnt;
        all = join(all, Stat{cnt, (c - x0) + m, s2 - s1 * m});
      }
      st[ty * CV + cv] = all;
    }
    __syncthreads();
    for (int g = tid >> 5; g < p.G; g += kThreads / 32) {
      Stat a = {0.f, 0.f, 0.f};
      for (int i = tid & 31; i < DV * TY; i += 32)
        a = join(a, st[(i / DV) * CV + g * DV + i % DV]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
        a = join(a, Stat{__shfl_xor_sync(0xffffffffu, a.n, off),
                         __shfl_xor_sync(0xffffffffu, a.mean, off),
                         __shfl_xor_sync(0xffffffffu, a.m2, off)});
      if ((tid & 31) == 0) {
        smean[g] = a.mean;
        srstd[g] = 1.f / sqrtf(fmaxf(a.m2 / a.n, 0.f) + p.eps);
        if (p.mean) p.mean[n * p.G + g] = to_f32(xs[base + g * p.D]) + a.mean;
        if (p.rstd) p.rstd[n * p.G + g] = srstd[g];
      }
    }
    __syncthreads();
    for (int cv = tx; cv < CV && ty < TY; cv += TX) {
      const int g = cv / DV;
      const float x0 = to_f32(xs[base + g * p.D]), mean = smean[g], rstd = srstd[g];
      float w[V], b[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        w[i] = p.w ? p.w[cv * V + i] : 1.f;
        b[i] = p.b ? p.b[cv * V + i] : 0.f;
      }
      for (int64_t r = ty; r < p.S; r += TY) {
        const int64_t at = base + r * p.C + cv * V;
        float v[V], z[V];
        load<V>(xs + at, v);
        if (zs) load<V>(zs + at, z);
#pragma unroll
        for (int i = 0; i < V; ++i)
          v[i] = activate(fmaf(((v[i] - x0) - mean) * rstd, w[i], b[i]), zs ? z[i] : 0.f, p.silu,
                          zs != nullptr);
        store<V>(static_cast<T *>(p.y) + at, v);
      }
    }
  }
}

// du of one value, and dz where there is a gate.
__device__ __forceinline__ float grad_u(float u, float z, float dy, bool silu, bool gated,
                                        float &dz) {
  float act = u, dact = 1.f;
  if (silu) {
    const float s = sigmoid(u);
    act = u * s;
    dact = s * (1.f + u * (1.f - s));
  }
  if (gated) {
    const float s = sigmoid(z);
    dz = dy * act * s * (1.f + z * (1.f - s));
    dy *= z * s;
  }
  return dy * dact;
}

// One CTA per sample: the group sums of dxh and dxh xh (and the channels' sums
// of du xh and du) in one pass, dx in a second.  Shared memory: two sums per
// channel vector and row of threads, two means per group, then the channels'
// running sums over the CTA's samples.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
gdn_norm_bwd_kernel(const Params p) {
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = CV < kThreads ? CV : kThreads, TY = kThreads / TX;
  const int tx = tid % TX, ty = tid / TX;
  float2 *st = reinterpret_cast<float2 *>(sm);          // [TY][CV]
  float2 *sg = st + (size_t)TY * CV;                    // [G]
  float2 *sc = sg + p.G;                                // [TY][C]: sums of du xh, du
  const T *xs = static_cast<const T *>(p.x), *zs = static_cast<const T *>(p.gate),
          *dys = static_cast<const T *>(p.dy);
  for (int i = tid; i < TY * p.C; i += kThreads) sc[i] = make_float2(0.f, 0.f);
  const float inv = 1.f / ((float)p.S * (float)p.D);
  for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
    const int64_t base = n * p.S * p.C;
    __syncthreads();
    for (int cv = tx; cv < CV && ty < TY; cv += TX) {
      const int g = cv / DV;
      const float mean = p.mean[n * p.G + g], rstd = p.rstd[n * p.G + g];
      float w[V], b[V], a1[V], a2[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        w[i] = p.w ? p.w[cv * V + i] : 1.f;
        b[i] = p.b ? p.b[cv * V + i] : 0.f;
        a1[i] = a2[i] = 0.f;
      }
      for (int64_t r = ty; r < p.S; r += TY) {
        const int64_t at = base + r * p.C + cv * V;
        float v[V], z[V], dy[V];
        load<V>(xs + at, v);
        load<V>(dys + at, dy);
        if (zs) load<V>(zs + at, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (v[i] - mean) * rstd;
          float dz;
          const float du = grad_u(fmaf(xh, w[i], b[i]), zs ? z[i] : 0.f, dy[i], p.silu,
                                  zs != nullptr, dz);
          a1[i] += du;
          a2[i] = fmaf(du, xh, a2[i]);
        }
      }
      float t1 = 0.f, t2 = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        t1 = fmaf(a1[i], w[i], t1);
        t2 = fmaf(a2[i], w[i], t2);
        float2 &acc = sc[ty * p.C + cv * V + i];
        acc.x += a2[i];
        acc.y += a1[i];
      }
      st[ty * CV + cv] = make_float2(t1, t2);
    }
    __syncthreads();
    for (int g = tid >> 5; g < p.G; g += kThreads / 32) {
      float t1 = 0.f, t2 = 0.f;
      for (int i = tid & 31; i < DV * TY; i += 32) {
        const float2 t = st[(i / DV) * CV + g * DV + i % DV];
        t1 += t.x;
        t2 += t.y;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        t1 += __shfl_xor_sync(0xffffffffu, t1, off);
        t2 += __shfl_xor_sync(0xffffffffu, t2, off);
      }
      if ((tid & 31) == 0) sg[g] = make_float2(t1 * inv, t2 * inv);
    }
    __syncthreads();
    for (int cv = tx; cv < CV && ty < TY; cv += TX) {
      const int g = cv / DV;
      const float mean = p.mean[n * p.G + g], rstd = p.rstd[n * p.G + g];
      const float2 m = sg[g];
      float w[V], b[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        w[i] = p.w ? p.w[cv * V + i] : 1.f;
        b[i] = p.b ? p.b[cv * V + i] : 0.f;
      }
      for (int64_t r = ty; r < p.S; r += TY) {
        const int64_t at = base + r * p.C + cv * V;
        float v[V], z[V], dy[V];
        load<V>(xs + at, v);
        load<V>(dys + at, dy);
        if (zs) load<V>(zs + at, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (v[i] - mean) * rstd;
          float dz = 0.f;
          const float du = grad_u(fmaf(xh, w[i], b[i]), zs ? z[i] : 0.f, dy[i], p.silu,
                                  zs != nullptr, dz);
          v[i] = rstd * (du * w[i] - m.x - xh * m.y);
          z[i] = dz;
        }
        store<V>(static_cast<T *>(p.dx) + at, v);
        if (zs) store<V>(static_cast<T *>(p.dgate) + at, z);
      }
    }
  }
  __syncthreads();
  for (int c = tid; c < p.C; c += kThreads) {
    float2 a = make_float2(0.f, 0.f);
    for (int r = 0; r < TY; ++r) {
      a.x += sc[r * p.C + c].x;
      a.y += sc[r * p.C + c].y;
    }
    p.part[(size_t)blockIdx.x * 2 * p.C + c] = a.x;
    p.part[(size_t)blockIdx.x * 2 * p.C + p.C + c] = a.y;
  }
}

// dw and db: the sums over the CTAs' partial sums, in their order.
__global__ void gdn_norm_dwdb_kernel(const Params p, int parts) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= 2 * p.C) return;
  float a = 0.f;
  for (int k = 0; k < parts; ++k) a += p.part[(size_t)k * 2 * p.C + i];
  float *to = i < p.C ? p.dw : p.db;
  if (to) to[i < p.C ? i : i - p.C] = a;
}

int ctas(int64_t N) { return (int)(N < 4 * kSMs ? N : 4 * kSMs); }
int tile_rows(int C, int V) { return C / V < kThreads ? kThreads / (C / V) : 1; }

template <typename T, int V>
cudaError_t run(const Params &p, bool backward, cudaStream_t stream) {
  const int CV = p.C / V, TY = tile_rows(p.C, V), grid = ctas(p.N);
  cudaError_t err;
  if (!backward) {
    const size_t bytes = ((size_t)3 * TY * CV + 2 * p.G) * 4;
    err = cudaFuncSetAttribute(gdn_norm_fwd_kernel<T, V>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (err != cudaSuccess) return err;
    gdn_norm_fwd_kernel<T, V><<<grid, kThreads, bytes, stream>>>(p);
    return cudaGetLastError();
  }
  const size_t bytes = ((size_t)TY * CV + p.G + (size_t)TY * p.C) * 8;
  err = cudaFuncSetAttribute(gdn_norm_bwd_kernel<T, V>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (err != cudaSuccess) return err;
  gdn_norm_bwd_kernel<T, V><<<grid, kThreads, bytes, stream>>>(p);
  err = cudaGetLastError();
  if (err != cudaSuccess || (!p.dw && !p.db)) return err;
  gdn_norm_dwdb_kernel<<<(2 * p.C + 255) / 256, 256, 0, stream>>>(p, grid);
  return cudaGetLastError();
}

// 16-byte vectors where a group holds whole ones, else single values.
cudaError_t dispatch(const Params &p, gdn_dtype dtype, bool backward, cudaStream_t stream) {
  if (dtype == GDN_F32)
    return p.D % 4 == 0 ? run<float, 4>(p, backward, stream) : run<float, 1>(p, backward, stream);
  return p.D % 8 == 0 ? run<__nv_bfloat16, 8>(p, backward, stream)
                      : run<__nv_bfloat16, 1>(p, backward, stream);
}

bool aligned16(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }
struct Range {
  const void *p;
  size_t n;
};
bool overlaps(const Range &a, const Range &b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

gdn_status check_sizes(int32_t batch, int32_t spatial, int32_t channels, int32_t groups,
                       gdn_dtype dtype, uint32_t flags) {
  if (batch < 0 || spatial < 0 || channels <= 0 || groups <= 0 || channels % groups)
    return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)GDN_NORM_SILU) return GDN_ERR_INVALID_ARG;
  if (channels > 8192) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

}  // namespace
}  // namespace norm
}  // namespace gdn

extern "C" {

size_t gdn_group_norm_workspace_size(int32_t batch, int32_t spatial, int32_t channels,
                                     int32_t groups) {
  if (batch <= 0 || spatial <= 0 || channels <= 0 || groups <= 0) return 0;
  return (size_t)4 * gdn::norm::kSMs * 2 * channels * 4;
}

gdn_status gdn_group_norm(const void *x, const float *weight, const float *bias, const void *gate,
                          void *y, float *mean, float *rstd, int32_t batch, int32_t spatial,
                          int32_t channels, int32_t groups, float eps, gdn_dtype dtype,
                          uint32_t flags, void *workspace, size_t workspace_bytes, void *stream) {
  using namespace gdn;
  using namespace gdn::norm;
  const gdn_status st = check_sizes(batch, spatial, channels, groups, dtype, flags);
  if (st != GDN_OK) return st;
  if (!(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (batch == 0 || spatial == 0) return GDN_OK;
  if (!x || !y) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {x, weight, bias, gate, y, mean, rstd};
  for (const void *q : ptrs)
    if (q && !aligned16(q)) return GDN_ERR_INVALID_ARG;
  if (!workspace ||
      workspace_bytes < gdn_group_norm_workspace_size(batch, spatial, channels, groups))
    return GDN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDN_ERR_INVALID_ARG;
  const size_t b_x = (size_t)batch * spatial * channels * (dtype == GDN_F32 ? 4 : 2);
  const size_t b_c = (size_t)channels * 4, b_g = (size_t)batch * groups * 4;
  const Range outs[] = {{y, b_x}, {mean, b_g}, {rstd, b_g}, {workspace, workspace_bytes}};
  const Range ins[] = {{x, b_x}, {weight, b_c}, {bias, b_c}, {gate, b_x}};
  for (int i = 0; i < 4; ++i) {
    for (const Range &r : ins)
      if (overlaps(outs[i], r)) return GDN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return GDN_ERR_INVALID_ARG;
  }
  Params p{};
  p.x = x; p.gate = gate; p.w = weight; p.b = bias; p.y = y; p.mean = mean; p.rstd = rstd;
  p.part = static_cast<float *>(workspace);
  p.N = batch; p.S = spatial; p.C = channels; p.G = groups; p.D = channels / groups;
  p.eps = eps; p.silu = (flags & GDN_NORM_SILU) != 0;
  return dispatch(p, dtype, false, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_group_norm_bwd(const void *x, const float *weight, const float *bias,
                              const void *gate, const float *mean, const float *rstd,
                              const void *d_y, void *dx, void *dgate, float *dweight, float *dbias,
                              int32_t batch, int32_t spatial, int32_t channels, int32_t groups,
                              gdn_dtype dtype, uint32_t flags, void *workspace,
                              size_t workspace_bytes, void *stream) {
  using namespace gdn;
  using namespace gdn::norm;
  const gdn_status st = check_sizes(batch, spatial, channels, groups, dtype, flags);
  if (st != GDN_OK) return st;
  const size_t b_c = (size_t)channels * 4;
  if (batch == 0 || spatial == 0) {  // no rows: the channels' sums are empty
    for (float *to : {dweight, dbias}) {
      if (to && !aligned16(to)) return GDN_ERR_INVALID_ARG;
      if (to && cudaMemsetAsync(to, 0, b_c, (cudaStream_t)stream) != cudaSuccess)
        return GDN_ERR_CUDA;
    }
    return GDN_OK;
  }
  if (!x || !mean || !rstd || !d_y || !dx || (gate && !dgate)) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {x, weight, bias, gate, mean, rstd, d_y, dx, dgate, dweight, dbias};
  for (const void *q : ptrs)
    if (q && !aligned16(q)) return GDN_ERR_INVALID_ARG;
  if (!workspace ||
      workspace_bytes < gdn_group_norm_workspace_size(batch, spatial, channels, groups))
    return GDN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDN_ERR_INVALID_ARG;
  const size_t b_x = (size_t)batch * spatial * channels * (dtype == GDN_F32 ? 4 : 2);
  const size_t b_g = (size_t)batch * groups * 4;
  const Range outs[] = {{dx, b_x}, {dgate, gate ? b_x : 0}, {dweight, b_c}, {dbias, b_c},
                        {workspace, workspace_bytes}};
  const Range ins[] = {{x, b_x}, {weight, b_c}, {bias, b_c}, {gate, b_x}, {mean, b_g},
                       {rstd, b_g}, {d_y, b_x}};
  for (int i = 0; i < 5; ++i) {
    for (const Range &r : ins)
      if (overlaps(outs[i], r)) return GDN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return GDN_ERR_INVALID_ARG;
  }
  Params p{};
  p.x = x; p.gate = gate; p.dy = d_y; p.w = weight; p.b = bias; p.dx = dx; p.dgate = dgate;
  p.mean = const_cast<float *>(mean);
  p.rstd = const_cast<float *>(rstd);
  p.dw = dweight; p.db = dbias; p.part = static_cast<float *>(workspace);
  p.N = batch; p.S = spatial; p.C = channels; p.G = groups; p.D = channels / groups;
  p.silu = (flags & GDN_NORM_SILU) != 0;
  return dispatch(p, dtype, true, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
