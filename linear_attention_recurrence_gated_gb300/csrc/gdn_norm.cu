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
constexpr int kParts = 4 * kSMs;   // partial sums of dweight and dbias at most

// Three forms, by the sample's size:
//   rows    S = 1 and a group fits a warp's registers: a group is a power of two
//           of lanes, its values never leave the registers (one read, one write);
//   slabs   fewer samples than SMs: a sample's rows are cut into slabs, one
//           launch sums them up, the next one applies (its reads hit L2 up to
//           some 100 MB);
//   sample  otherwise: one CTA per sample, two passes over it.
struct Params {
  const void *x, *gate, *dy;
  const float *w, *b;
  void *y, *dx, *dgate;
  float *mean, *rstd;        // forward: written (may be NULL); backward: read
  float *dw, *db;
  float *part;               // backward: [parts][2][C] sums of du xh and du
  float *sums;               // slabs: [N][slabs][G] Stat, or two sums
  int64_t N, S;
  int32_t C, G, D, slabs;
  float eps;
  bool silu;
};

template <int V>
__device__ __forceinline__ void load(const float *p, float (&v)[V]) {
  if constexpr (V == 2) {
    const float2 x = *reinterpret_cast<const float2 *>(p);
    v[0] = x.x; v[1] = x.y;
  } else if constexpr (V == 4) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[i];
  }
}
template <int V>
__device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[V]) {
  if constexpr (V == 2) {
    const uint32_t x = *reinterpret_cast<const uint32_t *>(p);
    v[0] = __uint_as_float(x << 16);
    v[1] = __uint_as_float(x & 0xffff0000u);
  } else if constexpr (V == 8) {
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
  if constexpr (V == 2) {
    *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = v[i];
  }
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[V]) {
  if constexpr (V == 2) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[0], v[1]);
    *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(&t);
  } else if constexpr (V == 8) {
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

// sigmoid to the accuracy of the storage type: 2^-22 or so for fp32; for bf16 the
// hardware's exp2 and reciprocal (2^-20 for |z| < 10) disappear in the output's
// own rounding.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(T) == 4) {
    return 1.f / (1.f + expf(-z));
  } else {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
  }
}

// What is applied after the norm: bit 0 SiLU, bit 1 a gate; or (kAny) what the
// arguments say at run time.  The widest vectors have an instance of each.
constexpr int kAny = -1;

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
template <typename T, int M>
__device__ __forceinline__ float activate(float u, float z, const Params &p) {
  const bool silu = M == kAny ? p.silu : (M & 1) != 0;
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  if (silu) u *= sigmoid<T>(u);
  return gated ? u * z * sigmoid<T>(z) : u;
}

// One CTA per sample: statistics in one pass over the sample's rows, the
// normalisation in a second (which finds a small sample in L1 or L2).  Threads
// are tiled over (row, vector of V channels).  Shared memory: a (count, mean,
// m2) triple per channel vector, then mean and rstd per group.
template <typename T, int V, int M>
__global__ void __launch_bounds__(kThreads)
gdn_norm_fwd_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
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
        if (gated) load<V>(zs + at, z);
#pragma unroll
        for (int i = 0; i < V; ++i)
          v[i] = activate<T, M>(fmaf(((v[i] - x0) - mean) * rstd, w[i], b[i]), gated ? z[i] : 0.f, p);
        store<V>(static_cast<T *>(p.y) + at, v);
      }
    }
  }
}

// du of one value, and dz where there is a gate.
template <typename T, int M>
__device__ __forceinline__ float grad_u(float u, float z, float dy, const Params &p, float &dz) {
  const bool silu = M == kAny ? p.silu : (M & 1) != 0;
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  float act = u, dact = 1.f;
  if (silu) {
    const float s = sigmoid<T>(u);
    act = u * s;
    dact = s * (1.f + u * (1.f - s));
  }
  if (gated) {
    const float s = sigmoid<T>(z);
    dz = dy * act * s * (1.f + z * (1.f - s));
    dy *= z * s;
  }
  return dy * dact;
}

// One CTA per sample: the group sums of dxh and dxh xh (and the channels' sums
// of du xh and du) in one pass, dx in a second.  Shared memory: two sums per
// channel vector and row of threads, two means per group, then the channels'
// running sums over the CTA's samples.
template <typename T, int V, int M>
__global__ void __launch_bounds__(kThreads)
gdn_norm_bwd_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
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
        if (gated) load<V>(zs + at, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (v[i] - mean) * rstd;
          float dz;
          const float du = grad_u<T, M>(fmaf(xh, w[i], b[i]), gated ? z[i] : 0.f, dy[i], p, dz);
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
        if (gated) load<V>(zs + at, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (v[i] - mean) * rstd;
          float dz = 0.f;
          const float du = grad_u<T, M>(fmaf(xh, w[i], b[i]), gated ? z[i] : 0.f, dy[i], p, dz);
          v[i] = rstd * (du * w[i] - m.x - xh * m.y);
          z[i] = dz;
        }
        store<V>(static_cast<T *>(p.dx) + at, v);
        if (gated) store<V>(static_cast<T *>(p.dgate) + at, z);
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

// ---- rows: S = 1, a group in the registers of LPG lanes -----------------------
// Thread t holds vectors l, l + LPG, ... (R at most) of group gx of a row; the
// group is the thread's own for every row, so its weights stay in registers.
// The lanes of a group add up by shuffles.  FULL: the group fills its lanes.
template <int R>
__device__ __forceinline__ float lanes_sum(float x, int lpg) {
  for (int off = 1; off < lpg; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
struct RowMap {
  int lpg, groups, rows;   // lanes of a group; groups and rows of a CTA at a time
};
__host__ __device__ inline RowMap row_map(int G, int DV) {
  int lpg = 1;
  while (lpg < 32 && lpg < DV) lpg <<= 1;
  const int slots = kThreads / lpg, groups = G < slots ? G : slots;
  return {lpg, groups, slots / groups};
}

template <typename T, int V, int R, bool FULL, int M>
__global__ void __launch_bounds__(kThreads)
gdn_norm_rows_fwd_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  const int DV = p.D / V, tid = threadIdx.x;
  const RowMap m = row_map(p.G, DV);
  const int l = tid % m.lpg, slot = tid / m.lpg, gx = blockIdx.y * m.groups + slot % m.groups;
  const int ry = slot / m.groups;
  const bool on = ry < m.rows && gx < p.G;
  const T *xs = static_cast<const T *>(p.x), *zs = static_cast<const T *>(p.gate);
  T *ys = static_cast<T *>(p.y);
  const float inv = 1.f / (float)p.D;
  float w[R][V], b[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int cv = l + r * m.lpg, c = gx * p.D + cv * V + i;
      const bool in = on && (FULL || cv < DV);
      w[r][i] = in && p.w ? p.w[c] : 1.f;
      b[r][i] = in && p.b ? p.b[c] : 0.f;
    }
  const int64_t step = (int64_t)gridDim.x * m.rows;
  for (int64_t n0 = (int64_t)blockIdx.x * m.rows; n0 < p.N; n0 += step) {  // uniform: shuffles
    const int64_t n = n0 + ry;
    const bool have = on && n < p.N;
    const int64_t base = n * p.C + (int64_t)gx * p.D;
    float v[R][V], z[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int cv = l + r * m.lpg;
      if (have && (FULL || cv < DV)) {
        load<V>(xs + base + cv * V, v[r]);
        if (gated) load<V>(zs + base + cv * V, z[r]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[r][i] = 0.f;
      }
    }
    // relative to the group's first value: a mean far from zero cancels nothing
    const float x0 = __shfl_sync(0xffffffffu, v[0][0], (tid & 31) - l);
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[r][i] -= x0;
        if (FULL || l + r * m.lpg < DV) s += v[r][i];
      }
    const float mean = lanes_sum<R>(s, m.lpg) * inv;
    s = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[r][i] -= mean;
        if (FULL || l + r * m.lpg < DV) s = fmaf(v[r][i], v[r][i], s);
      }
    const float rstd = rsqrtf(lanes_sum<R>(s, m.lpg) * inv + p.eps);
    if (!have) continue;
    if (l == 0) {
      if (p.mean) p.mean[n * p.G + gx] = x0 + mean;
      if (p.rstd) p.rstd[n * p.G + gx] = rstd;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int cv = l + r * m.lpg;
      if ((FULL || cv < DV)) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          v[r][i] = activate<T, M>(fmaf(v[r][i] * rstd, w[r][i], b[r][i]), gated ? z[r][i] : 0.f, p);
        store<V>(ys + base + cv * V, v[r]);
      }
    }
  }
}

template <typename T, int V, int R, bool FULL, int M>
__global__ void __launch_bounds__(kThreads)
gdn_norm_rows_bwd_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  extern __shared__ __align__(16) float sm[];   // [rows][groups D] float2
  const int DV = p.D / V, tid = threadIdx.x;
  const RowMap m = row_map(p.G, DV);
  const int l = tid % m.lpg, slot = tid / m.lpg, gx = blockIdx.y * m.groups + slot % m.groups;
  const int ry = slot / m.groups;
  const bool on = ry < m.rows && gx < p.G;
  const T *xs = static_cast<const T *>(p.x), *zs = static_cast<const T *>(p.gate),
          *dys = static_cast<const T *>(p.dy);
  const float inv = 1.f / (float)p.D;
  float w[R][V], b[R][V], a1[R][V], a2[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int cv = l + r * m.lpg, c = gx * p.D + cv * V + i;
      const bool in = on && (FULL || cv < DV);
      w[r][i] = in && p.w ? p.w[c] : 1.f;
      b[r][i] = in && p.b ? p.b[c] : 0.f;
      a1[r][i] = a2[r][i] = 0.f;
    }
  const int64_t step = (int64_t)gridDim.x * m.rows;
  for (int64_t n0 = (int64_t)blockIdx.x * m.rows; n0 < p.N; n0 += step) {
    const int64_t n = n0 + ry;
    const bool have = on && n < p.N;
    const int64_t base = n * p.C + (int64_t)gx * p.D;
    float xh[R][V], du[R][V], dz[R][V];
    float mean = 0.f, rstd = 0.f;
    if (have) {
      mean = p.mean[n * p.G + gx];
      rstd = p.rstd[n * p.G + gx];
    }
    float t1 = 0.f, t2 = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int cv = l + r * m.lpg;
      if (have && (FULL || cv < DV)) {
        float z[V];
        load<V>(xs + base + cv * V, xh[r]);
        load<V>(dys + base + cv * V, du[r]);
        if (gated) load<V>(zs + base + cv * V, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          xh[r][i] = (xh[r][i] - mean) * rstd;
          dz[r][i] = 0.f;
          du[r][i] = grad_u<T, M>(fmaf(xh[r][i], w[r][i], b[r][i]), gated ? z[i] : 0.f, du[r][i], p, dz[r][i]);
          a1[r][i] += du[r][i];
          a2[r][i] = fmaf(du[r][i], xh[r][i], a2[r][i]);
          du[r][i] *= w[r][i];
          t1 += du[r][i];
          t2 = fmaf(du[r][i], xh[r][i], t2);
        }
      }
    }
    t1 = lanes_sum<R>(t1, m.lpg) * inv;
    t2 = lanes_sum<R>(t2, m.lpg) * inv;
    if (!have) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int cv = l + r * m.lpg;
      if ((FULL || cv < DV)) {
#pragma unroll
        for (int i = 0; i < V; ++i) du[r][i] = rstd * (du[r][i] - t1 - xh[r][i] * t2);
        store<V>(static_cast<T *>(p.dx) + base + cv * V, du[r]);
        if (gated) store<V>(static_cast<T *>(p.dgate) + base + cv * V, dz[r]);
      }
    }
  }
  // the channels' sums of this CTA, over its rows of threads
  float2 *sc = reinterpret_cast<float2 *>(sm);
  const int width = m.groups * p.D;
  if (on)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int cv = l + r * m.lpg;
      if ((FULL || cv < DV))
#pragma unroll
        for (int i = 0; i < V; ++i)
          sc[(size_t)ry * width + (slot % m.groups) * p.D + cv * V + i] =
              make_float2(a2[r][i], a1[r][i]);
    }
  __syncthreads();
  for (int i = tid; i < width; i += kThreads) {
    const int c = blockIdx.y * width + i;
    if (c >= p.C) break;
    float2 a = make_float2(0.f, 0.f);
    for (int r = 0; r < m.rows; ++r) {
      a.x += sc[(size_t)r * width + i].x;
      a.y += sc[(size_t)r * width + i].y;
    }
    p.part[(size_t)blockIdx.x * 2 * p.C + c] = a.x;
    p.part[(size_t)blockIdx.x * 2 * p.C + p.C + c] = a.y;
  }
}

// ---- slabs: few samples, many rows ---------------------------------------------
// CTA (slab, n) owns rows [slab R, slab R + R) of sample n, threads tiled over
// (row, vector of V channels): TX vectors of one row, TY rows, blockDim.x = TX TY
// up to a whole warp.
constexpr int kSlabThreads = 512;
__host__ __device__ inline int slab_tx(int CV) { return CV < 256 ? CV : 256; }
__host__ __device__ inline int slab_ty(int CV) { return kSlabThreads / slab_tx(CV); }
__device__ __forceinline__ void slab_rows(const Params &p, int64_t &r0, int64_t &r1) {
  const int64_t per = (p.S + p.slabs - 1) / p.slabs;
  r0 = blockIdx.x * per;
  r1 = r0 + per < p.S ? r0 + per : p.S;
}

// The slab's (count, mean relative to the group's first value, m2) of each group.
template <typename T, int V>
__global__ void __launch_bounds__(kSlabThreads)
gdn_norm_slab_stats_kernel(const Params p) {
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = slab_tx(CV), TY = slab_ty(CV);
  const int tx = tid % TX, ty = tid / TX;
  Stat *st = reinterpret_cast<Stat *>(sm);  // [TY][CV]
  int64_t r0, r1;
  slab_rows(p, r0, r1);
  const int64_t base = (int64_t)blockIdx.y * p.S * p.C;
  const T *xs = static_cast<const T *>(p.x) + base;
  for (int cv = tx; cv < CV && ty < TY; cv += TX) {
    const float x0 = to_f32(xs[(cv / DV) * p.D]);
    Stat all = {0.f, 0.f, 0.f};
    for (int64_t ra = r0 + ty; ra < r1; ra += kBlock * TY) {
      float c = 0.f, s1 = 0.f, s2 = 0.f, cnt = 0.f;
#pragma unroll 4
      for (int k = 0; k < kBlock; ++k) {
        const int64_t r = ra + k * TY;
        if (r < r1) {
          float v[V];
          load<V>(xs + r * p.C + cv * V, v);
          if (k == 0) c = v[0];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float d = v[i] - c;
            s1 += d;
            s2 = fmaf(d, d, s2);
          }
          cnt += V;
        }
      }
      const float m = s1 / cnt;
      all = join(all, Stat{cnt, (c - x0) + m, s2 - s1 * m});
    }
    st[ty * CV + cv] = all;
  }
  __syncthreads();
  Stat *out = reinterpret_cast<Stat *>(p.sums) + ((size_t)blockIdx.y * p.slabs + blockIdx.x) * p.G;
  for (int g = tid >> 5; g < p.G; g += blockDim.x / 32) {
    Stat a = {0.f, 0.f, 0.f};
    for (int i = tid & 31; i < DV * TY; i += 32) a = join(a, st[(i / DV) * CV + g * DV + i % DV]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      a = join(a, Stat{__shfl_xor_sync(0xffffffffu, a.n, off),
                       __shfl_xor_sync(0xffffffffu, a.mean, off),
                       __shfl_xor_sync(0xffffffffu, a.m2, off)});
    if ((tid & 31) == 0) out[g] = a;
  }
}

template <typename T, int V, int M>
__global__ void __launch_bounds__(kSlabThreads)
gdn_norm_slab_apply_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = slab_tx(CV), TY = slab_ty(CV);
  const int tx = tid % TX, ty = tid / TX;
  float *smean = sm, *srstd = sm + p.G;
  const int64_t n = blockIdx.y;
  const Stat *in = reinterpret_cast<const Stat *>(p.sums) + (size_t)n * p.slabs * p.G;
  int64_t r0, r1;
  slab_rows(p, r0, r1);
  const int64_t base = n * p.S * p.C;
  const T *xs = static_cast<const T *>(p.x) + base;
  const T *zs = p.gate ? static_cast<const T *>(p.gate) + base : nullptr;
  for (int g = tid >> 5; g < p.G; g += blockDim.x / 32) {
    Stat a = {0.f, 0.f, 0.f};
    for (int i = tid & 31; i < p.slabs; i += 32) a = join(a, in[(size_t)i * p.G + g]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      a = join(a, Stat{__shfl_xor_sync(0xffffffffu, a.n, off),
                       __shfl_xor_sync(0xffffffffu, a.mean, off),
                       __shfl_xor_sync(0xffffffffu, a.m2, off)});
    if ((tid & 31) == 0) {
      smean[g] = a.mean;
      srstd[g] = 1.f / sqrtf(fmaxf(a.m2 / a.n, 0.f) + p.eps);
      if (blockIdx.x == 0) {
        if (p.mean) p.mean[n * p.G + g] = to_f32(xs[g * p.D]) + a.mean;
        if (p.rstd) p.rstd[n * p.G + g] = srstd[g];
      }
    }
  }
  __syncthreads();
  for (int cv = tx; cv < CV && ty < TY; cv += TX) {
    const int g = cv / DV;
    const float x0 = to_f32(xs[g * p.D]), mean = smean[g], rstd = srstd[g];
    float w[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[i] = p.w ? p.w[cv * V + i] : 1.f;
      b[i] = p.b ? p.b[cv * V + i] : 0.f;
    }
#pragma unroll 4
    for (int64_t r = r0 + ty; r < r1; r += TY) {
      const int64_t at = r * p.C + cv * V;
      float v[V], z[V];
      load<V>(xs + at, v);
      if (gated) load<V>(zs + at, z);
#pragma unroll
      for (int i = 0; i < V; ++i)
        v[i] = activate<T, M>(fmaf(((v[i] - x0) - mean) * rstd, w[i], b[i]), gated ? z[i] : 0.f, p);
      store<V>(static_cast<T *>(p.y) + base + at, v);
    }
  }
}

// The slab's channel sums of du xh and du, and its group sums of dxh and dxh xh.
template <typename T, int V, int M>
__global__ void __launch_bounds__(kSlabThreads)
gdn_norm_slab_grads_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = slab_tx(CV), TY = slab_ty(CV);
  const int tx = tid % TX, ty = tid / TX;
  float2 *sc = reinterpret_cast<float2 *>(sm);  // [TY][C]
  const int64_t n = blockIdx.y, base = n * p.S * p.C;
  const T *xs = static_cast<const T *>(p.x) + base, *dys = static_cast<const T *>(p.dy) + base;
  const T *zs = p.gate ? static_cast<const T *>(p.gate) + base : nullptr;
  int64_t r0, r1;
  slab_rows(p, r0, r1);
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
#pragma unroll 4
    for (int64_t r = r0 + ty; r < r1; r += TY) {
      const int64_t at = r * p.C + cv * V;
      float v[V], z[V], dy[V];
      load<V>(xs + at, v);
      load<V>(dys + at, dy);
      if (gated) load<V>(zs + at, z);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (v[i] - mean) * rstd;
        float dz;
        const float du = grad_u<T, M>(fmaf(xh, w[i], b[i]), gated ? z[i] : 0.f, dy[i], p, dz);
        a1[i] += du;
        a2[i] = fmaf(du, xh, a2[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sc[(size_t)ty * p.C + cv * V + i] = make_float2(a2[i], a1[i]);
  }
  __syncthreads();
  const size_t slab = (size_t)n * p.slabs + blockIdx.x;
  for (int c = tid; c < p.C; c += blockDim.x) {
    float2 a = sc[c];
    for (int r = 1; r < TY; ++r) {
      a.x += sc[(size_t)r * p.C + c].x;
      a.y += sc[(size_t)r * p.C + c].y;
    }
    p.part[slab * 2 * p.C + c] = a.x;
    p.part[slab * 2 * p.C + p.C + c] = a.y;
    sc[c] = a;
  }
  __syncthreads();
  float2 *out = reinterpret_cast<float2 *>(p.sums) + slab * p.G;
  for (int g = tid >> 5; g < p.G; g += blockDim.x / 32) {
    float t1 = 0.f, t2 = 0.f;
    for (int i = tid & 31; i < p.D; i += 32) {
      const float wc = p.w ? p.w[g * p.D + i] : 1.f;
      t1 = fmaf(sc[g * p.D + i].y, wc, t1);
      t2 = fmaf(sc[g * p.D + i].x, wc, t2);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      t1 += __shfl_xor_sync(0xffffffffu, t1, off);
      t2 += __shfl_xor_sync(0xffffffffu, t2, off);
    }
    if ((tid & 31) == 0) out[g] = make_float2(t1, t2);
  }
}

template <typename T, int V, int M>
__global__ void __launch_bounds__(kSlabThreads)
gdn_norm_slab_dx_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = slab_tx(CV), TY = slab_ty(CV);
  const int tx = tid % TX, ty = tid / TX;
  float2 *sg = reinterpret_cast<float2 *>(sm);
  const int64_t n = blockIdx.y, base = n * p.S * p.C;
  const T *xs = static_cast<const T *>(p.x) + base, *dys = static_cast<const T *>(p.dy) + base;
  const T *zs = p.gate ? static_cast<const T *>(p.gate) + base : nullptr;
  const float inv = 1.f / ((float)p.S * (float)p.D);
  int64_t r0, r1;
  slab_rows(p, r0, r1);
  const float2 *in = reinterpret_cast<const float2 *>(p.sums) + (size_t)n * p.slabs * p.G;
  for (int g = tid >> 5; g < p.G; g += blockDim.x / 32) {
    float t1 = 0.f, t2 = 0.f;
    for (int i = tid & 31; i < p.slabs; i += 32) {
      const float2 t = in[(size_t)i * p.G + g];
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
#pragma unroll 4
    for (int64_t r = r0 + ty; r < r1; r += TY) {
      const int64_t at = r * p.C + cv * V;
      float v[V], z[V], dy[V];
      load<V>(xs + at, v);
      load<V>(dys + at, dy);
      if (gated) load<V>(zs + at, z);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (v[i] - mean) * rstd;
        float dz = 0.f;
        const float du = grad_u<T, M>(fmaf(xh, w[i], b[i]), gated ? z[i] : 0.f, dy[i], p, dz);
        v[i] = rstd * (du * w[i] - m.x - xh * m.y);
        z[i] = dz;
      }
      store<V>(static_cast<T *>(p.dx) + base + at, v);
      if (gated) store<V>(static_cast<T *>(p.dgate) + base + at, z);
    }
  }
}

// dw and db: 32 columns a CTA, its 32 rows of threads over the partial sums, both
// in a fixed order.
__global__ void __launch_bounds__(1024) gdn_norm_dwdb_kernel(const Params p, int parts) {
  __shared__ float sm[32][33];
  const int tx = threadIdx.x, ty = threadIdx.y, i = blockIdx.x * 32 + tx;
  float a = 0.f;
  if (i < 2 * p.C)
#pragma unroll 4
    for (int k = ty; k < parts; k += 32) a += p.part[(size_t)k * 2 * p.C + i];
  sm[ty][tx] = a;
  __syncthreads();
  if (ty) return;
#pragma unroll
  for (int k = 1; k < 32; ++k) a += sm[k][tx];
  float *to = i < p.C ? p.dw : p.db;
  if (i < 2 * p.C && to) to[i < p.C ? i : i - p.C] = a;
}

int tile_rows(int C, int V) { return C / V < kThreads ? kThreads / (C / V) : 1; }
// Slabs of a sample when there are few: four CTAs for each SM, four rows of every
// row of threads at least.
int slab_count(int64_t N, int64_t S, int C, int V) {
  const int64_t want = (kParts + N - 1) / N, most = S / (4 * slab_ty(C / V));
  const int64_t n = want < most ? want : most;
  return n < 1 ? 1 : (int)n;
}
bool use_slabs(int64_t N, int64_t S) { return N < kSMs && S > 1; }

template <typename K>
cudaError_t go(K kernel, dim3 grid, size_t bytes, const Params &p, cudaStream_t stream,
               int threads = kThreads) {
  const cudaError_t err =
      bytes > 48 * 1024
          ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)
          : cudaSuccess;
  if (err != cudaSuccess) return err;
  kernel<<<grid, threads, bytes, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t sum_parts(const Params &p, int parts, cudaStream_t stream) {
  if (!p.dw && !p.db) return cudaSuccess;
  gdn_norm_dwdb_kernel<<<(2 * p.C + 31) / 32, dim3(32, 32), 0, stream>>>(p, parts);
  return cudaGetLastError();
}

template <typename T, int V, int R, bool FULL, int M>
cudaError_t run_rows(const Params &p, bool backward, cudaStream_t stream) {
  const RowMap m = row_map(p.G, p.D / V);
  const int gy = (p.G + m.groups - 1) / m.groups;
  int64_t gx = (p.N + m.rows - 1) / m.rows;
  const int64_t most = backward ? (kParts / 2 + gy - 1) / gy : 8 * kSMs;
  if (gx > most) gx = most;
  const dim3 grid((unsigned)gx, gy);
  if (!backward) return go(gdn_norm_rows_fwd_kernel<T, V, R, FULL, M>, grid, 0, p, stream);
  const size_t bytes = (size_t)8 * m.rows * m.groups * p.D;
  const cudaError_t err = go(gdn_norm_rows_bwd_kernel<T, V, R, FULL, M>, grid, bytes, p, stream);
  return err == cudaSuccess ? sum_parts(p, (int)gx, stream) : err;
}

template <typename T, int V, int M>
cudaError_t run_slabs(Params p, bool backward, cudaStream_t stream) {
  const int CV = p.C / V, TY = slab_ty(CV), threads = (slab_tx(CV) * TY + 31) / 32 * 32;
  p.slabs = slab_count(p.N, p.S, p.C, V);
  const int parts = (int)p.N * p.slabs;
  p.sums = p.part + (backward ? (size_t)parts * 2 * p.C : 0);
  const dim3 grid(p.slabs, (unsigned)p.N);
  cudaError_t err;
  if (!backward) {
    err = go(gdn_norm_slab_stats_kernel<T, V>, grid, (size_t)12 * TY * CV, p, stream, threads);
    return err != cudaSuccess
               ? err
               : go(gdn_norm_slab_apply_kernel<T, V, M>, grid, (size_t)8 * p.G, p, stream, threads);
  }
  err = go(gdn_norm_slab_grads_kernel<T, V, M>, grid, (size_t)8 * TY * p.C, p, stream, threads);
  if (err == cudaSuccess)
    err = go(gdn_norm_slab_dx_kernel<T, V, M>, grid, (size_t)8 * p.G, p, stream, threads);
  return err == cudaSuccess ? sum_parts(p, parts, stream) : err;
}

// The widest vectors: an instance for each activation.
template <typename T, int V, int M>
cudaError_t run_wide(const Params &p, bool backward, cudaStream_t stream) {
  return p.S == 1 ? run_rows<T, V, 1, true, M>(p, backward, stream)
                  : run_slabs<T, V, M>(p, backward, stream);
}

template <typename T, int V, bool WIDE>
cudaError_t run(const Params &p, bool backward, cudaStream_t stream) {
  const int CV = p.C / V, DV = p.D / V, TY = tile_rows(p.C, V);
  if constexpr (WIDE) {
    const bool full = p.S == 1 && DV <= 32 && (DV & (DV - 1)) == 0;
    if (full || use_slabs(p.N, p.S)) {
      const int mode = (p.silu ? 1 : 0) | (p.gate ? 2 : 0);
      return mode == 0   ? run_wide<T, V, 0>(p, backward, stream)
             : mode == 1 ? run_wide<T, V, 1>(p, backward, stream)
             : mode == 2 ? run_wide<T, V, 2>(p, backward, stream)
                         : run_wide<T, V, 3>(p, backward, stream);
    }
  }
  if (p.S == 1 && DV <= 32) return run_rows<T, V, 1, false, kAny>(p, backward, stream);
  if (p.S == 1 && DV <= 128) return run_rows<T, V, 4, false, kAny>(p, backward, stream);
  if constexpr (!WIDE)
    if (use_slabs(p.N, p.S)) return run_slabs<T, V, kAny>(p, backward, stream);
  const int grid = (int)(p.N < kParts ? p.N : kParts);
  if (!backward)
    return go(gdn_norm_fwd_kernel<T, V, kAny>, grid, ((size_t)3 * TY * CV + 2 * p.G) * 4, p, stream);
  const cudaError_t err = go(gdn_norm_bwd_kernel<T, V, kAny>, grid,
                             ((size_t)TY * CV + p.G + (size_t)TY * p.C) * 8, p, stream);
  return err == cudaSuccess ? sum_parts(p, grid, stream) : err;
}

// 16-byte vectors where a group holds whole ones, else pairs or single values.
cudaError_t dispatch(const Params &p, gdn_dtype dtype, bool backward, cudaStream_t stream) {
  if (dtype == GDN_F32)
    return p.D % 4 == 0   ? run<float, 4, true>(p, backward, stream)
           : p.D % 2 == 0 ? run<float, 2, false>(p, backward, stream)
                          : run<float, 1, false>(p, backward, stream);
  return p.D % 8 == 0   ? run<__nv_bfloat16, 8, true>(p, backward, stream)
         : p.D % 2 == 0 ? run<__nv_bfloat16, 2, false>(p, backward, stream)
                        : run<__nv_bfloat16, 1, false>(p, backward, stream);
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
  // partial sums of dweight and dbias, and of the groups of every slab
  using namespace gdn::norm;
  const size_t parts = use_slabs(batch, spatial) ? (size_t)(kParts + batch) : (size_t)kParts;
  return parts * ((size_t)8 * channels + (size_t)12 * groups);
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
