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
// The gradients' sums over rows and samples are taken in blocks of kSum, whose results
// are added up: one plain sum over the rows of a CTA was off by 4e-5 for 3449 rows of
// equal terms.  Sums over lanes, threads and CTAs run over 512 values at most.
#include <stdint.h>

#include "gdn_internal.cuh"
#include "gdn_launch.cuh"

namespace gdn {
namespace norm {
namespace {

constexpr int kThreads = 256;
constexpr int kSMs = 152;
constexpr int kBlock = 16;   // rows summed by a thread before it joins them
constexpr int kSum = 128;    // rows, or samples, that one plain sum of gradients runs over
constexpr int kParts = 4 * kSMs;   // partial sums of dweight and dbias (slabs: one each)

// Three forms, by the sample's size:
//   rows    S = 1 and a group fits a warp's registers: a group is a power of two
//           of lanes, its values never leave the registers (one read, one write);
//   slabs   few or large samples: a sample's rows are cut into slabs, one launch sums
//           them up, the next one applies, from the last rows to the first (some of
//           which L2 still holds);
//   sample  otherwise: one CTA per sample, two passes over it.
// All are bound by memory (forward: x, gate and y once; the slabs' backward pass reads x
// and dy twice).  Measured, bf16: rows, gated, [32768, 1, 1024], 201 MB, 35.9 us (5.6
// TB/s; a CTA for each place on the SMs: a second wave cost 1 us), backward, 336 MB, 82
// us (no row is sent for ahead of its turn); slabs backward with SiLU, [4, 4096, 1280],
// 126 MB, 41.5 us (two passes at 5 TB/s; without its arithmetic 34 us: five warps a
// scheduler cover most of it; at 64 registers a thread the widest bf16 instances spill,
// 32 bytes here, 86 and 40 in the two passes with SiLU and a gate).  One CTA a sample is
// left for many small samples and for groups beyond a warp's registers (gated, [16384, 1,
// 2048] as one group: 171 us, backward 299, six times its bytes).
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
template <typename T>
__device__ __forceinline__ float activate(float u, float z, const Params &p) {
  if (p.silu) u *= sigmoid<T>(u);
  return p.gate ? u * z * sigmoid<T>(z) : u;
}

// ---- pairs of values: two lanes of packed fp32 arithmetic ----------------------
using Pair = uint64_t;
__device__ __forceinline__ Pair pk(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 un(Pair x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair both(float x) { return pk(x, x); }

// V values as they lie in memory, unpacked when they are used.  A pair of a
// single value (V = 1) has a zero beside it.
template <typename T, int V>
struct Raw;
template <int V>
struct Raw<float, V> {
  float v[V];
  __device__ __forceinline__ void load(const float *p) {
    if constexpr (V == 4) {
      const float4 x = *reinterpret_cast<const float4 *>(p);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else if constexpr (V == 2) {
      const float2 x = *reinterpret_cast<const float2 *>(p);
      v[0] = x.x; v[1] = x.y;
    } else {
      v[0] = *p;
    }
  }
  __device__ __forceinline__ Pair at(int i) const { return pk(v[2 * i], V > 1 ? v[(2 * i + 1) % V] : 0.f); }
};
template <int V>
struct Raw<__nv_bfloat16, V> {
  uint32_t v[(V + 1) / 2];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    if constexpr (V == 8) {
      const uint4 x = *reinterpret_cast<const uint4 *>(p);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else if constexpr (V == 2) {
      v[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
      v[0] = *reinterpret_cast<const uint16_t *>(p);
    }
  }
  __device__ __forceinline__ Pair at(int i) const {
    return pk(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
  }
};
template <typename T, int V>
__device__ __forceinline__ void put(T *p, const Pair (&x)[(V + 1) / 2]) {
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = i & 1 ? un(x[i / 2]).y : un(x[i / 2]).x;
  store<V>(p, v);
}

template <typename T>
__device__ __forceinline__ Pair sigmoid2(Pair z) {
  if constexpr (sizeof(T) == 4) {
    const float2 x = un(z);
    return pk(sigmoid<T>(x.x), sigmoid<T>(x.y));
  } else {
    const float2 x = un(mul2(z, both(-1.4426950408889634f)));
    float e0, e1, r0, r1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(x.y));
    const float2 d = un(add2(pk(e0, e1), both(1.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d.y));
    return pk(r0, r1);
  }
}
template <typename T, int M>
__device__ __forceinline__ Pair activate2(Pair u, Pair z, const Params &p) {
  const bool silu = M == kAny ? p.silu : (M & 1) != 0;
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  if (silu) u = mul2(u, sigmoid2<T>(u));
  return gated ? mul2(u, mul2(z, sigmoid2<T>(z))) : u;
}
// silu'(x) = s (1 + x (1 - s)), s = sigmoid(x)
__device__ __forceinline__ Pair dsilu2(Pair x, Pair s) {
  return mul2(s, fma2(x, fma2(s, both(-1.f), both(1.f)), both(1.f)));
}
template <typename T, int M>
__device__ __forceinline__ Pair grad_u2(Pair u, Pair z, Pair dy, const Params &p, Pair &dz) {
  const bool silu = M == kAny ? p.silu : (M & 1) != 0;
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  Pair act = u, dact = both(1.f);
  if (silu) {
    const Pair s = sigmoid2<T>(u);
    act = mul2(u, s);
    dact = dsilu2(u, s);
  }
  if (gated) {
    const Pair s = sigmoid2<T>(z);
    dz = mul2(mul2(dy, act), dsilu2(z, s));
    dy = mul2(dy, mul2(z, s));
  }
  return silu ? mul2(dy, dact) : dy;
}
// V weights from channel c on (a missing vector reads as `other`).
template <int V>
__device__ __forceinline__ void weights(const float *w, int c, bool in, float other,
                                        Pair (&to)[(V + 1) / 2]) {
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = other;
  if (in && w) {
    if constexpr (V % 4 == 0) {   // (c is a multiple of V)
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(w + c + i);
        v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = w[c + i];
    }
  }
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) to[i] = pk(v[2 * i], 2 * i + 1 < V ? v[(2 * i + 1) % V] : 0.f);
}

// One CTA per sample: statistics in one pass over the sample's rows, the
// normalisation in a second (which finds a small sample in L1 or L2).  Threads
// are tiled over (row, vector of V channels).  Shared memory: a (count, mean,
// m2) triple per channel vector, then mean and rstd per group.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
gdn_norm_fwd_kernel(const Params p) {
  const bool gated = p.gate != nullptr;
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
          v[i] = activate<T>(fmaf(((v[i] - x0) - mean) * rstd, w[i], b[i]), gated ? z[i] : 0.f, p);
        store<V>(static_cast<T *>(p.y) + at, v);
      }
    }
  }
}

// du of one value, and dz where there is a gate.
template <typename T>
__device__ __forceinline__ float grad_u(float u, float z, float dy, const Params &p, float &dz) {
  float act = u, dact = 1.f;
  if (p.silu) {
    const float s = sigmoid<T>(u);
    act = u * s;
    dact = s * (1.f + u * (1.f - s));
  }
  if (p.gate) {
    const float s = sigmoid<T>(z);
    dz = dy * act * s * (1.f + z * (1.f - s));
    dy *= z * s;
  }
  return dy * dact;
}

// One CTA per sample: the group sums of dxh and dxh xh (and the channels' sums
// of du xh and du) in one pass, dx in a second.  Shared memory: two sums per
// channel vector and row of threads, two means per group, then the channels'
// running sums over the CTA's samples.  LONG: a thread has more than kSum rows of a sample.
template <typename T, int V, bool LONG>
__global__ void __launch_bounds__(kThreads)
gdn_norm_bwd_kernel(const Params p) {
  const bool gated = p.gate != nullptr;
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
  // the channels' running sums into the CTA's partial ones
  float *const part = p.part + (size_t)blockIdx.x * 2 * p.C;
  int samples = 0;
  bool fresh = true;
  const auto close = [&]() {
    __syncthreads();
    for (int c = tid; c < p.C; c += kThreads) {
      float2 a = make_float2(0.f, 0.f);
      for (int r = 0; r < TY; ++r) {
        a.x += sc[r * p.C + c].x;
        a.y += sc[r * p.C + c].y;
        sc[r * p.C + c] = make_float2(0.f, 0.f);
      }
      part[c] = fresh ? a.x : part[c] + a.x;
      part[p.C + c] = fresh ? a.y : part[p.C + c] + a.y;
    }
    fresh = false;
    samples = 0;
  };
  const float inv = 1.f / ((float)p.S * (float)p.D);
  for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
    if (samples == kSum) close();
    ++samples;
    const int64_t base = n * p.S * p.C;
    __syncthreads();
    for (int cv = tx; cv < CV && ty < TY; cv += TX) {
      const int g = cv / DV;
      const float mean = p.mean[n * p.G + g], rstd = p.rstd[n * p.G + g];
      float w[V], b[V], a1[V], a2[V], t1 = 0.f, t2 = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        w[i] = p.w ? p.w[cv * V + i] : 1.f;
        b[i] = p.b ? p.b[cv * V + i] : 0.f;
        a1[i] = a2[i] = 0.f;
      }
      const auto close_rows = [&]() {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          t1 = fmaf(a1[i], w[i], t1);
          t2 = fmaf(a2[i], w[i], t2);
          float2 &acc = sc[ty * p.C + cv * V + i];
          acc.x += a2[i];
          acc.y += a1[i];
          a1[i] = a2[i] = 0.f;
        }
      };
      int summed = 0;
      for (int64_t r = ty; r < p.S; r += TY) {
        if (LONG && summed++ == kSum) {
          close_rows();
          summed = 1;
        }
        const int64_t at = base + r * p.C + cv * V;
        float v[V], z[V], dy[V];
        load<V>(xs + at, v);
        load<V>(dys + at, dy);
        if (gated) load<V>(zs + at, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (v[i] - mean) * rstd;
          float dz;
          const float du = grad_u<T>(fmaf(xh, w[i], b[i]), gated ? z[i] : 0.f, dy[i], p, dz);
          a1[i] += du;
          a2[i] = fmaf(du, xh, a2[i]);
        }
      }
      close_rows();
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
          const float du = grad_u<T>(fmaf(xh, w[i], b[i]), gated ? z[i] : 0.f, dy[i], p, dz);
          v[i] = rstd * (du * w[i] - m.x - xh * m.y);
          z[i] = dz;
        }
        store<V>(static_cast<T *>(p.dx) + at, v);
        if (gated) store<V>(static_cast<T *>(p.dgate) + at, z);
      }
    }
  }
  close();
}

// dw and db: W columns for a CTA, its rows of threads over the partial sums, both in
// a fixed order.
template <int W>
__device__ __forceinline__ void sum_columns(const Params &p, int parts, int col0, float *sm) {
  const int tx = threadIdx.x % W, ty = threadIdx.x / W, rows = blockDim.x / W, i = col0 + tx;
  float a = 0.f;
  if (i < 2 * p.C)
    for (int k0 = ty; k0 < parts; k0 += kSum * rows) {
      float t = 0.f;
#pragma unroll 4
      for (int k = k0; k < parts && k < k0 + kSum * rows; k += rows)
        t += p.part[(size_t)k * 2 * p.C + i];
      a += t;
    }
  sm[ty * (W + 1) + tx] = a;
  __syncthreads();
  if (ty == 0) {
#pragma unroll 4
    for (int k = 1; k < rows; ++k) a += sm[k * (W + 1) + tx];
    float *to = i < p.C ? p.dw : p.db;
    if (i < 2 * p.C && to) to[i < p.C ? i : i - p.C] = a;
  }
  __syncthreads();
}
__global__ void __launch_bounds__(1024) gdn_norm_dwdb_kernel(const Params p, int parts) {
  __shared__ float sm[32 * 33];
  sum_columns<32>(p, parts, 32 * blockIdx.x, sm);
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
  constexpr int NP = (V + 1) / 2;
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  const int DV = p.D / V, tid = threadIdx.x;
  const RowMap m = row_map(p.G, DV);
  const int l = tid % m.lpg, slot = tid / m.lpg, gx = blockIdx.y * m.groups + slot % m.groups;
  const int ry = slot / m.groups;
  const bool on = ry < m.rows && gx < p.G;
  const T *xs = static_cast<const T *>(p.x), *zs = static_cast<const T *>(p.gate);
  T *ys = static_cast<T *>(p.y);
  const float inv = 1.f / (float)p.D;
  Pair w[R][NP], b[R][NP];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int cv = l + r * m.lpg;
    weights<V>(p.w, gx * p.D + cv * V, on && cv < DV, 1.f, w[r]);
    weights<V>(p.b, gx * p.D + cv * V, on && cv < DV, 0.f, b[r]);
  }
  const int64_t step = (int64_t)gridDim.x * m.rows;
  const auto read = [&](int64_t n, Raw<T, V> (&x)[R], Raw<T, V> (&z)[R]) {
    if (!on || n >= p.N) return;
    const int64_t base = n * p.C + (int64_t)gx * p.D;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int cv = l + r * m.lpg;
      if (FULL || cv < DV) {
        x[r].load(xs + base + cv * V);
        if (gated) z[r].load(zs + base + cv * V);
      }
    }
  };
  Raw<T, V> x[R] = {}, z[R] = {}, x_next[R] = {}, z_next[R] = {};
  int64_t n = (int64_t)blockIdx.x * m.rows + ry;
  read(n, x, z);
  // (a uniform count of turns: the lanes of a warp shuffle together)
  for (int64_t n0 = (int64_t)blockIdx.x * m.rows; n0 < p.N; n0 += step, n += step) {
    read(n + step, x_next, z_next);   // the next row is on its way
    const bool have = on && n < p.N;
    // relative to the group's first value: a mean far from zero cancels nothing
    const float first = un(x[0].at(0)).x;
    const float x0 = __shfl_sync(0xffffffffu, first, (tid & 31) - l);
    Pair v[R][NP], s = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (FULL || l + r * m.lpg < DV)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          v[r][i] = add2(x[r].at(i), pk(-x0, V > 1 ? -x0 : 0.f));
          s = add2(s, v[r][i]);
        }
    float2 t = un(s);
    const float mean = lanes_sum<R>(t.x + t.y, m.lpg) * inv;
    s = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (FULL || l + r * m.lpg < DV)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          v[r][i] = add2(v[r][i], pk(-mean, V > 1 ? -mean : 0.f));
          s = fma2(v[r][i], v[r][i], s);
        }
    t = un(s);
    const float rstd = rsqrtf(lanes_sum<R>(t.x + t.y, m.lpg) * inv + p.eps);
    if (have) {
      if (l == 0) {
        if (p.mean) p.mean[n * p.G + gx] = x0 + mean;
        if (p.rstd) p.rstd[n * p.G + gx] = rstd;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int cv = l + r * m.lpg;
        if (FULL || cv < DV) {
#pragma unroll
          for (int i = 0; i < NP; ++i)
            v[r][i] = activate2<T, M>(fma2(mul2(v[r][i], both(rstd)), w[r][i], b[r][i]), z[r].at(i), p);
          put<T, V>(ys + n * p.C + (int64_t)gx * p.D + cv * V, v[r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = x_next[r];
      z[r] = z_next[r];
    }
  }
}

template <typename T, int V, int R, bool FULL, int M>
__global__ void __launch_bounds__(kThreads)
gdn_norm_rows_bwd_kernel(const Params p) {
  extern __shared__ __align__(16) float sm[];   // [rows][groups D] float2
  constexpr int NP = (V + 1) / 2;
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  const int DV = p.D / V, tid = threadIdx.x;
  const RowMap m = row_map(p.G, DV);
  const int l = tid % m.lpg, slot = tid / m.lpg, gx = blockIdx.y * m.groups + slot % m.groups;
  const int ry = slot / m.groups;
  const bool on = ry < m.rows && gx < p.G;
  const T *xs = static_cast<const T *>(p.x), *zs = static_cast<const T *>(p.gate),
          *dys = static_cast<const T *>(p.dy);
  const float inv = 1.f / (float)p.D;
  Pair w[R][NP], b[R][NP], a1[R][NP], a2[R][NP];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int cv = l + r * m.lpg;
    weights<V>(p.w, gx * p.D + cv * V, on && cv < DV, 1.f, w[r]);
    weights<V>(p.b, gx * p.D + cv * V, on && cv < DV, 0.f, b[r]);
#pragma unroll
    for (int i = 0; i < NP; ++i) a1[r][i] = a2[r][i] = 0;
  }
  // the thread's sums into their place in shared memory
  float2 *sc = reinterpret_cast<float2 *>(sm);
  const int width = m.groups * p.D;
  bool fresh = true;
  const auto close = [&]() {
    if (on)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int cv = l + r * m.lpg;
        if (FULL || cv < DV)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 q1 = un(a1[r][i / 2]), q2 = un(a2[r][i / 2]);
            float2 &to = sc[(size_t)ry * width + (slot % m.groups) * p.D + cv * V + i];
            float2 sum = i & 1 ? make_float2(q2.y, q1.y) : make_float2(q2.x, q1.x);
            if (!fresh) sum.x += to.x, sum.y += to.y;
            to = sum;
          }
#pragma unroll
        for (int i = 0; i < NP; ++i) a1[r][i] = a2[r][i] = 0;
      }
    fresh = false;
  };
  const int64_t step = (int64_t)gridDim.x * m.rows;
  int64_t n0 = (int64_t)blockIdx.x * m.rows;
#pragma unroll 1
  for (int64_t stop = n0 + kSum * step;; stop += kSum * step) {
    for (const int64_t end = stop < p.N ? stop : p.N; n0 < end; n0 += step) {
      const int64_t n = n0 + ry;
      const bool have = on && n < p.N;
      const int64_t base = n * p.C + (int64_t)gx * p.D;
      Raw<T, V> x[R], dy[R], z[R];
      float mean = 0.f, rstd = 0.f;
      if (have) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int cv = l + r * m.lpg;
          if (FULL || cv < DV) {
            x[r].load(xs + base + cv * V);
            dy[r].load(dys + base + cv * V);
            if (gated) z[r].load(zs + base + cv * V);
          }
        }
        mean = p.mean[n * p.G + gx];
        rstd = p.rstd[n * p.G + gx];
      }
      Pair xh[R][NP], du[R][NP], t1 = 0, t2 = 0;
      if (have)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int cv = l + r * m.lpg;
          if (FULL || cv < DV) {
            Pair dz[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              xh[r][i] = mul2(add2(x[r].at(i), both(-mean)), both(rstd));
              dz[i] = 0;
              du[r][i] = grad_u2<T, M>(fma2(xh[r][i], w[r][i], b[r][i]),
                                       gated ? z[r].at(i) : 0, dy[r].at(i), p, dz[i]);
              a1[r][i] = add2(a1[r][i], du[r][i]);
              a2[r][i] = fma2(du[r][i], xh[r][i], a2[r][i]);
              du[r][i] = mul2(du[r][i], w[r][i]);
              t1 = add2(t1, du[r][i]);
              t2 = fma2(du[r][i], xh[r][i], t2);
            }
            if (gated) put<T, V>(static_cast<T *>(p.dgate) + base + cv * V, dz);
          }
        }
      // (a single value's empty second lane: du and w are zero there)
      const float2 u1 = un(t1), u2 = un(t2);
      const float c1 = lanes_sum<R>(u1.x + u1.y, m.lpg) * inv,
                  c2 = lanes_sum<R>(u2.x + u2.y, m.lpg) * inv;
      if (have)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int cv = l + r * m.lpg;
          if (FULL || cv < DV) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
              du[r][i] = mul2(both(rstd), fma2(xh[r][i], both(-c2), add2(du[r][i], both(-c1))));
            put<T, V>(static_cast<T *>(p.dx) + base + cv * V, du[r]);
          }
        }
    }
    close();
    if (n0 >= p.N) break;
  }
  // the channels' sums of this CTA, over its rows of threads
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

// A thread's rows first, first + step, ... below r1, of its vector at channel c: `run`
// calls `use(at, x, dy, z)` for each, `at` its offset in a sample; with `down` they are
// the mirror images of these rows in the slab.  With 16-byte
// vectors the rows come through a ring in shared memory, kDepth ahead: every
// thread copies its own vectors and reads only those, so no thread waits for
// another, and some 100 KB are on their way to an SM at any time.  `start` sends for
// the first ones.  (With the next two rows in registers instead, a backward pass over
// [4, 4096, 1280] took 79 us, each thread going through 14 latencies of memory one
// after the other.)
constexpr int kDepth = 4;
template <typename T, int V>
constexpr bool kRing = sizeof(T) * V == 16;
template <typename T, int V>
size_t ring_bytes(int threads, int tensors) {
  return kRing<T, V> ? (size_t)16 * kDepth * tensors * threads : 0;
}
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
template <typename T, int V, bool DY>
struct Rows {
  const T *xs, *dys, *zs;
  bool gated;
  int n;               // rows
  int64_t at, by;      // offset of the first one's channel 0, from one to the next
  uint4 *mine;         // [stage][tensor][thread]
  uint32_t to;
  int th;
  __device__ __forceinline__ Rows(uint4 *ring, const T *xs, const T *dys, const T *zs, bool gated,
                                  int64_t C, int64_t r0, int64_t r1, int64_t first, int64_t step,
                                  bool down)
      : xs(xs), dys(dys), zs(zs), gated(gated),
        n(first < r1 ? (int)((r1 - first + step - 1) / step) : 0),
        at((down ? r0 + r1 - 1 - first : first) * C), by(down ? -step * C : step * C),
        mine(ring + threadIdx.x), to((uint32_t)__cvta_generic_to_shared(mine)),
        th(blockDim.x) {}
  __device__ __forceinline__ int tensors() const { return 1 + (DY ? 1 : 0) + (gated ? 1 : 0); }
  __device__ __forceinline__ void ask(bool there, int64_t o, int stage) const {
    if (there) {
      uint32_t a = to + 16 * th * tensors() * stage;
      copy16(a, xs + o);
      if (DY) copy16(a += 16 * th, dys + o);
      if (gated) copy16(a += 16 * th, zs + o);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void start(int c) const {
    if constexpr (kRing<T, V>) {
#pragma unroll
      for (int k = 0; k < kDepth - 1; ++k) ask(k < n, at + k * by + c, k);
    }
  }
  template <typename F>
  __device__ __forceinline__ void run(int c, F use) const {
    int64_t o = at + c;
    if constexpr (kRing<T, V>) {
      int64_t next = o + (kDepth - 1) * by;
      int stage = 0, ahead = kDepth - 1;
#pragma unroll 1
      for (int i = 0; i < n; ++i, o += by, next += by) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
        ask(i + kDepth - 1 < n, next, ahead);
        const uint4 *from = mine + th * tensors() * stage;
        Raw<T, V> x, dy = {}, z = {};
        x.load(reinterpret_cast<const T *>(from));
        if (DY) dy.load(reinterpret_cast<const T *>(from += th));
        if (gated) z.load(reinterpret_cast<const T *>(from += th));
        use(i, o, x, dy, z);
        ahead = stage;
        stage = stage + 1 == kDepth ? 0 : stage + 1;
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
#pragma unroll 4
      for (int i = 0; i < n; ++i, o += by) {
        Raw<T, V> x, dy = {}, z = {};
        x.load(xs + o);
        if (DY) dy.load(dys + o);
        if (gated) z.load(zs + o);
        use(i, o, x, dy, z);
      }
    }
  }
};
// The second launch of a pair sends for its first rows (inputs of both) beside the
// first; what that has written is read after `wait_first`.

// The slab's (count, mean relative to the group's first value, m2) of each group.
template <typename T, int V>
__global__ void __launch_bounds__(kSlabThreads, 2)
gdn_norm_slab_stats_kernel(const Params p) {
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = slab_tx(CV), TY = slab_ty(CV);
  const int tx = tid % TX, ty = tid / TX;
  Stat *st = reinterpret_cast<Stat *>(sm);  // [TY][CV]
  uint4 *ring = reinterpret_cast<uint4 *>(sm + ((size_t)3 * TY * CV + 3) / 4 * 4);
  int64_t r0, r1;
  slab_rows(p, r0, r1);
  const int64_t base = (int64_t)blockIdx.y * p.S * p.C;
  const T *xs = static_cast<const T *>(p.x) + base;
  const Rows<T, V, false> rows(ring, xs, xs, nullptr, false, p.C, r0, r1, r0 + ty, TY, false);
  let_second();
  for (int cv = tx; cv < CV && ty < TY; cv += TX) {
    rows.start(cv * V);
    const float x0 = to_f32(xs[(cv / DV) * p.D]);
    Stat all = {0.f, 0.f, 0.f};
    float c = 0.f, cnt = 0.f;
    Pair s1 = 0, s2 = 0;
    const auto close = [&]() {
      const float2 t1 = un(s1), t2 = un(s2);
      const float t = t1.x + t1.y, m = t / cnt;
      all = join(all, Stat{cnt, (c - x0) + m, (t2.x + t2.y) - t * m});
      cnt = 0.f;
      s1 = s2 = 0;
    };
    rows.run(
        cv * V, [&](int, int64_t, const Raw<T, V> &x, const Raw<T, V> &, const Raw<T, V> &) {
          if (cnt == 0.f) c = un(x.at(0)).x;
#pragma unroll
          for (int i = 0; i < (V + 1) / 2; ++i) {
            const Pair d = add2(x.at(i), pk(-c, V > 1 ? -c : 0.f));
            s1 = add2(s1, d);
            s2 = fma2(d, d, s2);
          }
          cnt += V;
          if (cnt == (float)(kBlock * V)) close();
        });
    if (cnt > 0.f) close();
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
__global__ void __launch_bounds__(kSlabThreads, 2)
gdn_norm_slab_apply_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = slab_tx(CV), TY = slab_ty(CV);
  const int tx = tid % TX, ty = tid / TX;
  float *smean = sm, *srstd = sm + p.G;
  uint4 *ring = reinterpret_cast<uint4 *>(sm + (2 * p.G + 3) / 4 * 4);
  const int64_t n = blockIdx.y;
  const Stat *in = reinterpret_cast<const Stat *>(p.sums) + (size_t)n * p.slabs * p.G;
  int64_t r0, r1;
  slab_rows(p, r0, r1);
  const int64_t base = n * p.S * p.C;
  const T *xs = static_cast<const T *>(p.x) + base;
  const T *zs = p.gate ? static_cast<const T *>(p.gate) + base : nullptr;
  const Rows<T, V, false> rows(ring, xs, xs, zs, gated, p.C, r0, r1, r0 + ty, TY, true);
  if (ty < TY) rows.start(tx * V);
  wait_first();
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
    constexpr int NP = (V + 1) / 2;
    Pair w[NP], b[NP];
    weights<V>(p.w, cv * V, true, 1.f, w);
    weights<V>(p.b, cv * V, true, 0.f, b);
    if (cv != tx) rows.start(cv * V);
    rows.run(
        cv * V, [&](int, int64_t at, const Raw<T, V> &x, const Raw<T, V> &, const Raw<T, V> &z) {
          Pair y[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const Pair d = add2(add2(x.at(i), both(-x0)), both(-mean));
            y[i] = activate2<T, M>(fma2(mul2(d, both(rstd)), w[i], b[i]), gated ? z.at(i) : 0, p);
          }
          put<T, V>(static_cast<T *>(p.y) + base + at, y);
        });
  }
}

// The slab's channel sums of du xh and du, and its group sums of dxh and dxh xh.
template <typename T, int V, int M>
__global__ void __launch_bounds__(kSlabThreads, 2)
gdn_norm_slab_grads_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = slab_tx(CV), TY = slab_ty(CV);
  const int tx = tid % TX, ty = tid / TX;
  float2 *sc = reinterpret_cast<float2 *>(sm);  // [TY][C]
  uint4 *ring = reinterpret_cast<uint4 *>(sm + ((size_t)2 * TY * p.C + 3) / 4 * 4);
  const int64_t n = blockIdx.y, base = n * p.S * p.C;
  const T *xs = static_cast<const T *>(p.x) + base, *dys = static_cast<const T *>(p.dy) + base;
  const T *zs = p.gate ? static_cast<const T *>(p.gate) + base : nullptr;
  int64_t r0, r1;
  slab_rows(p, r0, r1);
  const Rows<T, V, true> rows(ring, xs, dys, zs, gated, p.C, r0, r1, r0 + ty, TY, false);
  let_second();
  for (int cv = tx; cv < CV && ty < TY; cv += TX) {
    rows.start(cv * V);
    const int g = cv / DV;
    const float mean = p.mean[n * p.G + g], rstd = p.rstd[n * p.G + g];
    constexpr int NP = (V + 1) / 2;
    Pair w[NP], b[NP], a1[NP], a2[NP];
    weights<V>(p.w, cv * V, true, 1.f, w);
    weights<V>(p.b, cv * V, true, 0.f, b);
#pragma unroll
    for (int i = 0; i < NP; ++i) a1[i] = a2[i] = 0;
    float2 *const mine = sc + (size_t)ty * p.C + cv * V;
    bool fresh = true;
    const auto close = [&]() {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 q1 = un(a1[i / 2]), q2 = un(a2[i / 2]);
        float2 sum = i & 1 ? make_float2(q2.y, q1.y) : make_float2(q2.x, q1.x);
        if (!fresh) sum.x += mine[i].x, sum.y += mine[i].y;
        mine[i] = sum;
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) a1[i] = a2[i] = 0;
      fresh = false;
    };
    rows.run(
        cv * V, [&](int row, int64_t, const Raw<T, V> &x, const Raw<T, V> &dy, const Raw<T, V> &z) {
          if (row % kSum == kSum - 1) close();
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const Pair xh = mul2(add2(x.at(i), both(-mean)), both(rstd));
            Pair dz;
            const Pair du =
                grad_u2<T, M>(fma2(xh, w[i], b[i]), gated ? z.at(i) : 0, dy.at(i), p, dz);
            a1[i] = add2(a1[i], du);
            a2[i] = fma2(du, xh, a2[i]);
          }
        });
    close();
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
__global__ void __launch_bounds__(kSlabThreads, 2)
gdn_norm_slab_dx_kernel(const Params p) {
  const bool gated = M == kAny ? p.gate != nullptr : (M & 2) != 0;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, CV = p.C / V, DV = p.D / V;
  const int TX = slab_tx(CV), TY = slab_ty(CV);
  const int tx = tid % TX, ty = tid / TX;
  __shared__ float cs[kSlabThreads / 8 * 9];
  float2 *sg = reinterpret_cast<float2 *>(sm);
  uint4 *ring = reinterpret_cast<uint4 *>(sm + (2 * p.G + 3) / 4 * 4);
  const int64_t n = blockIdx.y, base = n * p.S * p.C;
  const T *xs = static_cast<const T *>(p.x) + base, *dys = static_cast<const T *>(p.dy) + base;
  const T *zs = p.gate ? static_cast<const T *>(p.gate) + base : nullptr;
  const float inv = 1.f / ((float)p.S * (float)p.D);
  int64_t r0, r1;
  slab_rows(p, r0, r1);
  const Rows<T, V, true> rows(ring, xs, dys, zs, gated, p.C, r0, r1, r0 + ty, TY, true);
  if (ty < TY) rows.start(tx * V);
  wait_first();
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
  if (p.dw || p.db) {
    // dweight and dbias: eight columns of the slabs' sums at a time, spread over the
    // CTAs while their first rows are on their way
    const int all = (int)p.N * p.slabs, id = (int)(n * p.slabs) + blockIdx.x;
    for (int c0 = 8 * id; c0 < 2 * p.C; c0 += 8 * all) sum_columns<8>(p, all, c0, cs);
  }
  __syncthreads();
  for (int cv = tx; cv < CV && ty < TY; cv += TX) {
    const int g = cv / DV;
    const float mean = p.mean[n * p.G + g], rstd = p.rstd[n * p.G + g];
    const float2 m = sg[g];
    constexpr int NP = (V + 1) / 2;
    Pair w[NP], b[NP];
    weights<V>(p.w, cv * V, true, 1.f, w);
    weights<V>(p.b, cv * V, true, 0.f, b);
    if (cv != tx) rows.start(cv * V);
    rows.run(
        cv * V, [&](int, int64_t at, const Raw<T, V> &x, const Raw<T, V> &dy, const Raw<T, V> &z) {
          Pair dx[NP], dz[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const Pair xh = mul2(add2(x.at(i), both(-mean)), both(rstd));
            dz[i] = 0;
            const Pair du =
                grad_u2<T, M>(fma2(xh, w[i], b[i]), gated ? z.at(i) : 0, dy.at(i), p, dz[i]);
            dx[i] = mul2(both(rstd), fma2(xh, both(-m.y), fma2(du, w[i], both(-m.x))));
          }
          put<T, V>(static_cast<T *>(p.dx) + base + at, dx);
          if (gated) put<T, V>(static_cast<T *>(p.dgate) + base + at, dz);
        });
  }
}

int tile_rows(int C, int V) { return C / V < kThreads ? kThreads / (C / V) : 1; }
// Slabs of a sample when there are few: two CTAs (all that fit) for each SM, four
// rows of every row of threads at least.
int slab_count(int64_t N, int64_t S, int C, int V) {
  const int64_t want = (2 * kSMs + N - 1) / N, most = S / (4 * slab_ty(C / V));
  const int64_t n = want < most ? want : most;
  return n < 1 ? 1 : (int)n;
}
// Fewer samples than SMs, or large ones.  us, slabs against sample: forward N 300,
// [256, 512] each, 46 / 90; 1000 of [49, 512] 43 / 33; backward 70 / 134; 60 / 94; 16000
// of [8, 256] 405 / 282.  (The slabs' sums are 8 C bytes each: 16 rows at least keep them
// a small part of the samples.)
bool use_slabs(int64_t N, int64_t S, int64_t C, bool backward) {
  return S > 1 && (N < kSMs ||
                   (N <= 65535 && S >= 16 && S * C >= (backward ? 16384 : 65536)));
}

template <auto Kernel>
cudaError_t go(dim3 grid, size_t bytes, const Params &p, cudaStream_t stream,
               int threads = kThreads, bool second = false) {
  const cudaError_t err = allow_smem<Kernel>(bytes);
  if (err != cudaSuccess) return err;
  if (second) return launch_beside(Kernel, grid, threads, bytes, stream, p);
  Kernel<<<grid, threads, bytes, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t sum_parts(const Params &p, int parts, cudaStream_t stream) {
  if (!p.dw && !p.db) return cudaSuccess;
  gdn_norm_dwdb_kernel<<<(2 * p.C + 31) / 32, 1024, 0, stream>>>(p, parts);
  return cudaGetLastError();
}

template <typename T, int V, int R, bool FULL, int M>
cudaError_t run_rows(const Params &p, bool backward, cudaStream_t stream) {
  const RowMap m = row_map(p.G, p.D / V);
  const int gy = (p.G + m.groups - 1) / m.groups;
  int64_t gx = (p.N + m.rows - 1) / m.rows;
  const int64_t most = backward ? (kParts / 2 + gy - 1) / gy : 4 * kSMs;
  if (gx > most) gx = most;
  const dim3 grid((unsigned)gx, gy);
  if (!backward) return go<gdn_norm_rows_fwd_kernel<T, V, R, FULL, M>>(grid, 0, p, stream);
  const size_t bytes = (size_t)8 * m.rows * m.groups * p.D;
  const cudaError_t err = go<gdn_norm_rows_bwd_kernel<T, V, R, FULL, M>>(grid, bytes, p, stream);
  return err == cudaSuccess ? sum_parts(p, (int)gx, stream) : err;
}

template <typename T, int V, int M>
cudaError_t run_slabs(Params p, bool backward, cudaStream_t stream) {
  const int CV = p.C / V, TY = slab_ty(CV), threads = (slab_tx(CV) * TY + 31) / 32 * 32;
  p.slabs = slab_count(p.N, p.S, p.C, V);
  const int parts = (int)p.N * p.slabs;
  p.sums = p.part + (backward ? (size_t)parts * 2 * p.C : 0);
  const dim3 grid(p.slabs, (unsigned)p.N);
  const size_t groups = ((size_t)8 * p.G + 15) / 16 * 16;
  const int gates = p.gate ? 1 : 0;
  cudaError_t err;
  if (!backward) {
    const size_t own = ((size_t)12 * TY * CV + 15) / 16 * 16;
    err = go<gdn_norm_slab_stats_kernel<T, V>>(grid, own + ring_bytes<T, V>(threads, 1), p, stream,
             threads);
    return err != cudaSuccess
               ? err
               : go<gdn_norm_slab_apply_kernel<T, V, M>>(grid,
                    groups + ring_bytes<T, V>(threads, 1 + gates), p, stream, threads, true);
  }
  const size_t own = ((size_t)8 * TY * p.C + 15) / 16 * 16;
  err = go<gdn_norm_slab_grads_kernel<T, V, M>>(grid, own + ring_bytes<T, V>(threads, 2 + gates), p,
           stream, threads);
  if (err != cudaSuccess) return err;
  return go<gdn_norm_slab_dx_kernel<T, V, M>>(grid, groups + ring_bytes<T, V>(threads, 2 + gates), p,
            stream, threads, true);
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
    if (full || use_slabs(p.N, p.S, p.C, backward)) {
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
    if (use_slabs(p.N, p.S, p.C, backward)) return run_slabs<T, V, kAny>(p, backward, stream);
  const int grid = (int)(p.N < kParts ? p.N : kParts);
  if (!backward)
    return go<gdn_norm_fwd_kernel<T, V>>(grid, ((size_t)3 * TY * CV + 2 * p.G) * 4, p, stream);
  const size_t bytes = ((size_t)TY * CV + p.G + (size_t)TY * p.C) * 8;
  const cudaError_t err = p.S > (int64_t)kSum * TY
                              ? go<gdn_norm_bwd_kernel<T, V, true>>(grid, bytes, p, stream)
                              : go<gdn_norm_bwd_kernel<T, V, false>>(grid, bytes, p, stream);
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
  const size_t slabs = use_slabs(batch, spatial, channels, true) ? (size_t)(2 * kSMs + batch) : 0,
               parts = slabs > (size_t)kParts ? slabs : (size_t)kParts;
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
      if (to && taken(cudaMemsetAsync(to, 0, b_c, (cudaStream_t)stream)) != cudaSuccess)
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
