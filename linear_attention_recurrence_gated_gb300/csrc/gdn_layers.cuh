// What the short convolution, the selective scan and the q/k norm share: vectors of
// eight channels, packed fp32 arithmetic, the sequences of a call, host-side checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace layer {

constexpr int kSMs = 152;
constexpr float kLog2e = 1.4426950408889634f;

// Eight consecutive elements as they are stored: 16 bytes of bf16, 32 of fp32.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    a = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
    *reinterpret_cast<uint4 *>(p) = a;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {   // rounds to nearest even
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void store(float *p) const {
    reinterpret_cast<float4 *>(p)[0] = a;
    reinterpret_cast<float4 *>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// Two fp32 values in one 64-bit register pair.
__device__ __forceinline__ uint64_t pk(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpk(uint64_t a, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + exp(-z)); exact limits for infinite z.
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.f + ex2(-kLog2e * z)); }

// 1 / (1 + exp(-g)) of two values.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t g) {
  float a, b;
  unpk(mul2(g, pk(-kLog2e, -kLog2e)), a, b);
  unpk(add2(pk(ex2(a), ex2(b)), pk(1.f, 1.f)), a, b);
  return pk(rcp(a), rcp(b));
}
// Four consecutive elements: 8 bytes of bf16, 16 of fp32.
template <typename T> struct Raw4;
template <> struct Raw4<__nv_bfloat16> {
  uint2 a;
  __device__ __forceinline__ void zero() { a = make_uint2(0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint2 *>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint2 *>(p) = a; }
  __device__ __forceinline__ void get(uint64_t (&v)[2]) const {
    v[0] = pk(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u));
    v[1] = pk(__uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u));
  }
  __device__ __forceinline__ void set(const uint64_t (&v)[2]) {   // rounds to nearest even
    float x, y, z, w;
    unpk(v[0], x, y);
    unpk(v[1], z, w);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y), i = __floats2bfloat162_rn(z, w);
    a = make_uint2(*reinterpret_cast<const uint32_t *>(&h), *reinterpret_cast<const uint32_t *>(&i));
  }
};
template <> struct Raw4<float> {
  ulonglong2 a;
  __device__ __forceinline__ void zero() { a = make_ulonglong2(0, 0); }
  __device__ __forceinline__ void load(const float *p) { a = *reinterpret_cast<const ulonglong2 *>(p); }
  __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<ulonglong2 *>(p) = a; }
  __device__ __forceinline__ void get(uint64_t (&v)[2]) const { v[0] = a.x; v[1] = a.y; }
  __device__ __forceinline__ void set(const uint64_t (&v)[2]) { a = make_ulonglong2(v[0], v[1]); }
};

// The sequences of a call: rows of seq_len tokens, or packed ones between offsets in
// device memory.
struct Sequences {
  const int32_t *cu;
  DeviceStatus *status;
  int64_t seq_len;       // tokens of a row, or of all packed sequences together
  int32_t num_seqs;
  __device__ __forceinline__ int64_t tokens() const {
    return cu ? seq_len : seq_len * num_seqs;
  }
  // Bounds of sequence n; false (recorded) where the offsets break the rules.
  __device__ __forceinline__ bool bounds(int n, int64_t &start, int64_t &len) const {
    FwdParams f;
    f.cu = cu;
    f.seq_len = seq_len;
    f.num_seqs = num_seqs;
    f.status = status;
    return sequence_bounds(f, n, 0, start, len);
  }
  // The last sequence that begins at or before token t, found by the whole warp
  // together (t the same in every lane): 32 offsets at a time.
  __device__ __forceinline__ int find(int64_t t) const {
    const int lane = threadIdx.x & 31;
    int lo = 0, size = num_seqs;
    while (size > 1) {
      const int step = (size + 31) / 32;
      const bool before = lane * step < size && cu[lo + lane * step] <= t;
      const uint32_t is = __ballot_sync(0xffffffffu, before);
      const int k = is ? 31 - __clz(is) : 0;
      lo += k * step;
      size = size - k * step < step ? size - k * step : step;
    }
    return lo;
  }
};

// ---- host-side checks ----
struct Range {
  const void *p;
  size_t n;
};
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool overlaps(const Range &a, const Range &b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
// No output overlaps an input or another output.
template <int NO, int NI>
bool apart(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlaps(outs[i], ins[j])) return false;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return false;
  }
  return true;
}
template <int N>
bool all_aligned(const void *const (&ptrs)[N]) {
  for (const void *p : ptrs)
    if (p && !aligned16(p)) return false;
  return true;
}
// Elements between token rows: 0 stands for densely packed rows.  Returns 0 for a
// stride that cannot hold a row or breaks the 16-byte alignment.
inline int64_t row_stride(int64_t given, int64_t dense, size_t e) {
  if (given == 0) return dense;
  return given >= dense && given * (int64_t)e % 16 == 0 ? given : 0;
}
inline size_t span_bytes(size_t rows, int64_t stride, int64_t width, size_t e) {
  return rows ? ((rows - 1) * (size_t)stride + (size_t)width) * e : 0;
}

}  // namespace layer
}  // namespace gdn
