// Selective state space scan: what the forward, backward and step units share.
//
//   delta = softplus(dt + dt_bias),  A = -exp(A_log)                    [D], [D][S]
//   h_t = exp(delta_t A) h_{t-1} + delta_t x_t b_t,   s_t = c_t . h_t + D_skip x_t
//   y_t = s_t silu(gate_t)
//
// Every (channel, state) decays at a rate of its own, so there is no product that the
// tensor cores could take: each of the T D S elements costs an exponential and four
// multiply-adds on the CUDA cores, and that is what bounds the scan (a GB300 SM does 32
// exponentials and 128 multiply-adds a clock; the bytes of a token's channel, 8 in bf16,
// would take a third of the time of its 16 states).
//
// A thread holds 4 channels x 4 states in registers, pairs of channels in packed fp32
// arithmetic.  S / 4 lanes share 4 channels, so that a token's c . h is summed over S / 4
// lanes, its gradients of b and c over the 128 / S others; four states of b and c and four
// channels of delta and delta x come from shared memory in 16-byte loads that all lanes
// of a row share.  A CTA of 4 warps owns 2048 / S channels of one group.
//
// Sequences are cut along time where their channels alone leave SMs idle: a first launch
// leaves each segment's state from zero and its sum of delta, and a segment's start is
// joined from those before it, h <- exp(A sum delta) h + X, as the second launch begins.
#pragma once

#include "gdn_launch.cuh"
#include "gdn_layers.cuh"
#include "gdn_lin.cuh"

namespace gdn {
namespace ssm {

using namespace layer;

constexpr int kThreads = 128;

template <int S>
struct Geo {
  static constexpr int LS = S / 4;            // lanes that share a channel
  static constexpr int CL = 32 / LS;          // groups of 4 channels in a warp
  static constexpr int CW = 4 * CL;           // channels of a warp
  static constexpr int CB = CW * (kThreads / 32);   // ... of a CTA
};

struct Params {
  lin::Params seq;   // cu, status, seq_len, num_seqs and the split along time
  const void *x, *dt, *b, *c, *gate;
  const float *A_log, *d_skip, *dt_bias, *h0;
  void *y;
  float *hT;
  int64_t sx, sdt, sb, sc, sg;   // elements from token to token
  int32_t D, Dg, blocks;         // channels, of a group, CTAs a group
  bool softplus, keep;           // keep: hT is h0, and sequences are cut
  float *seg_x;                  // [slot][D][S] state of a segment, run from zero
  float *seg_d;                  // [slot][D] its sum of delta
};

// log(1 + exp(v)): with e = exp(-|v|) <= 1 and s = e / (2 + e) <= 1/3 it is
// max(v, 0) + 2 artanh(s), and the series of artanh leaves out s^15 / 15 < 2^-27 s.
template <typename T>
__device__ __forceinline__ float softplus(float v) {
  // (for bf16 inputs the exponent's rounding, some 2^-21, is far below dt's own)
  const float e = sizeof(T) == 4 ? expf(-fabsf(v)) : ex2(-kLog2e * fabsf(v));
  const float s = e * rcp(2.f + e), q = s * s;
  float r = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  r = fmaf(q, r, 1.f / 9.f);
  r = fmaf(q, r, 1.f / 7.f);
  r = fmaf(q, r, 1.f / 5.f);
  r = fmaf(q, r, 1.f / 3.f);
  r = fmaf(q * s, r, s);
  return fmaxf(v, 0.f) + (r + r);
}

// v[4] summed over the LS lanes that share channels, each lane keeping some of them:
// two lanes two values each (v[0], v[1] of lane 0 are channels 0 and 1), more lanes
// one each (v[0] of lane i is channel i & 3).
template <int LS>
__device__ __forceinline__ void sum_channels(float (&v)[4], int sl) {
  constexpr uint32_t kAll = 0xffffffffu;
  if constexpr (LS == 2) {
    const bool up = sl & 1;
    const float a = up ? v[0] : v[2], b = up ? v[1] : v[3];
    v[0] = (up ? v[2] : v[0]) + __shfl_xor_sync(kAll, a, 1);
    v[1] = (up ? v[3] : v[1]) + __shfl_xor_sync(kAll, b, 1);
  } else {
    const bool hi = sl & 2, up = sl & 1;
    const float a = hi ? v[0] : v[2], b = hi ? v[1] : v[3];
    v[0] = (hi ? v[2] : v[0]) + __shfl_xor_sync(kAll, a, 2);
    v[1] = (hi ? v[3] : v[1]) + __shfl_xor_sync(kAll, b, 2);
    const float c = up ? v[0] : v[1];
    v[0] = (up ? v[1] : v[0]) + __shfl_xor_sync(kAll, c, 1);
#pragma unroll
    for (int m = 4; m < LS; m *= 2) v[0] += __shfl_xor_sync(kAll, v[0], m);
  }
}
template <int LS>
__device__ __forceinline__ void store_channels(float *at, const float (&v)[4], int sl) {
  if constexpr (LS == 2)
    *reinterpret_cast<float2 *>(at + 2 * sl) = make_float2(v[0], v[1]);
  else if (sl < 4)
    at[sl] = v[0];
}

// What a thread owns: 4 states from st of the 4 channels from ch (numbered through all
// groups); `on` where there are such channels.
struct Own {
  int ch, st;
  bool on;
};
// a[channel pair][state]: elements of a [D][S] array, 0 where there is no channel.
template <int S>
__device__ __forceinline__ void load_own(const float *base, const Own &o, uint64_t (&a)[2][4]) {
  float v[4][4] = {};
  if (o.on && base)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = *reinterpret_cast<const float4 *>(base + (int64_t)(o.ch + i) * S + o.st);
      v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
    }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) a[k][j] = pk(v[2 * k][j], v[2 * k + 1][j]);
}
template <int S>
__device__ __forceinline__ void store_own(float *base, const Own &o, const uint64_t (&a)[2][4]) {
  if (!o.on) return;
  float v[4][4];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) unpk(a[k][j], v[2 * k][j], v[2 * k + 1][j]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4 *>(base + (int64_t)(o.ch + i) * S + o.st) =
        make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
}
// A log2(e), so that exp(delta A) is one exp2 of a product; finite, so that tokens that
// do not exist (delta = 0) leave a state as it is whatever A_log holds.
__device__ __forceinline__ float rate(float a_log) {
  const float a = -kLog2e * expf(a_log);
  return a < -3e38f ? -3e38f : a;
}
template <int S>
__device__ __forceinline__ void load_rates(const float *A_log, const Own &o, uint64_t (&a)[2][4]) {
  load_own<S>(A_log, o, a);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      unpk(a[k][j], lo, hi);
      a[k][j] = o.on ? pk(rate(lo), rate(hi)) : 0ull;
    }
}
__device__ __forceinline__ uint64_t ex2_pair(uint64_t x) {
  float lo, hi;
  unpk(x, lo, hi);
  return pk(ex2(lo), ex2(hi));
}
// h <- exp(A sum) h + X of the segment in `slot` (its arrays x [slot][D][S], d [slot][D]).
template <int S>
__device__ __forceinline__ void join(uint64_t (&h)[2][4], const uint64_t (&A)[2][4],
                                     const float *x, const float *d, int64_t slot, int D,
                                     const Own &o) {
  uint64_t add[2][4];
  load_own<S>(x + slot * D * S, o, add);
  const float4 sum = o.on ? *reinterpret_cast<const float4 *>(d + slot * D + o.ch)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
  const uint64_t s[2] = {pk(sum.x, sum.y), pk(sum.z, sum.w)};
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[k][j] = fma2(ex2_pair(mul2(s[k], A[k][j])), h[k][j], add[k][j]);
}
struct Pairs {
  uint64_t a, b;
};
__device__ __forceinline__ Pairs lds2(const float *p) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
  return {v.x, v.y};
}
// Eight values, each twice: the operand of packed arithmetic on two channels.
__device__ __forceinline__ void store_twice(float *at, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4 *>(at)[i] =
        make_float4(v[2 * i], v[2 * i], v[2 * i + 1], v[2 * i + 1]);
}

// The split along time of a launch of `blocks` CTAs per segment: chunks of 32 tokens, two
// CTAs an SM at a time; a segment's start costs about a chunk, the first launch of it
// `first` of the second.
constexpr int kChunkTokens = 32;
inline lin::Plan plan(int64_t num_seqs, int64_t seq_len, bool packed, int64_t blocks,
                      double first) {
  return lin::plan_segments(num_seqs, seq_len, packed, blocks, 2 * kSMs, kChunkTokens, 1.0, first);
}
inline int channel_blocks(int Dg, int S) { return (Dg + 2048 / S - 1) / (2048 / S); }
inline bool state_size(int S) { return S == 8 || S == 16 || S == 32 || S == 64; }

// Bytes of a call's arrays, and the checks that forward and backward share.
struct Sizes {
  size_t rows, e;
  int64_t D, gs;   // channels; elements of a token's b
  int64_t sx, sdt, sb, sc, sg;
  size_t state;
};
gdn_status check_sizes(int32_t batch, int32_t seq_len, int32_t channels, int32_t d_state,
                       int32_t groups, int32_t num_seqs, const void *cu, gdn_dtype dtype,
                       uint32_t flags);
bool strides_of(Sizes &z, int64_t x, int64_t dt, int64_t b, int64_t c, int64_t gate);

}  // namespace ssm
}  // namespace gdn
