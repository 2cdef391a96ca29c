// Selective state space scan: what the forward, backward and step units share.
//
//   delta = softplus(dt + dt_bias),  A = -exp(A_log)                    [D], [D][S]
//   h_t = exp(delta_t A) h_{t-1} + delta_t x_t b_t,   s_t = c_t . h_t + D_skip x_t
//   y_t = s_t silu(gate_t)
//
// Every (channel, state) decays at a rate of its own, so there is no product that the
// tensor cores could take: each of the T D S elements costs an exponential and four
// multiply-adds on the CUDA cores, and that is what bounds the scan (a GB300 SM does 32
// exponentials and 128 multiply-adds a clock: 33 us each for [4, 4096, 1280], S = 16, whose
// bytes take 25).
//
// A CTA of 4 warps owns 2048 / S channels of one group, a thread 16 elements in registers,
// in packed fp32 arithmetic.  Forward, 16 states of a channel (8 of two for S = 8): c . h is
// a sum inside the thread.  In the backward pass, 4 channels x 4 states: sums over states
// (b . G, A w) and over channels (db, dc) meet half-way, over S / 4 and 128 / S lanes.
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

// exp(-|v|).  The rounding of exp2's argument takes |v| 2^-24 of it and that of log2(e)
// |v| 1.3e-8, always the same way: 5e-7 together at the usual start of a step (v = -7) and
// 6e-6 at most (v = -80).  With fp32 storage they are put right; with bf16 storage, whose dt
// is itself off by up to 2^-9 of its value, they stay (put right there too, [4, 4096, 1280],
// S = 16: forward 180 us for 176, backward 564 for 558).
template <typename T>
__device__ __forceinline__ float exp_abs(float v) {
  const float t = -kLog2e * fabsf(v);
  const float e = ex2(t);
  if constexpr (sizeof(T) != 4) return e;
  constexpr float kLow = 1.9259629911266175e-8f;   // log2(e) - kLog2e
  const float low = fmaf(-fabsf(v), kLow, fmaf(-fabsf(v), kLog2e, -t));
  return e > 0.f ? fmaf(e, 0.6931472f * low, e) : e;   // (0 for -inf, whose low is NaN)
}
// log(1 + exp(v)) of two values: with e = exp(-|v|) <= 1 and s = e / (2 + e) <= 1/3 it is
// max(v, 0) + 2 artanh(s).  artanh(s) = s + s^3 f(s^2), f(q) = 1/3 + q/5 + q^2/7 + ..., by
// the cubic that minimises the largest q |error| over [0, 1/9] (4e-9, a fifteenth of
// fp32's half step).  Largest relative errors, measured over 2^14 arguments a range: from -1
// to 20 2.6e-7; below, with fp32 storage, 3.0e-7; with bf16 storage 5.2e-7 down to -8, 9.4e-7
// to -20, 3.7e-6 to -80.
template <typename T>
__device__ __forceinline__ uint64_t softplus2(uint64_t v) {
  float a, b;
  unpk(v, a, b);
  const uint64_t e = pk(exp_abs<T>(a), exp_abs<T>(b));
  float wa, wb;
  unpk(add2(e, pk(2.f, 2.f)), wa, wb);
  const uint64_t s = mul2(e, pk(rcp(wa), rcp(wb))), q = mul2(s, s);
  uint64_t r = fma2(pk(0.14012232422828674f, 0.14012232422828674f), q, pk(0.13999569416046143f, 0.13999569416046143f));
  r = fma2(r, q, pk(0.20010849833488464f, 0.20010849833488464f));
  r = fma2(r, q, pk(0.3333320617675781f, 0.3333320617675781f));
  r = fma2(mul2(q, s), r, s);
  return fma2(r, pk(2.f, 2.f), pk(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}
// Its derivative, 1 / (1 + exp(-v)), as exact as the step that it belongs to.
template <typename T>
__device__ __forceinline__ uint64_t softplus_slope2(uint64_t v) {
  if constexpr (sizeof(T) != 4) return sigmoid2(v);
  float a, b, ra, rb;
  unpk(v, a, b);
  const float ea = exp_abs<T>(a), eb = exp_abs<T>(b);
  unpk(add2(pk(ea, eb), pk(1.f, 1.f)), ra, rb);
  return mul2(pk(a < 0.f ? ea : 1.f, b < 0.f ? eb : 1.f), pk(rcp(ra), rcp(rb)));
}
// delta of eight channels: pairs of dt + dt_bias, its softplus if asked for.
template <typename T>
__device__ __forceinline__ void steps_of(const Raw8<T> &dt, const uint64_t (&bias)[4], bool soft,
                                         uint64_t (&d)[4]) {
  float v[8];
  dt.get(v);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = add2(pk(v[2 * i], v[2 * i + 1]), bias[i]);
  if (soft)
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = softplus2<T>(d[i]);
}
template <typename T>
__device__ __forceinline__ void pairs_of(const Raw8<T> &r, uint64_t (&p)[4]) {
  float v[8];
  r.get(v);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pk(v[2 * i], v[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ void set_pairs(Raw8<T> &r, const uint64_t (&p)[4]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpk(p[i], v[2 * i], v[2 * i + 1]);
  r.set(v);
}
__device__ __forceinline__ void put8(float *at, const uint64_t (&p)[4]) {
  reinterpret_cast<ulonglong2 *>(at)[0] = make_ulonglong2(p[0], p[1]);
  reinterpret_cast<ulonglong2 *>(at)[1] = make_ulonglong2(p[2], p[3]);
}
__device__ __forceinline__ void take8(const float *at, uint64_t (&p)[4]) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(at)[0];
  const ulonglong2 b = reinterpret_cast<const ulonglong2 *>(at)[1];
  p[0] = a.x; p[1] = a.y; p[2] = b.x; p[3] = b.y;
}
// Eight channels' values of an fp32 array, 0 without one.
__device__ __forceinline__ void load8(const float *base, int ch, bool on, uint64_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = base && on ? *reinterpret_cast<const uint64_t *>(base + ch + 2 * i) : 0ull;
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
// exp(delta A) of a token.  The hardware's exp2 is low on average, and a state adds up
// 1 / (1 - a) such errors.  Measured over 2^18 arguments an eighth of an octave: 4e-9 to 1e-8
// from -2^-8 to 0, 1.3e-8 at -2^-8, 3.0e-8 at -2^-7, 2.2e-8 on average from there to -1/2.
// A lift of the exponent takes the mean away: by the slowest rate of the 4 or 8 elements that
// share it, whose errors a state keeps longest, and one step of a tile.  (2^lift itself still
// gives 1: delta = 0 keeps a state.  One lift for all, 2.5e-8, left states of slow decays
// 1.1e-6 off for 2.9e-7, and dA_log 2.2e-6 for 1.3e-6, over some 1000 tokens; it takes the
// same time within 3 %, and so do lifts that go into a state once a tile.)
__device__ __forceinline__ float lift_of(float delta, float rate) {
  return fminf(fmaxf(-5e-6f * rate * delta, 0.85e-8f), 3.1e-8f);
}
__device__ __forceinline__ uint64_t decay(uint64_t delta, uint64_t A, uint64_t lift) {
  return ex2_pair(fma2(delta, A, lift));
}
__device__ __forceinline__ float slower(uint64_t a) {
  float lo, hi;
  unpk(a, lo, hi);
  return fmaxf(lo, hi);
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

// The forward scans' threads: 16 consecutive elements of [D][S], that is 16 states of one
// channel (8 of two for S = 8), pairs of states in packed arithmetic.  c . h is summed
// inside a thread up to S = 16, over S / 16 lanes beyond; b and c are read by whole warps
// from one address.  (With 4 channels x 4 states a thread the call took 204 us where this
// took 179, [4, 4096, 1280], S = 16: three shuffles and their selects a token.)
template <int S>
struct Run {
  static constexpr int SPT = S < 16 ? S : 16;   // states of a channel
  static constexpr int CPT = 16 / SPT;          // channels
  static constexpr int LS = S / SPT;            // lanes that share a channel
  static constexpr int NP = SPT / 2;            // pairs of states
};
__device__ __forceinline__ void load16(const float *at, bool on, uint64_t (&a)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const ulonglong2 v = on && at ? reinterpret_cast<const ulonglong2 *>(at)[i] : make_ulonglong2(0, 0);
    a[2 * i] = v.x;
    a[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void store16(float *at, bool on, const uint64_t (&a)[8]) {
  if (!on) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<ulonglong2 *>(at)[i] = make_ulonglong2(a[2 * i], a[2 * i + 1]);
}
__device__ __forceinline__ void rates16(const float *at, bool on, uint64_t (&a)[8]) {
  load16(at, on, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo, hi;
    unpk(a[i], lo, hi);
    a[i] = on ? pk(rate(lo), rate(hi)) : 0ull;
  }
}
// h <- exp(A sum) h + x, from a segment's state x and its sum of delta for the thread's
// channels.
template <int S>
__device__ __forceinline__ void join16(uint64_t (&h)[8], const uint64_t (&A)[8], const float *x,
                                       const float *sum, bool on) {
  uint64_t add[8];
  load16(x, on, add);
#pragma unroll
  for (int k = 0; k < Run<S>::CPT; ++k) {
    const float d = on ? sum[k] : 0.f;
#pragma unroll
    for (int i = 0; i < Run<S>::NP; ++i) {
      const int e = k * Run<S>::NP + i;
      h[e] = fma2(ex2_pair(mul2(pk(d, d), A[e])), h[e], add[e]);
    }
  }
}
// Shared memory: the steps of a thread's channels at token t, each twice; n pairs.
template <int CPT>
__device__ __forceinline__ void twice(const float *at, uint64_t (&d)[CPT]) {
  if constexpr (CPT == 2) {
    const float2 v = *reinterpret_cast<const float2 *>(at);
    d[0] = pk(v.x, v.x);
    d[1] = pk(v.y, v.y);
  } else {
    d[0] = pk(at[0], at[0]);
  }
}
// (S = 64: the upper half of a row's 16-byte pieces lies with neighbours exchanged, so that
// the four lanes of a channel read from different banks.)
template <int N>
__device__ __forceinline__ void pairs(const float *at, int swap, uint64_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const ulonglong2 w = reinterpret_cast<const ulonglong2 *>(at)[i ^ swap];
    v[2 * i] = w.x;
    v[2 * i + 1] = w.y;
  }
}
__device__ __forceinline__ float total(uint64_t v) {
  float lo, hi;
  unpk(v, lo, hi);
  return lo + hi;
}

// The lifts of a thread of 16 elements, one for eight of them; d: a step of each channel.
template <int CPT>
__device__ __forceinline__ void lifts16(const uint64_t (&A)[8], const float *d, uint64_t (&lift)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float slow = fmaxf(fmaxf(slower(A[4 * i]), slower(A[4 * i + 1])),
                             fmaxf(slower(A[4 * i + 2]), slower(A[4 * i + 3])));
    const float v = lift_of(d[CPT == 2 ? i : 0], slow);
    lift[i] = pk(v, v);
  }
}

struct Pairs {
  uint64_t a, b;
};
__device__ __forceinline__ Pairs lds2(const float *p) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
  return {v.x, v.y};
}
// b and c of a tile of L tokens for threads of 4 channels x 4 states, each value twice (the
// operand of packed arithmetic on two channels): [b, c][token][first, second two of four
// states][S / 4][2 x 2], so that the lanes of a channel read neighbouring 16 bytes.
// Vector v (eight states) of token t of b (w = 0) or c (1):
template <int S>
__device__ __forceinline__ void store_twice(float *sbc, int idx, const float (&v)[8]) {
  const int row = idx / (S / 8), k = idx % (S / 8);   // row: [b, c][token]
  float *at = sbc + row * 2 * S + 8 * k;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4 *>(at + (i & 1) * S + 4 * (i >> 1)) =
        make_float4(v[2 * i], v[2 * i], v[2 * i + 1], v[2 * i + 1]);
}
template <int S, int L = 8>
__device__ __forceinline__ void load_twice(const float *sbc, int t, int which, int sl, uint64_t (&v)[4]) {
  const float *at = sbc + (which * L + t) * 2 * S + 4 * sl;
  const Pairs a = lds2(at), b = lds2(at + S);
  v[0] = a.a; v[1] = a.b; v[2] = b.a; v[3] = b.b;
}

// The lifts of a thread of 4 channels x 4 states, one for each channel.
__device__ __forceinline__ void lifts4(const uint64_t (&A)[2][4], const float *d, uint64_t (&lift)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpk(A[k][j], lo[j], hi[j]);
    lift[k] = pk(lift_of(d[2 * k], fmaxf(fmaxf(lo[0], lo[1]), fmaxf(lo[2], lo[3]))),
                 lift_of(d[2 * k + 1], fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]))));
  }
}

// The split along time of launches of `blocks` CTAs per segment, `ctas` an SM at a time, in
// chunks of 32 tokens; a segment's start costs about half a chunk, the first launch of it
// `first` of the second.  (Forward, [4, 4096, 1280] / [1, 65536, 2048], before the lifts
// went by tiles: 179 / 992 us; a start of a whole chunk 179 / 1027, of two 179 / 1027; two
// CTAs an SM 241 / 1310, four 192 / 1031, six 186 / 992.)
constexpr int kChunkTokens = 32;
inline lin::Plan plan(int64_t num_seqs, int64_t seq_len, bool packed, int64_t blocks, int ctas,
                      double first) {
  return lin::plan_segments(num_seqs, seq_len, packed, blocks, ctas * kSMs, kChunkTokens, 0.4, first);
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
bool some_sizes(int32_t num_seqs, int32_t seq_len, int32_t channels, int32_t d_state,
                int32_t groups);   // that a workspace can be sized for
gdn_status check_sizes(int32_t batch, int32_t seq_len, int32_t channels, int32_t d_state,
                       int32_t groups, int32_t num_seqs, const void *cu, gdn_dtype dtype,
                       uint32_t flags);
bool strides_of(Sizes &z, int64_t x, int64_t dt, int64_t b, int64_t c, int64_t gate);

}  // namespace ssm
}  // namespace gdn
