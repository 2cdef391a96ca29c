// Selective state space scan, prompts: host checks and the forward kernels (gdn_ssm.cuh
// has the mathematics and the layout of the work).
//
// A CTA walks over its tokens in tiles: delta and delta x are formed from the tile's
// inputs by threads that own eight channels of a token, and left in shared memory as
// fp32 together with b and c; then every thread runs its 16 elements over the tile while
// the next tile's inputs are on their way to registers; then the tile's outputs take the
// skip and the gate on their way out.
//
// [4, 4096, 1280], S = 16, bf16 with a gate: 176 us, 73 of them the first launch; some 104
// instructions a token and 32 channels where outputs are formed, of which 32 packed
// multiply-adds and 16 exponentials are the scan itself, the rest its operands, softplus and
// the gate.  No pipe is full (multiply-adds 50 %, exponentials 43 %, shared memory 62 %,
// issue 56 %), but each is near what warps that take turns at them reach: fewer instructions
// help, more warps do not (four CTAs an SM without spills, inputs by asynchronous copies or
// gate and x read when they are needed: 189 and 185), nor the next token's exponentials
// between this one's products (192), nor 32 elements a thread, which halve the loads of b
// and c (200).  [1, 65536, 2048]: 995 us.
#include "gdn_ssm.cuh"

namespace gdn {
gdn_status pass_states(const float *from, float *to, size_t bytes, cudaStream_t s);

namespace ssm {
namespace {

template <int S>
struct Fwd : Geo<S> {
  using Geo<S>::CB;
  static constexpr int TT = S <= 16 ? S : 32;                    // tokens of a tile
  static constexpr int NV = (TT * CB / 8 + kThreads - 1) / kThreads;   // vectors of a thread
  static constexpr int NB = (2 * TT * S / 8 + kThreads - 1) / kThreads;
  static constexpr int VB = CB / 8;                               // vectors of a token
  static_assert(kThreads % VB == 0 && TT * CB / 8 == NV * kThreads, "whole rows of vectors");
};

template <typename T, int S, bool OUT>
__global__ void __launch_bounds__(kThreads, OUT ? 3 : 4)
gdn_ssm_scan_kernel(const Params p) {
  using F = Fwd<S>;
  using R = Run<S>;
  constexpr int TT = F::TT, CB = F::CB, LS = R::LS, CPT = R::CPT, NP = R::NP;
  __shared__ __align__(16) float sd[TT * CB], su[TT * CB], sy[OUT ? TT * CB : 4];
  __shared__ __align__(16) float sbc[(OUT ? 2 : 1) * TT * S];
  const int tid = threadIdx.x;
  const int group = blockIdx.x / p.blocks, cb = blockIdx.x % p.blocks, slot = blockIdx.y;
  const int first_ch = group * p.Dg + cb * CB, end_ch = (group + 1) * p.Dg;
  const int sl = tid % LS, cl = tid / LS * CPT;   // its part of the states, its first channel
  const int swap = S == 64 ? sl >> 1 : 0;
  const bool on = first_ch + cl < end_ch;
  const int64_t own = (int64_t)first_ch * S + 16 * tid;   // its elements of [D][S]

  uint64_t A[8], h[8];
  rates16(p.A_log + own, on, A);
  // its eight channels where tiles are formed and left
  const int vec = tid % F::VB, vch = first_ch + 8 * vec;
  const bool von = vch < end_ch;
  uint64_t bias[4], skip[4];
  load8(p.dt_bias, vch, von, bias);
  if (OUT) load8(p.d_skip, vch, von, skip);
  if (OUT && p.seq.seg_len) wait_first();   // every CTA: none may end before the first launch
  if (!OUT) let_second();
  lin::Span s;
  if (!lin::span_of(p.seq, slot, 0, s)) return;
  const int64_t state = (int64_t)p.D * S;
  if (!OUT && s.seg == s.count - 1) {   // nothing follows; keep what the last launch overwrites
    if (p.keep) {
      load16(p.h0 + s.n * state + own, on, h);
      store16(p.seg_x + slot * state + own, on, h);
    }
    return;
  }
  if (s.seg == 0) {
    const bool kept = OUT && p.keep && p.seq.seg_len;
    const float *from = kept ? p.seg_x + (slot + s.count - 1) * state : p.h0 ? p.h0 + s.n * state : nullptr;
    load16(from ? from + own : nullptr, on, h);
  } else if (!OUT) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 0ull;
  } else {
    const int64_t one = slot - s.seg;
    load16(p.seg_x + one * state + own, on, h);   // the first one's end state
    for (int i = 1; i < s.seg; ++i)
      join16<S>(h, A, p.seg_x + (one + i) * state + own, p.seg_d + (one + i) * p.D + first_ch + cl, on);
  }

  Raw8<T> xr[F::NV], dr[F::NV], gr[F::NV], br[F::NB];
  const T *x = static_cast<const T *>(p.x) + s.start * p.sx + vch;
  const T *dt = static_cast<const T *>(p.dt) + s.start * p.sdt + vch;
  const T *gate = OUT && p.gate ? static_cast<const T *>(p.gate) + s.start * p.sg + vch : nullptr;
  const T *b = static_cast<const T *>(p.b) + s.start * p.sb + group * S;
  const T *c = static_cast<const T *>(p.c) + s.start * p.sc + group * S;
  const auto fetch = [&](int64_t t0) {
    const int cnt = (int)(s.len - t0 < TT ? s.len - t0 : TT);
#pragma unroll
    for (int i = 0; i < F::NV; ++i) {
      const int row = tid / F::VB + i * (kThreads / F::VB);
      const bool on = von && row < cnt;
      xr[i].zero();
      dr[i].zero();
      gr[i].zero();
      if (on) {
        xr[i].load(x + (t0 + row) * p.sx);
        dr[i].load(dt + (t0 + row) * p.sdt);
        if (gate) gr[i].load(gate + (t0 + row) * p.sg);
      }
    }
#pragma unroll
    for (int i = 0; i < F::NB; ++i) {
      const int idx = tid + i * kThreads, row = idx % (TT * S / 8) / (S / 8), v = idx % (S / 8);
      const bool second = idx >= TT * S / 8;
      br[i].zero();
      if (row < cnt && idx < 2 * TT * S / 8) {
        if (!second) br[i].load(b + (t0 + row) * p.sb + 8 * v);
        else if (OUT) br[i].load(c + (t0 + row) * p.sc + 8 * v);
      }
    }
  };

  float sums[CPT] = {};
  fetch(0);
  for (int64_t t0 = 0; t0 < s.len; t0 += TT) {
    const int cnt = (int)(s.len - t0 < TT ? s.len - t0 : TT);
#pragma unroll
    for (int i = 0; i < F::NV; ++i) {
      const int row = tid / F::VB + i * (kThreads / F::VB);
      uint64_t xv[4], dv[4];
      steps_of(dr[i], bias, p.softplus, dv);
      if (row >= cnt)   // tokens that do not exist leave the states as they are
#pragma unroll
        for (int j = 0; j < 4; ++j) dv[j] = 0ull;
      pairs_of(xr[i], xv);
#pragma unroll
      for (int j = 0; j < 4; ++j) xv[j] = mul2(dv[j], xv[j]);
      put8(sd + row * CB + 8 * vec, dv);
      put8(su + row * CB + 8 * vec, xv);
    }
#pragma unroll
    for (int i = 0; i < F::NB; ++i) {
      const int idx = tid + i * kThreads;
      if (idx < (OUT ? 2 : 1) * TT * S / 8) {
        uint64_t v[4];
        pairs_of(br[i], v);
        if (S == 64 && (idx & 4)) {   // see pairs()
          const uint64_t w[4] = {v[2], v[3], v[0], v[1]};
          put8(sbc + 8 * idx, w);
        } else {
          put8(sbc + 8 * idx, v);
        }
      }
    }
    Raw8<T> xo[F::NV], go[F::NV];   // kept for the tile's outputs
#pragma unroll
    for (int i = 0; i < F::NV; ++i) {
      xo[i] = xr[i];
      go[i] = gr[i];
    }
    __syncthreads();
    if (t0 + TT < s.len) fetch(t0 + TT);

    float part[CPT] = {};
    uint64_t lift[2];
    lifts16<CPT>(A, sd + cl, lift);
    // (rows past the last token are zeros: no change.  Four tokens at a time 185 us, two 189)
    const int steps = (cnt + 7) & ~7;
#pragma unroll 8
    for (int t = 0; t < steps; ++t) {
      uint64_t d[CPT], u[CPT], b2[NP], c2[NP];
      twice<CPT>(sd + t * CB + cl, d);
      twice<CPT>(su + t * CB + cl, u);
      pairs<NP>(sbc + t * S + 16 * sl, swap, b2);
      if constexpr (OUT) pairs<NP>(sbc + TT * S + t * S + 16 * sl, swap, c2);
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        uint64_t y;   // (one chain of additions: with two of them 178 us for 176, with four 180)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          uint64_t &e = h[k * NP + i];
          e = fma2(decay(d[k], A[k * NP + i], lift[(k * NP + i) / 4]), e, mul2(u[k], b2[i]));
          if constexpr (OUT) y = i ? fma2(c2[i], e, y) : mul2(c2[i], e);
        }
        if constexpr (OUT) {
          float v = total(y);
#pragma unroll
          for (int m = 1; m < LS; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
          if (LS == 1 || sl == 0) sy[t * CB + cl + k] = v;
        } else {
          float lo, hi;
          unpk(d[k], lo, hi);
          part[k] += lo;
        }
      }
    }
    if constexpr (!OUT)   // a sum of sums over tiles: no long run of one accumulator
#pragma unroll
      for (int k = 0; k < CPT; ++k) sums[k] += part[k];
    __syncthreads();
    if constexpr (OUT) {
      T *y = static_cast<T *>(p.y) + (s.start + t0) * p.D + vch;
#pragma unroll
      for (int i = 0; i < F::NV; ++i) {
        const int row = tid / F::VB + i * (kThreads / F::VB);
        if (!von || row >= cnt) continue;
        uint64_t v[4], yv[4];
        take8(sy + row * CB + 8 * vec, yv);
        if (p.d_skip) {   // (an infinite x has no part in y without a skip)
          pairs_of(xo[i], v);
#pragma unroll
          for (int j = 0; j < 4; ++j) yv[j] = fma2(skip[j], v[j], yv[j]);
        }
        if (gate) {
          pairs_of(go[i], v);
#pragma unroll
          for (int j = 0; j < 4; ++j) yv[j] = mul2(yv[j], mul2(v[j], sigmoid2(v[j])));
        }
        Raw8<T> out;
        set_pairs(out, yv);
        out.store(y + (int64_t)row * p.D);
      }
    }
  }
  if (!OUT) {
    store16(p.seg_x + slot * state + own, on, h);
    if (on && sl == 0)
#pragma unroll
      for (int k = 0; k < CPT; ++k) p.seg_d[(int64_t)slot * p.D + first_ch + cl + k] = sums[k];
  } else if (p.hT && s.seg == s.count - 1) {
    store16(p.hT + s.n * state + own, on, h);
  }
}

template <typename T, int S>
cudaError_t launch_s(const Params &p, int groups, cudaStream_t stream) {
  const dim3 grid(groups * p.blocks, p.seq.slots);
  if (p.seq.seg_len == 0) {
    gdn_ssm_scan_kernel<T, S, true><<<grid, kThreads, 0, stream>>>(p);
    return taken(cudaGetLastError());
  }
  gdn_ssm_scan_kernel<T, S, false><<<grid, kThreads, 0, stream>>>(p);
  const cudaError_t err = taken(cudaGetLastError());
  if (err != cudaSuccess) return err;
  return launch_beside(gdn_ssm_scan_kernel<T, S, true>, grid, kThreads, 0, stream, p);
}
template <typename T>
cudaError_t launch_t(const Params &p, int S, int groups, cudaStream_t stream) {
  switch (S) {
    case 8: return launch_s<T, 8>(p, groups, stream);
    case 16: return launch_s<T, 16>(p, groups, stream);
    case 32: return launch_s<T, 32>(p, groups, stream);
    default: return launch_s<T, 64>(p, groups, stream);
  }
}
constexpr double kFirst = 0.7;   // the first launch forms no outputs
constexpr int kCtas = 3;         // an SM (the outputs' kernel's registers)

// What the segments of a call take behind the status word.
size_t segment_bytes(int32_t num_seqs, int32_t seq_len, bool packed, int32_t channels,
                     int32_t d_state, int32_t groups) {
  const int64_t blocks = (int64_t)groups * channel_blocks(channels / groups, d_state);
  const auto pl = plan(num_seqs, seq_len, packed, blocks, kCtas, kFirst);
  return pl.seg_len ? (size_t)pl.slots * channels * (d_state + 1) * 4 : 0;
}

}  // namespace

bool some_sizes(int32_t num_seqs, int32_t seq_len, int32_t channels, int32_t d_state,
                int32_t groups) {
  return num_seqs > 0 && seq_len >= 0 && channels > 0 && d_state > 0 && groups > 0 &&
         channels % groups == 0 && state_size(d_state);
}
gdn_status check_sizes(int32_t batch, int32_t seq_len, int32_t channels, int32_t d_state,
                       int32_t groups, int32_t num_seqs, const void *cu, gdn_dtype dtype,
                       uint32_t flags) {
  if (batch <= 0 || seq_len < 0 || channels <= 0 || d_state <= 0 || groups <= 0 || num_seqs <= 0)
    return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)GDN_DT_SOFTPLUS) return GDN_ERR_INVALID_ARG;
  if (cu ? batch != 1 : num_seqs != batch) return GDN_ERR_INVALID_ARG;
  if (channels % groups) return GDN_ERR_INVALID_ARG;
  if (!state_size(d_state) || channels / groups % 8) return GDN_ERR_UNSUPPORTED;
  if (num_seqs > 16384 || channels > (1 << 20)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
bool strides_of(Sizes &z, int64_t x, int64_t dt, int64_t b, int64_t c, int64_t gate) {
  z.sx = row_stride(x, z.D, z.e);
  z.sdt = row_stride(dt, z.D, z.e);
  z.sb = row_stride(b, z.gs, z.e);
  z.sc = row_stride(c, z.gs, z.e);
  z.sg = row_stride(gate, z.D, z.e);
  return z.sx && z.sdt && z.sb && z.sc && z.sg;
}

}  // namespace ssm
}  // namespace gdn

extern "C" {

size_t gdn_ssm_workspace_size(int32_t num_seqs, int32_t seq_len, int32_t channels,
                              int32_t d_state, int32_t groups) {
  using namespace gdn::ssm;
  if (!some_sizes(num_seqs, seq_len, channels, d_state, groups)) return 0;
  const size_t dense = segment_bytes(num_seqs, seq_len, false, channels, d_state, groups);
  const size_t packed = segment_bytes(num_seqs, seq_len, true, channels, d_state, groups);
  return gdn::kStatusBytes + (dense > packed ? dense : packed);
}
size_t gdn_ssm_packed_workspace_size(int32_t num_seqs, int32_t total_tokens, int32_t channels,
                                     int32_t d_state, int32_t groups) {
  using namespace gdn::ssm;
  if (!some_sizes(num_seqs, total_tokens, channels, d_state, groups)) return 0;
  return gdn::kStatusBytes +
         segment_bytes(num_seqs, total_tokens, true, channels, d_state, groups);
}

gdn_status gdn_ssm_fwd(const void *x, const void *dt, const float *A_log, const void *b,
                       const void *c, const float *D_skip, const void *gate, const float *dt_bias,
                       const float *initial_state, const int32_t *cu_seqlens, void *y,
                       float *final_state, int32_t batch, int32_t seq_len, int32_t channels,
                       int32_t d_state, int32_t groups, int32_t num_seqs, int64_t x_stride,
                       int64_t dt_stride, int64_t b_stride, int64_t c_stride, int64_t gate_stride,
                       gdn_dtype dtype, uint32_t flags, void *workspace, size_t workspace_bytes,
                       void *stream) {
  using namespace gdn;
  using namespace gdn::ssm;
  const gdn_status st = check_sizes(batch, seq_len, channels, d_state, groups, num_seqs,
                                    cu_seqlens, dtype, flags);
  if (st != GDN_OK) return st;
  Sizes z{(size_t)batch * seq_len, dtype == GDN_F32 ? 4u : 2u, channels,
          (int64_t)groups * d_state};
  z.state = (size_t)num_seqs * channels * d_state * 4;
  if (seq_len == 0) return pass_states(initial_state, final_state, z.state, (cudaStream_t)stream);
  if (!strides_of(z, x_stride, dt_stride, b_stride, c_stride, gate_stride))
    return GDN_ERR_INVALID_ARG;
  if (!x || !dt || !A_log || !b || !c || !y) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {x, dt, A_log, b, c, D_skip, gate, dt_bias, initial_state, cu_seqlens, y,
                        final_state, workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kStatusBytes) return GDN_ERR_WORKSPACE;

  const Range outs[] = {{y, z.rows * channels * z.e}, {final_state, z.state}};
  const Range ins[] = {{x, span_bytes(z.rows, z.sx, z.D, z.e)},
                       {dt, span_bytes(z.rows, z.sdt, z.D, z.e)},
                       {b, span_bytes(z.rows, z.sb, z.gs, z.e)},
                       {c, span_bytes(z.rows, z.sc, z.gs, z.e)},
                       {gate, span_bytes(z.rows, z.sg, z.D, z.e)},
                       {A_log, (size_t)channels * d_state * 4},
                       {D_skip, (size_t)channels * 4},
                       {dt_bias, (size_t)channels * 4},
                       {cu_seqlens, (size_t)(num_seqs + 1) * 4},
                       {initial_state == final_state ? nullptr : initial_state, z.state},
                       {workspace, workspace_bytes}};
  if (!apart(outs, ins)) return GDN_ERR_INVALID_ARG;
  for (int i = 0; i < 10; ++i)
    if (overlaps(ins[10], ins[i])) return GDN_ERR_INVALID_ARG;
  if (overlaps(outs[0], {initial_state, z.state}) || overlaps(ins[10], {initial_state, z.state}))
    return GDN_ERR_INVALID_ARG;

  Params p{};
  p.x = x; p.dt = dt; p.b = b; p.c = c; p.gate = gate;
  p.A_log = A_log; p.d_skip = D_skip; p.dt_bias = dt_bias; p.h0 = initial_state;
  p.y = y; p.hT = final_state;
  p.sx = z.sx; p.sdt = z.sdt; p.sb = z.sb; p.sc = z.sc; p.sg = z.sg;
  p.D = channels;
  p.Dg = channels / groups;
  p.blocks = channel_blocks(p.Dg, d_state);
  p.softplus = flags & GDN_DT_SOFTPLUS;
  p.seq.cu = cu_seqlens;
  p.seq.status = static_cast<DeviceStatus *>(workspace);
  p.seq.seq_len = seq_len;
  p.seq.num_seqs = num_seqs;
  const int64_t blocks = (int64_t)groups * p.blocks;
  const auto pl = plan(num_seqs, seq_len, cu_seqlens != nullptr, blocks, kCtas, kFirst);
  const bool cut = pl.seg_len && (size_t)pl.slots * channels * (d_state + 1) * 4 <=
                                     workspace_bytes - kStatusBytes;
  p.seq.seg_len = cut ? pl.seg_len : 0;
  p.seq.slots = cut ? pl.slots : num_seqs;
  p.seq.ranked = cu_seqlens && !cut && num_seqs > 1 && num_seqs <= lin::kRanked &&
                 blocks * num_seqs > kCtas * kSMs;
  p.seg_x = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kStatusBytes);
  p.seg_d = p.seg_x + (size_t)p.seq.slots * channels * d_state;
  p.keep = initial_state && initial_state == final_state;
  const cudaError_t err = dtype == GDN_F32
                              ? launch_t<float>(p, d_state, groups, (cudaStream_t)stream)
                              : launch_t<__nv_bfloat16>(p, d_state, groups, (cudaStream_t)stream);
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
