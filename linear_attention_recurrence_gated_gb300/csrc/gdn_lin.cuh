// Linear attention with a decay for each head: what the forward, backward and
// decode translation units share.
//
//   S_t = lam S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   lam = exp(log_decay[h])
//
// One scan serves all three directions of the operator.  With "read" rows a,
// "write" rows b and values c (head sizes da, da, dc) it gives
//
//   forward in time:  o_t = sum_{s<=t} lam^(t-s) (a_t.b_s) c_s + lam^(t+1) S_0^T a_t
//                     S_T = lam^T S_0 + sum_s lam^(T-1-s) b_s c_s^T
//   backward in time: o_t = sum_{s>=t} lam^(s-t) (a_t.b_s) c_s + lam^(T-1-t) R_T^T a_t
//                     R_0 = lam^T R_T + sum_s lam^(s+1) b_s c_s^T
//
// The output is the forward scan of (q, k, v) from the initial state; the
// gradients, with G_t = q_t do_t^T + lam G_{t+1} and R = lam G, are scans too:
//   dq: forward  scan of (do, v, k) from the transposed initial state (S_t do_t)
//   dk: backward scan of (v, do, q) from the transposed d_final_state (G_t v_t)
//   dv: backward scan of (k, q, do) from d_final_state            (G_t^T k_t),
//       whose last state is the gradient of the initial state.
//
// Tokens are cut into chunks; inside a chunk the sum over s is a masked
// product, across chunks the state carries.  Powers lam^n are exp(n log_decay)
// with n >= 0 for every decay below one, never a quotient of two powers, so
// they cannot overflow.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {
namespace lin {

// One scan.  Token rows of a, b, c are sa, sb, sc elements apart (head h at
// h * size inside a row), rows of o are H * dc apart.
struct Scan {
  const void *a, *b, *c;
  void *o;
  const float *s_in;   // [N][H] states of da x dc (or transposed), or NULL (zeros)
  float *s_out;        // [N][H][da][dc], or NULL
  int64_t sa, sb, sc;
  int32_t da, dc;
  int32_t s_in_t;      // s_in holds the transposed states, [dc][da]
  int32_t reverse;
};

struct Params {
  Scan scan[3];
  const float *log_decay;
  const int32_t *cu;
  DeviceStatus *status;
  int64_t seq_len;     // tokens of a batch row, or of all packed sequences
  int32_t num_heads, num_seqs, num_scans;
};

// Bounds of sequence n as sequence_bounds (gdn_internal.cuh) gives them.
__device__ __forceinline__ bool bounds(const Params &p, int n, int h, int64_t &start,
                                       int64_t &len) {
  FwdParams f;
  f.cu = p.cu;
  f.seq_len = p.seq_len;
  f.num_seqs = p.num_seqs;
  f.status = p.status;
  return sequence_bounds(f, n, h, start, len);
}

// Element (i, j) of the state of (n, h) that scan s starts from.
__device__ __forceinline__ float state_in(const Scan &s, int64_t unit, int i, int j) {
  if (s.s_in == nullptr) return 0.f;
  const int64_t base = unit * s.da * s.dc;
  return s.s_in[base + (s.s_in_t ? (int64_t)j * s.da + i : (int64_t)i * s.dc + j)];
}

// The tensor-core form: bf16 storage, da 64 or 128, dc a multiple of 64.
bool tc_scan(const Scan &s);
cudaError_t launch_tc(const Params &p, cudaStream_t stream);
cudaError_t launch_simt(const Params &p, gdn_dtype dtype, cudaStream_t stream);

}  // namespace lin
}  // namespace gdn
