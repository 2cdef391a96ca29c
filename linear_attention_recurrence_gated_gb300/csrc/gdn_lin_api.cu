// Host side of the linear-attention entry points of include/gdn.h: argument
// checks, the choice of the kernels and their launches.
#include <stdint.h>

#include "gdn_lin.cuh"

namespace gdn {
gdn_status pass_states(const float *from, float *to, size_t bytes, cudaStream_t s);

namespace lin {
namespace {

struct Range {
  const void *p;
  size_t n;
};
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool overlaps(const Range &a, const Range &b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
bool head_size(int d) { return d >= 32 && d <= 256 && d % 32 == 0; }

// Elements between token rows: 0 stands for densely packed rows.  Returns 0
// for a stride that cannot hold a row or breaks the 16-byte alignment.
int64_t row_stride(int64_t given, int64_t dense, size_t e) {
  if (given == 0) return dense;
  return given >= dense && given * (int64_t)e % 16 == 0 ? given : 0;
}

// The checks that forward and backward share.
gdn_status check_sizes(int32_t batch, int32_t seq_len, int32_t num_heads, int32_t dk, int32_t dv,
                       int32_t num_seqs, const void *cu, gdn_dtype dtype, uint32_t flags) {
  if (batch <= 0 || seq_len < 0 || num_heads <= 0 || dk <= 0 || dv <= 0 || num_seqs <= 0)
    return GDN_ERR_INVALID_ARG;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)GDN_FORCE_SIMT) return GDN_ERR_INVALID_ARG;
  if (cu ? batch != 1 : num_seqs != batch) return GDN_ERR_INVALID_ARG;
  if (!head_size(dk) || !head_size(dv)) return GDN_ERR_UNSUPPORTED;
  if (num_seqs > 16384 || num_heads > 65535) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// Every scan on the tensor cores where its sizes allow, else on the CUDA cores.
cudaError_t launch(const Params &p, gdn_dtype dtype, uint32_t flags, cudaStream_t stream) {
  Params on = p, off = p;
  on.num_scans = off.num_scans = 0;
  for (int i = 0; i < p.num_scans; ++i) {
    const bool tensor = dtype == GDN_BF16 && !(flags & GDN_FORCE_SIMT) && tc_scan(p.scan[i]);
    Params &to = tensor ? on : off;
    to.scan[to.num_scans++] = p.scan[i];
  }
  cudaError_t err = on.num_scans ? launch_tc(on, stream) : cudaSuccess;
  if (err == cudaSuccess && off.num_scans) err = launch_simt(off, dtype, stream);
  return err;
}

}  // namespace
}  // namespace lin
}  // namespace gdn

extern "C" {

size_t gdn_lin_workspace_size(int32_t num_seqs, int32_t seq_len, int32_t num_heads,
                              int32_t head_dim_k, int32_t head_dim_v, uint32_t flags) {
  using namespace gdn::lin;
  if (num_seqs <= 0 || seq_len < 0 || num_heads <= 0 || head_dim_k <= 0 || head_dim_v <= 0)
    return 0;
  (void)flags;   // enough for either form
  // the largest of every launch that a forward or backward call of these sizes
  // may make (packed or not, each storage type)
  size_t most = 0;
  const auto room = [&](const Plan &plan, int scans) {
    const size_t n = split_bytes(plan, scans, num_heads, head_dim_k, head_dim_v);
    most = n > most ? n : most;
  };
  for (int scans = 1; scans <= 3; ++scans)
    for (int d : {head_dim_k, head_dim_v})
      for (int tile : {32, 64})
        for (bool packed : {false, true}) {
          const int64_t units = (int64_t)(d / tile) * scans * num_heads;
          if (units == 0) continue;
          room(plan_segments(num_seqs, seq_len, packed, units, kSimtWidth, 64, 0.4, 0.4), scans);
          if (tile == 64)
            room(plan_segments(num_seqs, seq_len, packed, units, kSMs, 128, 3.0, 0.6), scans);
        }
  return gdn::kStatusBytes + most;
}

gdn_status gdn_lin_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                       const float *initial_state, const int32_t *cu_seqlens, void *o,
                       float *final_state, int32_t batch, int32_t seq_len, int32_t num_heads,
                       int32_t head_dim_k, int32_t head_dim_v, int32_t num_seqs,
                       int64_t q_stride, int64_t k_stride, int64_t v_stride, gdn_dtype dtype,
                       uint32_t flags, void *workspace, size_t workspace_bytes, void *stream) {
  using namespace gdn;
  using namespace gdn::lin;
  gdn_status st = check_sizes(batch, seq_len, num_heads, head_dim_k, head_dim_v, num_seqs,
                              cu_seqlens, dtype, flags);
  if (st != GDN_OK) return st;
  const size_t e = dtype == GDN_F32 ? 4 : 2;
  const int64_t H = num_heads, dk = head_dim_k, dv = head_dim_v;
  const size_t b_state = (size_t)num_seqs * H * dk * dv * 4;
  if (seq_len == 0) return pass_states(initial_state, final_state, b_state, (cudaStream_t)stream);
  const int64_t sq = row_stride(q_stride, H * dk, e), sk = row_stride(k_stride, H * dk, e),
                sv = row_stride(v_stride, H * dv, e);
  if (!sq || !sk || !sv) return GDN_ERR_INVALID_ARG;
  if (!q || !k || !v || !log_decay || !o) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {q, k, v, initial_state, cu_seqlens, o, final_state, log_decay};
  for (const void *x : ptrs)
    if (x && !aligned16(x)) return GDN_ERR_INVALID_ARG;
  if (!workspace) return GDN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDN_ERR_INVALID_ARG;
  if (workspace_bytes < kStatusBytes) return GDN_ERR_WORKSPACE;

  const size_t rows = (size_t)batch * seq_len;
  const Range out = {o, rows * H * dv * e}, sT = {final_state, b_state},
              s0 = {initial_state, b_state};
  const Range inputs[] = {{q, ((rows - 1) * sq + H * dk) * e}, {k, ((rows - 1) * sk + H * dk) * e},
                          {v, ((rows - 1) * sv + H * dv) * e}, {log_decay, (size_t)H * 4},
                          {cu_seqlens, cu_seqlens ? (size_t)(num_seqs + 1) * 4 : 0},
                          {workspace, workspace_bytes}};
  for (const Range &r : inputs)
    if (overlaps(out, r) || overlaps(sT, r)) return GDN_ERR_INVALID_ARG;
  if (overlaps(out, s0) || overlaps(out, sT) || overlaps({workspace, workspace_bytes}, s0))
    return GDN_ERR_INVALID_ARG;
  if (initial_state != final_state && overlaps(s0, sT)) return GDN_ERR_INVALID_ARG;

  Params p{};
  p.scan[0] = {q, k, v, o, initial_state, final_state, sq, sk, sv, head_dim_k, head_dim_v, 0, 0};
  p.num_scans = 1;
  p.log_decay = log_decay;
  p.cu = cu_seqlens;
  p.status = static_cast<DeviceStatus *>(workspace);
  p.seg_x = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kStatusBytes);
  p.seg_x_bytes = workspace_bytes - kStatusBytes;
  p.seq_len = seq_len;
  p.num_heads = num_heads;
  p.num_seqs = num_seqs;
  return launch(p, dtype, flags, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_lin_bwd(const void *q, const void *k, const void *v, const float *log_decay,
                       const float *initial_state, const int32_t *cu_seqlens, const void *d_o,
                       const float *d_final_state, void *dq, void *dk, void *dv,
                       float *d_initial_state, int32_t batch, int32_t seq_len, int32_t num_heads,
                       int32_t head_dim_k, int32_t head_dim_v, int32_t num_seqs, int64_t q_stride,
                       int64_t k_stride, int64_t v_stride, gdn_dtype dtype, uint32_t flags,
                       void *workspace, size_t workspace_bytes, void *stream) {
  using namespace gdn;
  using namespace gdn::lin;
  gdn_status st = check_sizes(batch, seq_len, num_heads, head_dim_k, head_dim_v, num_seqs,
                              cu_seqlens, dtype, flags);
  if (st != GDN_OK) return st;
  const size_t e = dtype == GDN_F32 ? 4 : 2;
  const int64_t H = num_heads, nk = head_dim_k, nv = head_dim_v;
  const size_t b_state = (size_t)num_seqs * H * nk * nv * 4;
  if (seq_len == 0)
    return pass_states(d_final_state, d_initial_state, b_state, (cudaStream_t)stream);
  const int64_t sq = row_stride(q_stride, H * nk, e), sk = row_stride(k_stride, H * nk, e),
                sv = row_stride(v_stride, H * nv, e);
  if (!sq || !sk || !sv) return GDN_ERR_INVALID_ARG;
  if (!q || !k || !v || !log_decay || !d_o || !dq || !dk || !dv) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {q,  k,  v,  log_decay, initial_state, cu_seqlens, d_o, d_final_state,
                        dq, dk, dv, d_initial_state};
  for (const void *x : ptrs)
    if (x && !aligned16(x)) return GDN_ERR_INVALID_ARG;
  if (!workspace) return GDN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDN_ERR_INVALID_ARG;
  if (workspace_bytes < kStatusBytes) return GDN_ERR_WORKSPACE;

  const size_t rows = (size_t)batch * seq_len;
  const Range outs[] = {{dq, rows * H * nk * e}, {dk, rows * H * nk * e}, {dv, rows * H * nv * e},
                        {d_initial_state, b_state}};
  const Range inputs[] = {{q, ((rows - 1) * sq + H * nk) * e}, {k, ((rows - 1) * sk + H * nk) * e},
                          {v, ((rows - 1) * sv + H * nv) * e}, {log_decay, (size_t)H * 4},
                          {cu_seqlens, cu_seqlens ? (size_t)(num_seqs + 1) * 4 : 0},
                          {d_o, rows * H * nv * e}, {initial_state, b_state},
                          {d_final_state, b_state}, {workspace, workspace_bytes}};
  for (int i = 0; i < 4; ++i) {
    for (const Range &r : inputs)
      if (overlaps(outs[i], r)) return GDN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return GDN_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 8; ++i)
    if (overlaps(inputs[8], inputs[i])) return GDN_ERR_INVALID_ARG;

  Params p{};
  const int64_t sdo = H * nv;
  p.scan[0] = {d_o, v, k, dq, initial_state, nullptr, sdo, sv, sk, head_dim_v, head_dim_k, 1, 0};
  p.scan[1] = {v, d_o, q, dk, d_final_state, nullptr, sv, sdo, sq, head_dim_v, head_dim_k, 1, 1};
  p.scan[2] = {k, q, d_o, dv, d_final_state, d_initial_state, sk, sq, sdo, head_dim_k, head_dim_v,
               0, 1};
  p.num_scans = 3;
  p.log_decay = log_decay;
  p.cu = cu_seqlens;
  p.status = static_cast<DeviceStatus *>(workspace);
  p.seg_x = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kStatusBytes);
  p.seg_x_bytes = workspace_bytes - kStatusBytes;
  p.seq_len = seq_len;
  p.num_heads = num_heads;
  p.num_seqs = num_seqs;
  return launch(p, dtype, flags, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
