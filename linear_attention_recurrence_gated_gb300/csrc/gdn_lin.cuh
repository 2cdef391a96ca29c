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
  int32_t ranked;      // slot z holds the z-th longest packed sequence (uncut ones only)
  // Split along time (seg_len 0: none): sequences are cut into segments of
  // seg_len tokens, whole chunks, each run by CTAs of its own.  A first
  // launch leaves every segment's state increment, run from zero, in seg_x
  // ([scan][slot][H][da][dc]); the second starts each segment from the states of
  // those before it, joined in order: S <- lam^len S + X.  The segments of
  // sequence n have the slots first(n) + 0, 1, ... with first(n) = n ceil(T /
  // seg_len) for dense rows and cu[n] / seg_len + n for packed sequences.
  int64_t seg_len;
  int32_t slots;
  float *seg_x;
  size_t seg_x_bytes;  // room there; calls that need more are not split
};

// What one CTA runs: segment `seg` of `count` of sequence n, its first token and
// length; `total` tokens in the sequence.
struct Span {
  int n, seg, count;
  int64_t start, len, total;
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

// The z-th longest of up to kRanked packed sequences (of equal ones the first).  The
// whole warp together.  (140k tokens in 32 sequences 423 us in their own order, 405 by
// length; 128 of them are four lengths a lane; the limit itself has not been measured.)
constexpr int kRanked = 128;
__device__ __forceinline__ int longest(const Params &p, int z) {
  const int lane = threadIdx.x & 31;
  int len[kRanked / 32], rank[kRanked / 32] = {}, n = 0;
#pragma unroll
  for (int k = 0; k < kRanked / 32; ++k) {
    const int i = 32 * k + lane;
    len[k] = i < p.num_seqs ? p.cu[i + 1] - p.cu[i] : 0;
  }
#pragma unroll
  for (int b = 0; b < kRanked / 32; ++b) {
    const int m = p.num_seqs - 32 * b < 32 ? p.num_seqs - 32 * b : 32;
#pragma unroll 4
    for (int u = 0; u < m; ++u) {
      const int other = __shfl_sync(0xffffffffu, len[b], u);
#pragma unroll
      for (int k = 0; k < kRanked / 32; ++k)
        rank[k] += other > len[k] || (other == len[k] && 32 * b + u < 32 * k + lane);
    }
  }
#pragma unroll
  for (int k = 0; k < kRanked / 32; ++k) {
    const uint32_t is =
        __ballot_sync(0xffffffffu, rank[k] == z && 32 * k + lane < p.num_seqs);
    if (is) n = 32 * k + __ffs(is) - 1;
  }
  return n;
}

// The span of slot z; false if it has none (or the offsets are bad: recorded).
// Uniform over the CTA.
__device__ __forceinline__ bool span_of(const Params &p, int z, int h, Span &s) {
  s.seg = 0;
  s.count = 1;
  s.n = z;
  if (p.seg_len == 0) {
    if (p.ranked) s.n = longest(p, z);
    if (!bounds(p, s.n, h, s.start, s.len)) return false;
    s.total = s.len;
    return true;
  }
  if (p.cu == nullptr) {
    const int segs = (int)((p.seq_len + p.seg_len - 1) / p.seg_len);
    s.n = z / segs;
    s.seg = z % segs;
  } else {
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {  // the last n with first(n) <= z
      const int mid = (lo + hi + 1) / 2;
      if (p.cu[mid] / p.seg_len + mid <= z) lo = mid;
      else hi = mid - 1;
    }
    s.n = lo;
    const int64_t at = z - (p.cu[lo] / p.seg_len + lo);
    int64_t a, b;  // every sequence's bounds are looked at, also one that no slot finds
    if (z < p.num_seqs && z != lo && !bounds(p, z, h, a, b)) return false;
    if (at < 0 || at > p.slots) return false;
    s.seg = (int)at;
  }
  if (!bounds(p, s.n, h, s.start, s.total)) return false;
  s.count = s.total > 0 ? (int)((s.total + p.seg_len - 1) / p.seg_len) : 1;
  if (s.seg >= s.count) return false;
  const int64_t from = s.seg * p.seg_len;
  s.start += from;
  s.len = s.total - from < p.seg_len ? s.total - from : p.seg_len;
  return true;
}

// A scan forward in time may leave its last state where the first one is.  Cut into
// segments, the last one's CTA could then write it before another's has read it: the
// first launch keeps a copy, in the last segment's place in seg_x (which has no
// increment), and the second reads that.
__device__ __forceinline__ bool keeps_copy(const Params &p, const Scan &s) {
  return p.seg_len != 0 && s.s_in != nullptr && s.s_in == s.s_out;
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

// Segments for a launch of `units` CTAs per slot (value tiles and scans, times
// heads) on a GPU that runs `width` of them at a time.  A segment costs its chunks
// of `chunk` tokens, `start` more to begin, and in the first launch the share
// `first` of its chunks; joining reads a state for every segment before.  One
// segment per sequence unless a split gains a tenth.  On the tensor cores a chunk
// of 128 tokens takes some 2 us, a CTA's start 3 of them and the first launch 0.6
// (half the reads, one product of four); on the CUDA cores a chunk of 64 tokens
// takes some 8 us, next to which a start is 0.4.
struct Plan {
  int64_t seg_len;
  int32_t slots;
};
constexpr int kSMs = 152;
constexpr int kSimtWidth = 2 * kSMs;   // CTAs of the CUDA-core form at a time
inline size_t split_bytes(const Plan &plan, int64_t scans, int64_t heads, int64_t dk, int64_t dv) {
  return plan.seg_len ? (size_t)(4 * scans * plan.slots * heads * dk * dv) : 0;
}
inline Plan plan_segments(int64_t num_seqs, int64_t seq_len, bool packed, int64_t units,
                          int64_t width, int64_t chunk, double start, double first) {
  const int64_t rows = packed ? 1 : num_seqs;           // packed: as one long row
  if (units * num_seqs >= 4 * width) return {0, (int32_t)num_seqs};
  const int64_t chunks = (seq_len + chunk - 1) / chunk;
  const auto waves = [&](int64_t ctas) { return (double)((ctas + width - 1) / width); };
  // packed sequences: of their mean length, if they are not cut
  const double whole = packed ? (double)chunks / (double)num_seqs : (double)chunks;
  double best = 0.9 * (waves(units * num_seqs) * (whole + start));
  if (packed && num_seqs * units < width)               // a single one may hold nearly all
    best = 0.9 * ((double)chunks + start);
  Plan plan{0, (int32_t)num_seqs};
  for (int64_t s = 2; s <= 64 && s <= chunks; ++s) {
    const int64_t len = (chunks + s - 1) / s, count = (chunks + len - 1) / len;
    if (count < 2) continue;
    const int64_t slots = packed ? seq_len / (chunk * len) + num_seqs : rows * count;
    const double cost =
        waves(units * slots) * ((double)len + start + 0.03 * start * (double)count) +
        waves(units * rows * (count - 1)) * (first * (double)len + start);
    if (cost < best) {
      best = cost;
      plan = {chunk * len, (int32_t)slots};
    }
  }
  return plan;
}
// Fills in the split of a launch of `tiles` value tiles per scan and head.
inline void split(Params &p, int64_t tiles, int64_t width, int64_t chunk, double start,
                  double first) {
  const Plan plan = plan_segments(p.num_seqs, p.seq_len, p.cu != nullptr,
                                  tiles * p.num_scans * p.num_heads, width, chunk, start, first);
  const bool fits = split_bytes(plan, p.num_scans, p.num_heads, p.scan[0].da, p.scan[0].dc) <=
                    p.seg_x_bytes;
  p.seg_len = fits ? plan.seg_len : 0;
  p.slots = fits ? plan.slots : p.num_seqs;
  // More CTAs than run at a time: those of the longest sequences begin first, or one
  // of them may run alone at the end
  p.ranked = p.cu != nullptr && p.seg_len == 0 && p.num_seqs > 1 && p.num_seqs <= kRanked &&
             tiles * p.num_scans * p.num_heads * p.num_seqs > width;
}

}  // namespace lin
}  // namespace gdn
