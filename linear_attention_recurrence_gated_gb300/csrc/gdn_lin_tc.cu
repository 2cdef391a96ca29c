// Linear attention with a decay for each head on the tensor cores: the scan of
// gdn_lin.cuh for bf16 storage, read/write size 64 or 128 and value sizes that
// are multiples of 64.
//
// One CTA owns 64 value columns of one (sequence, head) and walks its chunks of
// C = 128 tokens.  With tile rows i, j, e valid rows and lam^n a table of fp32
// powers, a chunk is four tcgen05 products (M = 128, fp32 accumulators in
// tensor memory):
//   P  = A B^T                        (A, B: the read and write rows)
//   X  = B^T V^                       V^_j = w_j c_j, w_j = lam^(e-1-j) (lam^(j+1) backward)
//   O1 = A S                          S: the state as bf16
//   O2 = P' V                         P'_ij = lam^|i-j| P_ij on the causal side, else 0
//   o_i = lam^(i+1) O1_i + O2_i       (lam^(e-1-i) backward)
//   S  <- lam^e S + X                 (fp32, in registers)
// No product but O1 waits for the state, and X does not, so the serial chain of
// a chunk is one read of X, one multiply-add and one bf16 store of S.
//
// Rounding.  The state is a sum that runs over the whole sequence and is
// returned in fp32, so X must be exact to fp32: b and c are bf16 already, and
// V^ is split into three bf16 terms (8 + 8 + 8 bits of the 24 of w_j c_j), or
// two where what they leave out has decayed below 2^-24 by the returned state, or
// where none is returned (the S that O1 reads has 8 bits).  P' and the S that O1
// reads are rounded to bf16 once: each enters an output that is itself rounded
// to bf16, so an output carries two such roundings in all.
//
// Tile.  128 tokens fill the 128 lanes of tensor memory with P; 64 value columns leave
// room for two stages of a 128-wide head's tiles (227 KB hold five tiles a stage, the
// three terms of V^ and S).  The three tiles of a stage are freed and loaded one by one:
// B after P and X, A after P and O1, V after O2.
//
// Bound.  Head size 64: memory.  [8, 4096, 16 heads, 64/64], 270 MB, takes 49 us, 5.5
// TB/s with the start and the end of its one wave; in between a chunk takes as long as
// its tiles at the copy bandwidth.  Its backward pass takes 139 us (0.48 GB at least;
// three scans ask for twelve tensors' bytes where seven would do, 384 CTAs are 2.5
// waves).  Head size 128: the chain O1, O2, read o, O1 of the next chunk (each
// accumulator is there once: with P in whole columns, twice, X, O1 and O2 fill the 512),
// some 3100 cycles a chunk of which the tensor pipe is busy for half:
//   packed, 140k tokens, 8 heads, 128/256    415 us (1.54 GB: 3.7 TB/s)
//   [1, 65536, 16, 128/128], cut along time  316 us (1.08 GB; 781 us uncut)
//   backward [4, 8192, 16, 128/128]          321 us (0.95 GB; 384 CTAs: 2.5 waves)
// Tried and slower (packed 440 us before each): O1 twice in place of X's second half
// (448 us: X then reads B twice; not tried: P' packed into half of its P, which leaves
// room for a second O1), o by the V^ warps (503 us), shares of equal size handed
// on between resident CTAs (532 us: the heads of one token are no longer read together).
//
// Roles (16 warps): P' (warps 0-3), S and o (4-7), V^ (8-11), TMA (12), and the
// issue of X (13), of P (14), of O1 and O2 (15): none of the three waits for what
// another needs.  V^ and X go by halves, so that one half is weighed while the
// other is multiplied.  Every wait is bounded; a timeout records GDN_ERR_TIMEOUT.
//
// Rows past a sequence's end in its last tile may belong to a neighbour.  Their
// b and c rows are overwritten with zeros before any product reads them as a
// term of a sum (0 * NaN would spoil it); their P' columns are zeros by
// selection, their o rows are not stored.
//
// Values that are not finite.  O2 multiplies every value of the tile, those beyond the
// mask by zero, and 0 * NaN makes NaN of a token's output that only a later token's
// value could spoil.  The o warps look for it (one packed operation for four outputs) and
// take such an output's sum again, over the tokens that it may see (`causal_sums`).  It
// happens in the tile where a bad value first appears; from then on S has it too.  The
// look costs 4 us of 139 ([8, 4096, 16, 64/64] backward) and 6 of 321 (by the V^ warps,
// on the values themselves: 10 in place of 6); such a tile takes 0.35 ms once with
// 64-wide heads and 0.6 with 128-wide ones, latencies of memory one after the other (with
// more loads on their way the call needs registers of the loops: 321 -> 355 us).
#include "gdn_lin.cuh"
#include "gdn_launch.cuh"
#include "gdn_tc_common.cuh"

namespace gdn {
namespace lin {
namespace {

using namespace ptx;
using tc::swz;

constexpr int kC = 128;
constexpr int kTile = kC * 128;   // [128][64] bf16
constexpr int kThreads = 16 * 32;   // 128 registers a thread: P' spilled with 20 warps
constexpr uint32_t kWaitTries = 1u << 19;   // probes of 4 us each before a wait gives up (2 s)
constexpr uint32_t kColP = 0, kColO1 = 256, kColO2 = 320, kColX = 384, kCols = 512;

template <int DK, bool STATES>
struct Lay {
  static constexpr int SUB = DK / 64;
  // The states alone read no A: with DK 128 its room is a third stage's ([1, 65536, 16,
  // 128/128] 340 -> 311 us)
  static constexpr bool NO_A = STATES && DK == 128;
  static constexpr int STAGES = DK == 64 || NO_A ? 3 : 2;
  static constexpr int A = 0, B = NO_A ? 0 : SUB * kTile, V = B + SUB * kTile, STAGE = V + kTile;
  static constexpr int VH = STAGES * STAGE;               // three terms of V^
  static constexpr int S = VH + 3 * kTile;                // [DK][64] bf16
  // the o tile: its own buffer, or (DK 128: no room) the A tile of its stage
  static constexpr int O = S + DK * 128;
  // 32 zeros, lam^0 .. lam^128 (at 32), lam^128 .. lam^0 (at 168), 31 zeros
  static constexpr int TAB = O + (DK == 64 ? kTile : 0);
  static constexpr int BAR = TAB + 328 * 4;
  static constexpr int BYTES = BAR + 384;
  static constexpr int ALLOC = BYTES + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget");
};

// mbarriers
enum Bar { kFullA = 0, kFullB = 3, kFullV = 6, kEmptyA = 9, kEmptyB = 12, kEmptyV = 15, kPFull = 18,
           kPReady = 20, kVhReady = 22, kPFree = 24, kXHalf = 26, kXFull, kClean, kXRead, kSReady,
           kSRead, kOFull, kOFree, kOBuf, kOWritten, kLast, kBars = kLast + 3 };

struct TcArgs {
  Params p;
  CUtensorMap map[3][4];   // a, b, c, o of each scan
  int32_t tiles;           // value tiles of the widest scan
};

struct Waits {
  uint32_t bars;
  volatile int *abort_flag;
  __device__ __forceinline__ uint32_t at(int b) const { return bars + 8 * b; }
};

// Wait for the phase that completes for the `count`-th time (from 0), for at most
// kWaitTries probes.  A wait that gives up leaves its number in the abort flag;
// the CTA reports it as it ends, each role leaving its loop at its own next wait.
// A handful of instructions: every wait of every role is inline, and the roles'
// loops have to fit the instruction cache together.
__device__ __forceinline__ bool wait(const Waits &w, int b, uint32_t count) {
  uint32_t left;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mov.u32 %0, %3;\n"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "sub.u32 %0, %0, 1;\n\t"
      "setp.ne.u32 q, %0, 0;\n\t"
      "@q bra AGAIN;\n"
      "DONE:\n\t}"
      : "=&r"(left)
      : "r"(w.at(b)), "r"(count & 1u), "r"(kWaitTries)
      : "memory");
  if (left == 0) *w.abort_flag = 60 + b;
  return left != 0;
}
// The same for a whole warp that goes on together.
__device__ __forceinline__ bool wait_all(const Waits &w, int b, uint32_t count) {
  return __all_sync(0xffffffffu, wait(w, b, count));
}

// tcgen05.mma by the lane whose `leader` is set.  The whole warp comes here with
// equal operands, so that they stay in uniform registers; issued from a branch
// of one lane each product cost some 70 cycles of moves.
__device__ __forceinline__ void mma(uint32_t leader, uint32_t d, uint64_t a, uint64_t b,
                                    uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ta(uint32_t leader, uint32_t d, uint32_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elect() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(is));
  return is;
}

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  return pair(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t x) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
  return pack_bf16(lo, hi);
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) {
  return *reinterpret_cast<const __nv_bfloat162 *>(&x);
}
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 x) {
  return *reinterpret_cast<const uint32_t *>(&x);
}

// A warp's arrival, after the shared- or tensor-memory accesses of its lanes.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ float power(float ld, float n) { return n == 0.f ? 1.f : expf(ld * n); }

// A tile's row of o once more, for outputs whose O2 is NaN where O1 is not: the sum over
// tokens from the row's own to the tile's first (backward: last of e) of lam^|i-j|
// (a_i.b_j) c_j, in fp32 and from memory, goes over O2 in tensor memory (`t`: the warp's
// lanes of it).  The whole warp together, a row a lane; registers are the caller's, so
// the sums wait in local memory.
__device__ __noinline__ void causal_sums(const Scan &s, int64_t tok, int h, int col0, int e,
                                         const float *lam, uint32_t t) {
  const int i = threadIdx.x & 127, H8 = s.da / 8;
  const bool rev = s.reverse != 0;
  bool some = false;
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    uint32_t x[8], y[8];
    tmem_ld8(t + kColO1 + 8 * q, x);
    tmem_ld8(t + kColO2 + 8 * q, y);
    tmem_wait_ld();
#pragma unroll
    for (int u = 0; u < 8; ++u)
      some = some || (isnan(__uint_as_float(y[u])) && isfinite(__uint_as_float(x[u])));
  }
  some = some && i < e;
  if (!__any_sync(0xffffffffu, some)) return;
  float sum[64];
#pragma unroll 1
  for (int q = 0; q < 64; ++q) sum[q] = 0.f;
  const auto row = [&](const void *p, int64_t stride, int j, int first) {
    return reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) +
                                           (tok + j) * stride + first);
  };
  if (some) {
    const uint4 *ai = row(s.a, s.sa, i, h * s.da);
#pragma unroll 1
    for (int j = i; rev ? j < e : j >= 0; j += rev ? 1 : -1) {
      const uint4 *bj = row(s.b, s.sb, j, h * s.da), *cj = row(s.c, s.sc, j, h * s.dc + col0);
      float p = 0.f;
#pragma unroll 1
      for (int k = 0; k < H8; ++k) {
        const uint4 a = ai[k], b = bj[k];
        const uint32_t as[4] = {a.x, a.y, a.z, a.w}, bs[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          p = fmaf(bf16_lo(as[u]), bf16_lo(bs[u]), p);
          p = fmaf(bf16_hi(as[u]), bf16_hi(bs[u]), p);
        }
      }
      p *= lam[rev ? j - i : i - j];
#pragma unroll 1
      for (int q = 0; q < 8; ++q) {
        const uint4 c = cj[q];
        const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          sum[8 * q + 2 * u] = fmaf(p, bf16_lo(cs[u]), sum[8 * q + 2 * u]);
          sum[8 * q + 2 * u + 1] = fmaf(p, bf16_hi(cs[u]), sum[8 * q + 2 * u + 1]);
        }
      }
    }
  }
  __syncwarp();
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    uint32_t y[8];
    tmem_ld8(t + kColO2 + 8 * q, y);
    tmem_wait_ld();
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (some && isnan(__uint_as_float(y[u]))) y[u] = __float_as_uint(sum[8 * q + u]);
    tmem_st8(t + kColO2 + 8 * q, y);
  }
  tmem_wait_st();
}

// STATES: the first launch of a split along time, which runs a segment from a zero
// state and leaves its state increment (X and S alone).
template <int DK, bool STATES>
__global__ void __launch_bounds__(kThreads, 1)
gdn_lin_tc_kernel(const __grid_constant__ TcArgs args) {
  using L = Lay<DK, STATES>;
  if (STATES) let_second();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t *smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  const Params &p = args.p;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wq = warp & 3;
  const int tile = blockIdx.x % args.tiles, sc = blockIdx.x / args.tiles;
  const int h = blockIdx.y, z = blockIdx.z, H = p.num_heads;
  const Scan &scan = p.scan[sc];
  const int dc = scan.dc, col0 = tile * 64;
  const bool second = !STATES && p.seg_len;   // (a CTA ends after the first launch in any case)
  if (col0 >= dc) {
    if (second) wait_first();
    return;
  }
  const bool rev = scan.reverse != 0;

  Span span;
  if (!span_of(p, z, h, span)) {  // uniform over the CTA
    if (second) wait_first();
    return;
  }
  const int64_t start = span.start, len = span.len;
  const int64_t unit = (int64_t)span.n * H + h;
  // the segment whose end is the sequence's, in the scan's direction
  const bool last = span.seg == (rev ? 0 : span.count - 1);
  const int64_t x_unit = ((int64_t)sc * p.slots + z) * H + h;   // of seg_x
  if (STATES && last) {
    if (keeps_copy(p, scan))
      for (int i = tid; i < DK * 64; i += kThreads) {
        const int64_t at = (int64_t)(i >> 6) * dc + col0 + (i & 63);
        p.seg_x[x_unit * DK * dc + at] = scan.s_in[unit * DK * dc + at];
      }
    return;
  }
  float *const s_out = STATES ? p.seg_x + x_unit * DK * dc
                              : scan.s_out && last ? scan.s_out + unit * DK * dc : nullptr;
  if (len == 0) {  // the state passes through
    if (second) wait_first();
    if (s_out)
      for (int i = tid; i < DK * 64; i += kThreads)
        s_out[(int64_t)(i >> 6) * dc + col0 + (i & 63)] =
            state_in(scan, unit, i >> 6, col0 + (i & 63));
    return;
  }
  const int nc = (int)((len + kC - 1) / kC);
  const int e_last = (int)(len - (int64_t)(nc - 1) * kC);   // rows of the ragged tile
  // tile of step c, and its valid rows
  auto tile_of = [&](int c) { return rev ? nc - 1 - c : c; };
  auto rows_of = [&](int c) { return tile_of(c) == nc - 1 ? e_last : kC; };

  float *lam = reinterpret_cast<float *>(smem + L::TAB) + 32;  // lam^n, n = 0 .. 128
  float *mal = lam + 136;                                      // lam^(128 - n)
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::BAR + 8 * kBars);
  volatile uint32_t *tmem_at = reinterpret_cast<volatile uint32_t *>(smem + L::BAR + 8 * kBars + 8);
  const Waits w{sb + L::BAR, abort_flag};
  const float ld = p.log_decay[h];
  // the tiles of step c into its stage (one thread)
  auto load_ab = [&](int c, bool of_a) {
    const int s = c % L::STAGES, tok = (int)(start + (int64_t)tile_of(c) * kC);
    const uint32_t to = sb + s * L::STAGE + (of_a ? L::A : L::B), full = w.at((of_a ? kFullA : kFullB) + s);
    mbar_arrive_expect_tx(full, L::SUB * kTile);
#pragma unroll
    for (int u = 0; u < L::SUB; ++u)
      tma_load_3d(to + u * kTile, &args.map[sc][of_a ? 0 : 1], 64 * u, h, tok, full);
  };
  auto load_v = [&](int c) {
    const int s = c % L::STAGES, tok = (int)(start + (int64_t)tile_of(c) * kC);
    mbar_arrive_expect_tx(w.at(kFullV + s), kTile);
    tma_load_3d(sb + s * L::STAGE + L::V, &args.map[sc][2], col0, h, tok, w.at(kFullV + s));
  };
  if (tid == 12 * 32) {
    *abort_flag = 0;
    for (int i = 0; i < kBars; ++i) {
      const bool role = i == kPReady || i == kPReady + 1 || i == kVhReady || i == kVhReady + 1 ||
                        i == kClean || i == kXRead || i == kSReady || i == kOFree || i == kOWritten;
      // one arrival per warp; a tile is freed by the two products that read it (V: by
      // O2 and, through V^, by X; A: by the o warps where they use it)
      const bool two = !STATES && i >= kEmptyA && i < kPFull;
      mbar_init(w.at(i), role ? 4 : two ? 2 : 1);
    }
    fence_mbar_init();
    // the first tiles, ahead of the tables and of the other warps
    for (int c = 0; c < L::STAGES && c < nc; ++c) {
      load_ab(c, false);
      load_v(c);
      if (!STATES) load_ab(c, true);
    }
  }
  for (int i = tid; i < 328; i += kThreads) {
    const int up = i - 32, down = 32 + 136 + kC - i;
    const int e = up >= 0 && up <= kC ? up : down >= 0 && down <= kC ? down : -1;
    lam[up] = e < 0 ? 0.f : power(ld, (float)e);
  }
  if (warp == 12) tmem_alloc(sb + L::BAR + 8 * kBars + 8, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const uint32_t tlane = tmem + ((uint32_t)(32 * wq) << 16);
  auto S4 = [&](uint32_t addr) -> uint4 & {
    return *reinterpret_cast<uint4 *>(smem + (addr - sb));
  };

  // Steps from c3 on weigh with three terms, earlier ones with two.  Two leave out up to
  // 2^-16 of what a token writes; it reaches the returned state times lam^rest, rest the
  // tokens that follow the tile.  Below lam^rest = 2^-8 that is 2^-24 of what was written,
  // as much as one fp32 rounding of the state at that time.
  int c3 = nc;
  if (scan.s_out && (STATES || last)) {
    const int64_t after =
        rev ? span.seg * p.seg_len : span.total - span.seg * p.seg_len - len;
    const float reach = ld < 0.f ? 5.5452f / -ld : 1e9f;   // lam^reach = 2^-8
    if (reach >= (float)after) c3 = nc - 2 - (int)(fminf(reach - (float)after, 1e9f) / kC);
  }
  // Where the o tile of step c waits for its store: a buffer of its own, or with DK
  // 128 (no room) the third term's, or while that is in use the A tile of the
  // step's stage.  (Two steps apart from the first third term: the store has read
  // the buffer before the S warps let that step's X begin.)
  auto own_buffer = [&](int c) { return DK == 64 || c + 2 < c3; };
  // Half a row of V^ (columns 32 (t >> 6) .. + 31 of row j): w_j c_j as bf16
  // terms.  A row past the end is zeros, whatever lies there.
  const float w_full[2] = {lam[rev ? (tid & 63) + 1 : kC - 1 - (tid & 63)],
                           lam[rev ? (tid & 63) + 65 : 63 - (tid & 63)]};
  auto weigh = [&](int c, int half, int t) -> bool {
    const int e = rows_of(c), j = 64 * half + (t & 63), q0 = 4 * (t >> 6);
    const uint32_t stage = sb + (c % L::STAGES) * L::STAGE, v = stage + L::V;
    if (e < kC && half == 0) {  // (one ragged tile per sequence)
      if (!wait(w, kFullB + c % L::STAGES, c / L::STAGES)) return false;
      if (t >= e) {
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          S4(swz<kTile>(v, t, 8 * q)) = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int u = 0; u < L::SUB; ++u)
            S4(swz<kTile>(stage + L::B + u * kTile, t, 8 * q)) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();
      warp_arrive(w.at(kClean));
    }
    if (c > 0 && !wait(w, half ? kXFull : kXHalf, c - 1)) return false;  // V^ has been read
    float wj = half ? w_full[1] : w_full[0];
    if (e < kC) wj = j < e ? lam[rev ? j + 1 : e - 1 - j] : 0.f;
    const uint32_t to = sb + L::VH;
    if (c < c3) {
      // two terms on bf16 pairs: with w = wa + wb (8 bits each), t1 = c wa rounded
      // and its remainder c wa - t1 are exact together, t2 = c wb + remainder
      const __nv_bfloat162 wa = __float2bfloat162_rn(wj),
                           wb = __float2bfloat162_rn(wj - __low2float(wa));
      uint4 x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        x[q] = j < e ? S4(swz<kTile>(v, j, 8 * (q0 + q))) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t xs[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
        uint32_t t1[4], t2[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const __nv_bfloat162 y = as_bf162(xs[u]), m = __hmul2_rn(y, wa);
          t1[u] = bits(m);
          t2[u] = bits(__hfma2(y, wb, __hfma2(y, wa, __hneg2(m))));
        }
        S4(swz<kTile>(to, j, 8 * (q0 + q))) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
        S4(swz<kTile>(to, j, 8 * (q0 + q)) + kTile) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
      }
    } else {
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const uint4 x = j < e ? S4(swz<kTile>(v, j, 8 * (q0 + q))) : make_uint4(0, 0, 0, 0);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
        uint32_t t1[4], t2[4], t3[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float lo = bf16_lo(xs[u]) * wj, hi = bf16_hi(xs[u]) * wj;
          t1[u] = pack_bf16(lo, hi);
          lo -= bf16_lo(t1[u]);
          hi -= bf16_hi(t1[u]);
          t2[u] = pack_bf16(lo, hi);
          t3[u] = pack_bf16(lo - bf16_lo(t2[u]), hi - bf16_hi(t2[u]));
        }
        const uint32_t at = swz<kTile>(to, j, 8 * (q0 + q));
        S4(at) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
        S4(at + kTile) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
        S4(at + 2 * kTile) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
      }
    }
    fence_proxy_async_smem();
    warp_arrive(w.at(kVhReady + half));
    return true;
  };

  // P' : lane l of a group's warp w holds row i = 32 w + l; columns in units of 16
  // from the diagonal outwards (k = 0, 1: the diagonal block), the next one on its
  // way while one is weighed.  At a distance of d units from the row's own,
  // lam^|i-j| = (lam^|i - edge| lam^(16 (d-1))) lam^|edge - j| with the edge
  // between them, so 16 powers of the column, 16 of the triangle (d = 0) and a
  // running scalar serve them all, from registers.  A unit of P' (two columns a
  // word) goes over the first half of its own P.
  const int l16 = lane & 15;
  const int units = rev ? 8 - 2 * wq : 2 * wq + 2;
  const uint32_t half16 = lane >> 4;
  auto unit_at = [&](int k) { return rev ? 2 * wq + k : 2 * wq + 1 - k; };
  auto drop = [&](uint32_t (&pk)[8], uint32_t keep) {
    // columns that do not count, by selection: a product with 0 keeps a NaN
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      if (!(keep & (1u << (2 * x)))) pk[x] &= 0xffff0000u;
      if (!(keep & (2u << (2 * x)))) pk[x] &= 0xffffu;
    }
  };
  auto ragged = [&](int e, int u) { return e > 16 * u ? 0xffffu >> (16 * u + 16 - e) : 0u; };
  auto far_unit = [&](uint32_t P, int k, int e, float &sd, const uint64_t (&g)[8],
                      const uint32_t (&v)[16]) {
    const int u = unit_at(k);
    uint32_t pk[8];
    const uint64_t s2 = pair(sd, sd);
#pragma unroll
    for (int x = 0; x < 8; ++x)
      pk[x] = pack_pair(mul2(pair(v[2 * x], v[2 * x + 1]), mul2(s2, g[x])));
    if (e < 16 * u + 16) drop(pk, ragged(e, u));
    tmem_st8(P + 16 * u, pk);
    sd *= lam[16];
  };
  // units k0 .. k1 - 1 (an even number), all beyond the diagonal block
  auto far_units = [&](uint32_t P, int k0, int k1, int e, float sd, const uint64_t (&g)[8]) {
    uint32_t va[16], vb[16];
    tmem_ld16(P + 16 * unit_at(k0), va);
#pragma unroll 1
    for (int k = k0; k < k1; k += 2) {
      tmem_wait_ld();
      tmem_ld16(P + 16 * unit_at(k + 1), vb);
      far_unit(P, k, e, sd, g, va);
      tmem_wait_ld();
      if (k + 2 < k1) tmem_ld16(P + 16 * unit_at(k + 2), va);
      far_unit(P, k + 1, e, sd, g, vb);
    }
  };
  uint64_t g[8];
#pragma unroll
  for (int x = 0; x < 8; ++x)
    g[x] = rev ? pair(lam[2 * x], lam[2 * x + 1]) : pair(lam[16 - 2 * x], lam[15 - 2 * x]);
  // the running scalar of unit k of this lane (k >= 2)
  auto scalar_at = [&](int k) {
    const int d = k - (int)(rev ? half16 : 1 - half16);
    return lam[(rev ? 16 - l16 : l16) + 16 * (d - 1)];
  };

  if (warp < 4) {
    if constexpr (!STATES) {
    // ---- P' ----
    uint64_t tri[8];   // (the table's zeros on the far side; they are not kept)
#pragma unroll
    for (int x = 0; x < 8; ++x)
      tri[x] = rev ? pair(lam[2 * x - l16], lam[2 * x + 1 - l16])
                   : pair(mal[kC + 2 * x - l16], mal[kC + 2 * x + 1 - l16]);
    const uint32_t tri_keep = rev ? 0xffffu << l16 : 0xffffu >> (15 - l16);
    const float s_far = units > 2 ? scalar_at(2) : 0.f, s_near = lam[rev ? 16 - l16 : l16];
    const bool mine = rev ? half16 == 0 : half16 == 1;   // k = 0 holds this lane's triangle
    for (int c = 0; c < nc; ++c) {
      const int b = c & 1, e = rows_of(c);
      if (!wait(w, kPFull + b, c >> 1)) break;
      tc_fence_after();
      const uint32_t P = tlane + kColP + 128 * b;
      uint32_t va[16], vb[16], pk[8];
      tmem_ld16(P + 16 * unit_at(0), va);
      tmem_ld16(P + 16 * unit_at(1), vb);
      tmem_wait_ld();
#pragma unroll
      for (int x = 0; x < 8; ++x) pk[x] = pack_pair(mul2(pair(va[2 * x], va[2 * x + 1]), tri[x]));
      drop(pk, (mine ? tri_keep : 0u) & (e < 16 * unit_at(0) + 16 ? ragged(e, unit_at(0)) : ~0u));
      tmem_st8(P + 16 * unit_at(0), pk);
      const uint64_t s2 = pair(s_near, s_near);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint64_t wt = mul2(s2, g[x]);
        pk[x] = pack_pair(mul2(pair(vb[2 * x], vb[2 * x + 1]), mine ? wt : tri[x]));
      }
      drop(pk, (mine ? 0xffffu : tri_keep) & (e < 16 * unit_at(1) + 16 ? ragged(e, unit_at(1)) : ~0u));
      tmem_st8(P + 16 * unit_at(1), pk);
      if (units > 2) far_units(P, 2, units, e, s_far, g);
      const uint32_t zero[8] = {};
#pragma unroll 1
      for (int u = rev ? 0 : 2 * wq + 2; u < (rev ? 2 * wq : 8); ++u) tmem_st8(P + 16 * u, zero);
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(w.at(kPReady + b));
    }
    }
  } else if (warp < 8) {
    // ---- S and o ----
    // DK 128: lane i holds row i of S, 64 columns; DK 64: X holds its rows
    // twice, lanes 0-63 take columns 0-31 of them and lanes 64-127 the others
    constexpr int N = DK == 64 ? 32 : 64;
    const int si = (32 * wq + lane) & (DK - 1), c0 = DK == 64 ? 32 * (wq >> 1) : 0;
    uint64_t s[N / 2];   // pairs of columns
#pragma unroll
    for (int x = 0; x < N / 2; ++x) s[x] = 0;
    const auto add_row = [&](const float *state, float f) {  // s <- f s + row si of it
      const float4 *row = reinterpret_cast<const float4 *>(state + (int64_t)si * dc + col0 + c0);
#pragma unroll
      for (int x = 0; x < N / 4; ++x) {
        const float4 y = row[x];
        s[2 * x] = fma2(pair(f, f), s[2 * x], pair(y.x, y.y));
        s[2 * x + 1] = fma2(pair(f, f), s[2 * x + 1], pair(y.z, y.w));
      }
    };
    if (second) wait_first();
    if (!STATES && scan.s_in) {
      if (scan.s_in_t) {
        const float *at = scan.s_in + unit * DK * dc + (int64_t)(col0 + c0) * DK + si;
#pragma unroll
        for (int x = 0; x < N / 2; ++x) s[x] = pair(at[2 * x * DK], at[(2 * x + 1) * DK]);
      } else {
        add_row(keeps_copy(p, scan)
                    ? p.seg_x + (x_unit + (int64_t)(span.count - 1 - span.seg) * H) * DK * dc
                    : scan.s_in + unit * DK * dc,
                0.f);
      }
    }
    if (!STATES)  // the segments before this one, in order
      for (int k = rev ? span.count - 1 : 0; k != span.seg; k += rev ? -1 : 1) {
        const int64_t length = k == span.count - 1 ? span.total - k * p.seg_len : p.seg_len;
        add_row(p.seg_x + (x_unit + (int64_t)(k - span.seg) * H) * DK * dc,
                power(ld, (float)length));
      }
    auto put = [&]() {
#pragma unroll
      for (int q = 0; q < N / 8; ++q)
        S4(swz<kTile>(sb + L::S, si, c0 + 8 * q)) =
            make_uint4(pack_pair(s[4 * q]), pack_pair(s[4 * q + 1]), pack_pair(s[4 * q + 2]),
                       pack_pair(s[4 * q + 3]));
      fence_proxy_async_smem();
      warp_arrive(w.at(kSReady));
    };
    if (!STATES) put();
    const float lam_c = lam[kC];
    // o : lane i holds row i
    const int i = 32 * wq + lane;
    const bool lead = warp == 4 && lane == 0;
    const CUtensorMap *mo = &args.map[sc][3];
    const float f_full = lam[rev ? kC - 1 - i : i + 1];
    int stores = 0, own_stores = 0;  // whole tiles so far
    int done = 0;
    for (int c = 0; c < nc; ++c) {
      const int e = rows_of(c);
      if (!wait(w, kXFull, c)) break;
      tc_fence_after();
      const float le = e == kC ? lam_c : lam[e];
#pragma unroll
      for (int q = 0; q < N / 8; ++q) {
        uint32_t x[8], y[8];  // first (and third) term's sum; the second's
        tmem_ld8(tlane + kColX + c0 + 8 * q, x);
        tmem_ld8(tlane + kColX + 64 + c0 + 8 * q, y);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 4; ++u)
          s[4 * q + u] = fma2(pair(le, le), s[4 * q + u],
                              add2(pair(x[2 * u], x[2 * u + 1]), pair(y[2 * u], y[2 * u + 1])));
      }
      tc_fence_before();
      warp_arrive(w.at(kXRead));
      if (STATES) {
        ++done;
        continue;
      }
      const int64_t tok = start + (int64_t)tile_of(c) * kC;
      const uint32_t stage = sb + (c % L::STAGES) * L::STAGE;
      const bool own = own_buffer(c);
      const uint32_t so = DK == 64 ? sb + L::O : own ? sb + L::VH + 2 * kTile : stage + L::A;
      float f = f_full;
      if (e < kC) f = i < e ? lam[rev ? e - 1 - i : i + 1] : 0.f;
      if (own && e == kC) {  // the last store has read the buffer
        if (lead) {
          bulk_wait_read<0>();
          mbar_arrive(w.at(kOBuf));
        }
        if (!wait(w, kOBuf, own_stores)) break;
        ++own_stores;
      }
      if (c + 1 < nc) {
        if (!wait(w, kSRead, c)) break;   // O1 has read the last state
        put();
      }
      if (!wait(w, kOFull, c)) break;
      tc_fence_after();
      ++done;
      uint4 *row = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(scan.o) +
                                             ((tok + i) * H + h) * dc + col0);
#pragma unroll 1
      for (bool again = false;; again = true) {
        __nv_bfloat162 bad = __float2bfloat162_rn(0.f);   // NaN once one has been read
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t x[16], y[16], out[8];
          tmem_ld16(tlane + kColO1 + 16 * q, x);
          tmem_ld16(tlane + kColO2 + 16 * q, y);
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            out[u] = pack_pair(fma2(pair(f, f), pair(x[2 * u], x[2 * u + 1]),
                                    pair(y[2 * u], y[2 * u + 1])));
#pragma unroll
          for (int u = 0; u < 8; u += 2) bad = __hfma2(as_bf162(out[u]), as_bf162(out[u + 1]), bad);
          const uint4 lo = make_uint4(out[0], out[1], out[2], out[3]),
                      hi = make_uint4(out[4], out[5], out[6], out[7]);
          if (e == kC) {
            S4(swz<kTile>(so, i, 16 * q)) = lo;
            S4(swz<kTile>(so, i, 16 * q + 8)) = hi;
          } else if (i < e) {
            row[2 * q] = lo;
            row[2 * q + 1] = hi;
          }
        }
        const bool nan = __hisnan(__low2bfloat16(bad)) || __hisnan(__high2bfloat16(bad));
        if (again || !__any_sync(0xffffffffu, nan && i < e)) break;
        causal_sums(scan, tok, h, col0, e, lam, tlane);
      }
      tc_fence_before();
      warp_arrive(w.at(kOFree));
      if (e == kC) {
        fence_proxy_async_smem();
        warp_arrive(w.at(kOWritten));
        if (lead) {
          if (!wait(w, kOWritten, stores)) break;
          tma_store_3d(mo, col0, h, (int)tok, so);
          bulk_commit();
        }
        ++stores;
      }
      if (DK == 128 && lead && (!own || !own_buffer(c + 1))) {
        bulk_wait_read<0>();
        if (!own) mbar_arrive(w.at(kEmptyA + c % L::STAGES));
      }
    }
    if (lead) bulk_wait_all();
    if (s_out && done == nc) {
      ulonglong2 *row = reinterpret_cast<ulonglong2 *>(s_out + (int64_t)si * dc + col0 + c0);
#pragma unroll
      for (int x = 0; x < N / 4; ++x) row[x] = make_ulonglong2(s[2 * x], s[2 * x + 1]);
    }
  } else if (warp < 12) {
    // ---- V^ ----
    for (int c = 0; c < nc; ++c) {
      if (!wait(w, kFullV + c % L::STAGES, c / L::STAGES) || !weigh(c, 0, tid & 127) ||
          !weigh(c, 1, tid & 127))
        break;
    }
  } else if (warp == 12) {
    // ---- TMA ----
    if (lane == 0) {
      const int ahead = nc < L::STAGES ? nc : L::STAGES;
      int in_a = STATES ? 0 : ahead, in_b = ahead, in_v = ahead;   // steps loaded
      for (int c = L::STAGES; c < nc; ++c) {
        const int s = c % L::STAGES, round = c / L::STAGES - 1;
        if (!wait(w, kEmptyB + s, round)) break;
        load_ab(c, false);
        ++in_b;
        if (!STATES) {
          if (!wait(w, kEmptyA + s, round)) break;
          load_ab(c, true);
          ++in_a;
        }
        if (!wait(w, kEmptyV + s, round)) break;
        load_v(c);
        ++in_v;
      }
      // loads still in flight land before the CTA leaves
      auto landed = [&](int bar, int n) {
        for (int c = n > L::STAGES ? n - L::STAGES : 0; c < n; ++c)
          wait(w, bar + c % L::STAGES, c / L::STAGES);
      };
      landed(kFullA, in_a);
      landed(kFullB, in_b);
      landed(kFullV, in_v);
    }
  } else if (warp == 13) {
    // ---- issue of X: the warp together, one lane elected ----
    const uint32_t leader = elect();
    bool ok = true;
    int s = 0;
    for (int c = 0; ok && c < nc; ++c) {
      const uint32_t stage = sb + s * L::STAGE;
      if (!(ok = wait_all(w, kFullB + s, c / L::STAGES))) break;
      // X in two halves of 64 tokens; the first two terms side by side (N = 128:
      // one read of B for both), the third onto the first
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        ok = ok && wait_all(w, kVhReady + half, c) &&
             (half > 0 || c == 0 || wait_all(w, kXRead, c - 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t dx = umma_desc_sw128_mn(stage + L::B + half * 8192, DK == 64 ? 0 : kTile),
                       dv = umma_desc_sw128_mn(sb + L::VH + half * 8192, kTile);
#pragma unroll 1
        for (int kk = 0; kk < 4; ++kk)
          mma(leader, tmem + kColX, dx + 128 * kk, dv + 128 * kk, umma_idesc_bf16(128, 128, 1, 1),
              half + kk > 0);
        if (c >= c3) {
#pragma unroll 1
          for (int kk = 0; kk < 4; ++kk)
            mma(leader, tmem + kColX, dx + 128 * kk, dv + 2 * (kTile >> 4) + 128 * kk,
                umma_idesc_bf16(128, 64, 1, 1), 1);
        }
        if (leader) {
          umma_commit(w.at(half ? kXFull : kXHalf));
          if (half) {
            umma_commit(w.at(kEmptyB + s));
            umma_commit(w.at(kEmptyV + s));
          }
        }
        __syncwarp();
      }
      if (++s == L::STAGES) s = 0;
    }
    // products still in flight end before the CTA leaves
    if (leader) {
      umma_commit(w.at(kLast));
      wait(w, kLast, 0);
    }
    __syncwarp();
  } else if (!STATES && warp == 14) {
    // ---- issue of P ----
    const uint32_t leader = elect();
    int s = 0;
    for (int c = 0; c < nc; ++c) {
      const uint32_t stage = sb + s * L::STAGE;
      // the P buffer is free once O2 of the chunk before last has read it
      if (!wait_all(w, kFullA + s, c / L::STAGES) || !wait_all(w, kFullB + s, c / L::STAGES) ||
          (c >= 2 && !wait_all(w, kPFree + (c & 1), (c >> 1) - 1)) ||
          (rows_of(c) < kC && !wait_all(w, kClean, 0)))
        break;
      tc_fence_after();
      const uint64_t da = umma_desc_sw128(stage + L::A), db = umma_desc_sw128(stage + L::B);
#pragma unroll 1
      for (int u = 0; u < L::SUB; ++u)
#pragma unroll 1
        for (int kk = 0; kk < 4; ++kk)
          mma(leader, tmem + kColP + 128 * (c & 1), da + u * (kTile >> 4) + 2 * kk,
              db + u * (kTile >> 4) + 2 * kk, umma_idesc_bf16(128, 128), u + kk > 0);
      if (leader) {
        umma_commit(w.at(kPFull + (c & 1)));
        umma_commit(w.at(kEmptyA + s));
        umma_commit(w.at(kEmptyB + s));
      }
      __syncwarp();
      if (++s == L::STAGES) s = 0;
    }
    if (leader) {
      umma_commit(w.at(kLast + 2));
      wait(w, kLast + 2, 0);
    }
    __syncwarp();
  } else if (!STATES) {
    // ---- issue of O1 and O2 ----
    const uint32_t leader = elect();
    int s = 0;
    for (int c = 0; c < nc; ++c) {
      const uint32_t stage = sb + s * L::STAGE;
      if (!wait_all(w, kFullA + s, c / L::STAGES) || !wait_all(w, kFullV + s, c / L::STAGES) ||
          !wait_all(w, kSReady, c) || (c > 0 && !wait_all(w, kOFree, c - 1)))
        break;
      tc_fence_after();
      const uint64_t da = umma_desc_sw128(stage + L::A), ds = umma_desc_sw128_mn(sb + L::S, 8192),
                     dv = umma_desc_sw128_mn(stage + L::V, 8192);
#pragma unroll 1
      for (int u = 0; u < L::SUB; ++u)
#pragma unroll 1
        for (int kk = 0; kk < 4; ++kk)
          mma(leader, tmem + kColO1, da + u * (kTile >> 4) + 2 * kk, ds + 512 * u + 128 * kk,
              umma_idesc_bf16(128, 64, 0, 1), u + kk > 0);
      if (leader) {
        umma_commit(w.at(kSRead));
        if (own_buffer(c)) umma_commit(w.at(kEmptyA + s));
      }
      __syncwarp();
      if (!wait_all(w, kPReady + (c & 1), c >> 1)) break;
      tc_fence_after();
#pragma unroll 1
      for (int kk = 0; kk < kC / 16; ++kk)
        mma_ta(leader, tmem + kColO2, tmem + kColP + 128 * (c & 1) + 16 * kk,
               dv + 128 * kk,
               umma_idesc_bf16(128, 64, 0, 1), kk > 0);
      if (leader) {
        umma_commit(w.at(kOFull));
        umma_commit(w.at(kPFree + (c & 1)));
        umma_commit(w.at(kEmptyV + s));
      }
      __syncwarp();
      if (++s == L::STAGES) s = 0;
    }
    if (leader) {
      umma_commit(w.at(kLast + 1));
      wait(w, kLast + 1, 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag)
    report(p.status, GDN_ERR_TIMEOUT, (uint32_t)span.n, (uint32_t)h, (uint32_t)*abort_flag);
  if (warp == 12) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// [tokens][heads][cols] bf16, token rows `stride` elements apart, as a 3-D
// tensor; box = 64 cols x 1 head x 128 tokens.
bool make_map(CUtensorMap *m, const void *ptr, int cols, int heads, int64_t tokens,
              int64_t stride) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, kC};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, bool STATES>
cudaError_t run(const TcArgs &args, cudaStream_t stream) {
  constexpr auto kernel = gdn_lin_tc_kernel<DK, STATES>;
  const cudaError_t err = allow_smem<kernel>(Lay<DK, STATES>::ALLOC);
  if (err != cudaSuccess) return err;
  const dim3 grid(args.tiles * args.p.num_scans, args.p.num_heads, args.p.slots);
  if (!STATES && args.p.seg_len)
    return launch_beside(kernel, grid, kThreads, Lay<DK, STATES>::ALLOC, stream, args);
  kernel<<<grid, kThreads, Lay<DK, STATES>::ALLOC, stream>>>(args);
  return cudaGetLastError();
}

template <int DK>
cudaError_t launch_dk(const Params &p, cudaStream_t stream) {
  TcArgs args;
  args.p = p;
  args.p.num_scans = 0;
  args.tiles = 0;
  const int64_t tokens = p.cu ? p.seq_len : (int64_t)p.num_seqs * p.seq_len;
  for (int i = 0; i < p.num_scans; ++i) {
    const Scan &s = p.scan[i];
    if (s.da != DK) continue;
    const int at = args.p.num_scans++;
    args.p.scan[at] = s;
    if (!make_map(&args.map[at][0], s.a, s.da, p.num_heads, tokens, s.sa) ||
        !make_map(&args.map[at][1], s.b, s.da, p.num_heads, tokens, s.sb) ||
        !make_map(&args.map[at][2], s.c, s.dc, p.num_heads, tokens, s.sc) ||
        !make_map(&args.map[at][3], s.o, s.dc, p.num_heads, tokens, (int64_t)p.num_heads * s.dc))
      return cudaErrorInvalidValue;
    if (s.dc / 64 > args.tiles) args.tiles = s.dc / 64;
  }
  if (args.p.num_scans == 0) return cudaSuccess;
  split(args.p, args.tiles, kSMs, kC, 3.0, 0.6);
  if (args.p.seg_len) {
    const cudaError_t err = run<DK, true>(args, stream);
    if (err != cudaSuccess) return err;
  }
  return run<DK, false>(args, stream);
}

}  // namespace

bool tc_scan(const Scan &s) { return (s.da == 64 || s.da == 128) && s.dc % 64 == 0; }

cudaError_t launch_tc(const Params &p, cudaStream_t stream) {
  const cudaError_t err = launch_dk<64>(p, stream);
  return err == cudaSuccess ? launch_dk<128>(p, stream) : err;
}

}  // namespace lin
}  // namespace gdn
