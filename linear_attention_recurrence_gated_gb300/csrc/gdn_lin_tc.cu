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
// V^ is split into three bf16 terms (8 + 8 + 8 bits of the 24 of w_j c_j).  P'
// and the S that O1 reads are rounded to bf16 once: each enters an output that
// is itself rounded to bf16, so an output carries two such roundings in all.
//
// Roles (18 warps): P' (warps 0-3), o (4-7), V^ (8-11), S (12-15), TMA (16),
// MMA issue (17).  Every wait is bounded; a timeout records GDN_ERR_TIMEOUT,
// raises the abort flag and every role leaves its loop.
//
// Rows past a sequence's end in its last tile may belong to a neighbour.  Their
// b and c rows are overwritten with zeros before any product reads them as a
// term of a sum (0 * NaN would spoil it); their P' columns are zeros by
// selection, their o rows are not stored.
#include "gdn_lin.cuh"
#include "gdn_tc_common.cuh"

namespace gdn {
namespace lin {
namespace {

using namespace ptx;
using tc::kWaitTimeoutNs;
using tc::swz;

constexpr int kC = 128;
constexpr int kTile = kC * 128;   // [128][64] bf16
constexpr int kThreads = 18 * 32;
constexpr uint32_t kColP = 0, kColO1 = 256, kColO2 = 320, kColX = 384, kCols = 512;

template <int DK>
struct Lay {
  static constexpr int SUB = DK / 64;
  static constexpr int STAGES = DK == 64 ? 3 : 2;
  static constexpr int A = 0, B = SUB * kTile, V = 2 * SUB * kTile, STAGE = (2 * SUB + 1) * kTile;
  static constexpr int VH = STAGES * STAGE;               // three terms of V^
  static constexpr int S = VH + 3 * kTile;                // [DK][64] bf16
  // the o tile: its own buffer, or (DK 128: no room) the A tile of its stage
  static constexpr int O = S + DK * 128;
  static constexpr int TAB = O + (DK == 64 ? kTile : 0);  // lam^0 .. lam^128, then reversed
  static constexpr int BAR = TAB + 272 * 4;
  static constexpr int BYTES = BAR + 256;
  static constexpr int ALLOC = BYTES + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget");
};

// mbarriers
enum Bar { kFull = 0, kEmpty = 3, kPFull = 6, kPReady = 8, kClean = 10, kVhReady, kXFull, kXRead,
           kSReady, kOFull, kOFree, kOBuf, kOWritten, kLast, kBars };

struct TcArgs {
  Params p;
  CUtensorMap map[3][4];   // a, b, c, o of each scan
  int32_t tiles;           // value tiles of the widest scan
};

struct Waits {
  uint32_t bars;
  volatile int *abort_flag;
  DeviceStatus *status;
  int n, h;
  __device__ __forceinline__ uint32_t at(int b) const { return bars + 8 * b; }
};

__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                       DeviceStatus *status, int n, int h, uint32_t where) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 15u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
        *abort_flag = 1;
        report(status, GDN_ERR_TIMEOUT, (uint32_t)n, (uint32_t)h, where);
        return false;
      }
    }
  }
}
// Wait for the phase that completes for the `count`-th time (from 0).
__device__ __forceinline__ bool wait(const Waits &w, int b, uint32_t count) {
  const uint32_t parity = count & 1u;
  if (mbar_try_wait(w.at(b), parity)) return true;
  return wait_slow(w.at(b), parity, w.abort_flag, w.status, w.n, w.h, 60u + (uint32_t)b);
}

__device__ __forceinline__ float power(float ld, float n) { return n == 0.f ? 1.f : expf(ld * n); }

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
gdn_lin_tc_kernel(const __grid_constant__ TcArgs args) {
  using L = Lay<DK>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t *smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  const Params &p = args.p;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wq = warp & 3;
  const int tile = blockIdx.x % args.tiles, sc = blockIdx.x / args.tiles;
  const int h = blockIdx.y, n = blockIdx.z, H = p.num_heads;
  const Scan &scan = p.scan[sc];
  const int dc = scan.dc, col0 = tile * 64;
  if (col0 >= dc) return;
  const bool rev = scan.reverse != 0;
  const int64_t unit = (int64_t)n * H + h;

  int64_t start, len;
  if (!bounds(p, n, h, start, len)) return;  // uniform over the CTA
  if (len == 0) {  // the state passes through
    if (scan.s_out)
      for (int i = tid; i < DK * 64; i += kThreads)
        scan.s_out[unit * DK * dc + (int64_t)(i >> 6) * dc + col0 + (i & 63)] =
            state_in(scan, unit, i >> 6, col0 + (i & 63));
    return;
  }
  const int nc = (int)((len + kC - 1) / kC);
  const int e_last = (int)(len - (int64_t)(nc - 1) * kC);   // rows of the ragged tile
  // tile of step c, and its valid rows
  auto tile_of = [&](int c) { return rev ? nc - 1 - c : c; };
  auto rows_of = [&](int c) { return tile_of(c) == nc - 1 ? e_last : kC; };

  float *lam = reinterpret_cast<float *>(smem + L::TAB);    // lam^n, n = 0 .. 128
  float *mal = lam + 136;                                   // lam^(128 - n)
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::BAR + 8 * kBars);
  volatile uint32_t *tmem_at = reinterpret_cast<volatile uint32_t *>(smem + L::BAR + 8 * kBars + 8);
  const Waits w{sb + L::BAR, abort_flag, p.status, n, h};
  const float ld = p.log_decay[h];
  for (int i = tid; i <= kC; i += kThreads) {
    const float x = power(ld, (float)i);
    lam[i] = x;
    mal[kC - i] = x;
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kBars; ++i) {
      const bool all = i == kPReady || i == kPReady + 1 || i == kClean || i == kVhReady ||
                       i == kXRead || i == kSReady || i == kOFree || i == kOWritten;
      mbar_init(w.at(i), all ? 128 : 1);
    }
    fence_mbar_init();
  }
  if (warp == 17) tmem_alloc(sb + L::BAR + 8 * kBars + 8, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const uint32_t tlane = tmem + ((uint32_t)(32 * wq) << 16);
  auto S4 = [&](uint32_t addr) -> uint4 & {
    return *reinterpret_cast<uint4 *>(smem + (addr - sb));
  };

  if (warp < 4) {
    // ---- P' : lane l of warp w holds row 32 w + l; columns in blocks of 32 ----
    for (int c = 0; c < nc; ++c) {
      const int b = c & 1;
      if (!wait(w, kPFull + b, c >> 1)) break;
      tc_fence_after();
      const uint32_t P = tlane + kColP + 128 * b;
#pragma unroll 1
      for (int jb = 0; jb < 4; ++jb) {
        uint32_t pk[16];
        if (rev ? jb < wq : jb > wq) {
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[x] = 0;
        } else {
          uint32_t v[32];
          tmem_ld32(P + 32 * jb, v);
          tmem_wait_ld();
          const int e = rows_of(c) - 32 * jb;  // columns past the end are zeros
          if (jb == wq) {
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              float f[2];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int d = rev ? 2 * x + u - lane : lane - (2 * x + u);
                f[u] = d >= 0 && 2 * x + u < e ? __uint_as_float(v[2 * x + u]) * lam[d >= 0 ? d : 0]
                                                 : 0.f;
              }
              pk[x] = pack_bf16(f[0], f[1]);
            }
          } else {
            // lam^|i-j| as a power up to the row block's edge times one from
            // there (both exponents >= 0)
            const float r = rev ? lam[32 - lane] : lam[lane];
            const float *col = rev ? lam + 32 * (jb - wq - 1) : mal + 128 - 32 * (wq - jb);
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              const float4 f = *reinterpret_cast<const float4 *>(col + 2 * x);
              const float y0 = __uint_as_float(v[2 * x]) * (r * f.x),
                          y1 = __uint_as_float(v[2 * x + 1]) * (r * f.y),
                          y2 = __uint_as_float(v[2 * x + 2]) * (r * f.z),
                          y3 = __uint_as_float(v[2 * x + 3]) * (r * f.w);
              pk[x] = pack_bf16(2 * x < e ? y0 : 0.f, 2 * x + 1 < e ? y1 : 0.f);
              pk[x + 1] = pack_bf16(2 * x + 2 < e ? y2 : 0.f, 2 * x + 3 < e ? y3 : 0.f);
            }
          }
        }
        tmem_st16(P + 16 * jb, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(w.at(kPReady + b));
    }
  } else if (warp < 8) {
    // ---- o : lane i holds row i ----
    const int i = 32 * wq + lane;
    const bool lead = warp == 4 && lane == 0;
    const CUtensorMap *mo = &args.map[sc][3];
    int stores = 0;  // whole tiles so far
    for (int c = 0; c < nc; ++c) {
      if (!wait(w, kOFull, c)) break;
      tc_fence_after();
      const int e = rows_of(c);
      const int64_t tok = start + (int64_t)tile_of(c) * kC;
      const uint32_t stage = sb + (c % L::STAGES) * L::STAGE;
      const uint32_t so = DK == 64 ? sb + L::O : stage + L::A;
      const float f = i < e ? lam[rev ? e - 1 - i : i + 1] : 0.f;
      uint32_t out[32];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t x[16], y[16];
        tmem_ld16(tlane + kColO1 + 16 * q, x);
        tmem_ld16(tlane + kColO2 + 16 * q, y);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 8; ++u)
          out[8 * q + u] = pack_bf16(
              fmaf(f, __uint_as_float(x[2 * u]), __uint_as_float(y[2 * u])),
              fmaf(f, __uint_as_float(x[2 * u + 1]), __uint_as_float(y[2 * u + 1])));
      }
      tc_fence_before();
      mbar_arrive(w.at(kOFree));
      if (e == kC) {
        if (DK == 64) {  // the last store has read the buffer
          if (lead) {
            bulk_wait_read<0>();
            mbar_arrive(w.at(kOBuf));
          }
          if (!wait(w, kOBuf, stores)) break;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          S4(swz<kTile>(so, i, 8 * q)) =
              make_uint4(out[4 * q], out[4 * q + 1], out[4 * q + 2], out[4 * q + 3]);
        fence_proxy_async_smem();
        mbar_arrive(w.at(kOWritten));
        if (lead) {
          if (!wait(w, kOWritten, stores)) break;
          tma_store_3d(mo, col0, h, (int)tok, so);
          bulk_commit();
        }
        ++stores;
      } else if (i < e) {
        uint4 *row = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(scan.o) +
                                               ((tok + i) * H + h) * dc + col0);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          row[q] = make_uint4(out[4 * q], out[4 * q + 1], out[4 * q + 2], out[4 * q + 3]);
      }
      if (DK == 128 && lead) {
        bulk_wait_read<0>();
        mbar_arrive(w.at(kEmpty + c % L::STAGES));
      }
    }
    if (lead) bulk_wait_all();
  } else if (warp < 12) {
    // ---- V^ : thread j holds row j ----
    const int j = tid - 256;
    for (int c = 0; c < nc; ++c) {
      const int s = c % L::STAGES, e = rows_of(c);
      const uint32_t stage = sb + s * L::STAGE;
      if (!wait(w, kFull + s, c / L::STAGES)) break;
      if (e < kC) {
        if (j >= e) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            S4(swz<kTile>(stage + L::V, j, 8 * q)) = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < L::SUB; ++u)
              S4(swz<kTile>(stage + L::B + u * kTile, j, 8 * q)) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(w.at(kClean));  // (one ragged tile per sequence)
      }
      if (c > 0 && !wait(w, kXFull, c - 1)) break;  // V^ has been read
      const float wj = j < e ? lam[rev ? j + 1 : e - 1 - j] : 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint4 x = S4(swz<kTile>(stage + L::V, j, 8 * q));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
        uint32_t t[3][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float lo = bf16_lo(xs[u]) * wj, hi = bf16_hi(xs[u]) * wj;
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            t[k][u] = pack_bf16(lo, hi);
            lo -= bf16_lo(t[k][u]);
            hi -= bf16_hi(t[k][u]);
          }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
          S4(swz<kTile>(sb + L::VH + k * kTile, j, 8 * q)) =
              make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(w.at(kVhReady));
    }
  } else if (warp < 16) {
    // ---- S : DK 128: lane i holds row i, 64 columns; DK 64: X holds its rows
    // twice, lanes 0-63 take columns 0-31 of them and lanes 64-127 the others ----
    constexpr int N = DK == 64 ? 32 : 64;
    const int i = (32 * wq + lane) & (DK - 1), c0 = DK == 64 ? 32 * (wq >> 1) : 0;
    float s[N];
#pragma unroll
    for (int x = 0; x < N; ++x) s[x] = 0.f;
    if (scan.s_in && scan.s_in_t) {
#pragma unroll
      for (int x = 0; x < N; ++x) s[x] = state_in(scan, unit, i, col0 + c0 + x);
    } else if (scan.s_in) {
      const float4 *row =
          reinterpret_cast<const float4 *>(scan.s_in + (unit * DK + i) * dc + col0 + c0);
#pragma unroll
      for (int x = 0; x < N / 4; ++x) {
        const float4 y = row[x];
        s[4 * x] = y.x;
        s[4 * x + 1] = y.y;
        s[4 * x + 2] = y.z;
        s[4 * x + 3] = y.w;
      }
    }
    auto put = [&]() {
#pragma unroll
      for (int q = 0; q < N / 8; ++q)
        S4(swz<kTile>(sb + L::S, i, c0 + 8 * q)) = make_uint4(
            pack_bf16(s[8 * q], s[8 * q + 1]), pack_bf16(s[8 * q + 2], s[8 * q + 3]),
            pack_bf16(s[8 * q + 4], s[8 * q + 5]), pack_bf16(s[8 * q + 6], s[8 * q + 7]));
      fence_proxy_async_smem();
      mbar_arrive(w.at(kSReady));
    };
    put();
    int done = 0;
    for (int c = 0; c < nc; ++c) {
      if (!wait(w, kXFull, c)) break;
      tc_fence_after();
      const float le = lam[rows_of(c)];
#pragma unroll
      for (int q = 0; q < N / 16; ++q) {
        uint32_t x[16];
        tmem_ld16(tlane + kColX + c0 + 16 * q, x);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 16; ++u)
          s[16 * q + u] = fmaf(le, s[16 * q + u], __uint_as_float(x[u]));
      }
      tc_fence_before();
      mbar_arrive(w.at(kXRead));
      ++done;
      if (c + 1 < nc) {
        if (!wait(w, kOFull, c)) break;  // O1 has read the last state
        put();
      }
    }
    if (scan.s_out && done == nc) {
      float4 *row = reinterpret_cast<float4 *>(scan.s_out + (unit * DK + i) * dc + col0 + c0);
#pragma unroll
      for (int x = 0; x < N / 4; ++x)
        row[x] = make_float4(s[4 * x], s[4 * x + 1], s[4 * x + 2], s[4 * x + 3]);
    }
  } else if (warp == 16) {
    // ---- TMA ----
    if (lane == 0) {
      int issued = 0;
      for (int c = 0; c < nc; ++c) {
        const int s = c % L::STAGES;
        if (c >= L::STAGES && !wait(w, kEmpty + s, c / L::STAGES - 1)) break;
        if (*abort_flag) break;
        const int tok = (int)(start + (int64_t)tile_of(c) * kC);
        const uint32_t stage = sb + s * L::STAGE, full = w.at(kFull + s);
        mbar_arrive_expect_tx(full, L::STAGE);
#pragma unroll
        for (int u = 0; u < L::SUB; ++u) {
          tma_load_3d(stage + L::A + u * kTile, &args.map[sc][0], 64 * u, h, tok, full);
          tma_load_3d(stage + L::B + u * kTile, &args.map[sc][1], 64 * u, h, tok, full);
        }
        tma_load_3d(stage + L::V, &args.map[sc][2], col0, h, tok, full);
        ++issued;
      }
      // loads still in flight land before the CTA leaves
      for (int c = issued > L::STAGES ? issued - L::STAGES : 0; c < issued; ++c)
        mbar_wait_bounded(w.at(kFull + c % L::STAGES), (c / L::STAGES) & 1, kWaitTimeoutNs);
    }
  } else if (lane == 0) {
    // ---- MMA issue ----
    auto issue_p = [&](int c) -> bool {
      if (!wait(w, kFull + c % L::STAGES, c / L::STAGES)) return false;
      if (rows_of(c) < kC && !wait(w, kClean, 0)) return false;
      tc_fence_after();
      const uint32_t stage = sb + (c % L::STAGES) * L::STAGE;
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kTile + (kk & 3) * 32;
        umma_bf16(tmem + kColP + 128 * (c & 1), umma_desc_sw128(stage + L::A + off),
                  umma_desc_sw128(stage + L::B + off), umma_idesc_bf16(128, 128), kk > 0);
      }
      umma_commit(w.at(kPFull + (c & 1)));
      return true;
    };
    bool ok = issue_p(0);
    for (int c = 0; ok && c < nc; ++c) {
      const uint32_t stage = sb + (c % L::STAGES) * L::STAGE;
      ok = wait(w, kVhReady, c) && (c == 0 || wait(w, kXRead, c - 1));
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk)
          umma_bf16(tmem + kColX, umma_desc_sw128_mn(stage + L::B + kk * 2048, DK == 64 ? 0 : kTile),
                    umma_desc_sw128_mn(sb + L::VH + k * kTile + kk * 2048, 8192),
                    umma_idesc_bf16(128, 64, 1, 1), k + kk > 0);
      umma_commit(w.at(kXFull));
      // the next chunk's P, now if its tiles are there, else after this chunk
      // (P' of the chunk before last has been read: its O2 is done)
      ok = c == 0 || wait(w, kOFull, c - 1);
      if (!ok) break;
      const bool early = c + 1 < nc && mbar_test(w.at(kFull + (c + 1) % L::STAGES),
                                                 ((c + 1) / L::STAGES) & 1);
      if (early && !(ok = issue_p(c + 1))) break;
      ok = wait(w, kSReady, c) && (c == 0 || wait(w, kOFree, c - 1));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk)
        umma_bf16(tmem + kColO1,
                  umma_desc_sw128(stage + L::A + (kk >> 2) * kTile + (kk & 3) * 32),
                  umma_desc_sw128_mn(sb + L::S + kk * 2048, 8192), umma_idesc_bf16(128, 64, 0, 1),
                  kk > 0);
      if (!(ok = wait(w, kPReady + (c & 1), c >> 1))) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kC / 16; ++kk)
        umma_bf16_ta(tmem + kColO2, tmem + kColP + 128 * (c & 1) + 8 * kk,
                     umma_desc_sw128_mn(stage + L::V + kk * 2048, 8192),
                     umma_idesc_bf16(128, 64, 0, 1), kk > 0);
      umma_commit(w.at(kOFull));
      if (DK == 64) umma_commit(w.at(kEmpty + c % L::STAGES));
      if (c + 1 < nc && !early) ok = issue_p(c + 1);
    }
    // products still in flight end before the CTA leaves
    umma_commit(w.at(kLast));
    mbar_wait_bounded(w.at(kLast), 0, kWaitTimeoutNs);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
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
  const cudaError_t err =
      cudaFuncSetAttribute(gdn_lin_tc_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Lay<DK>::ALLOC);
  if (err != cudaSuccess) return err;
  const dim3 grid(args.tiles * args.p.num_scans, p.num_heads, p.num_seqs);
  gdn_lin_tc_kernel<DK><<<grid, kThreads, Lay<DK>::ALLOC, stream>>>(args);
  return cudaGetLastError();
}

}  // namespace

bool tc_scan(const Scan &s) { return (s.da == 64 || s.da == 128) && s.dc % 64 == 0; }

cudaError_t launch_tc(const Params &p, cudaStream_t stream) {
  const cudaError_t err = launch_dk<64>(p, stream);
  return err == cudaSuccess ? launch_dk<128>(p, stream) : err;
}

}  // namespace lin
}  // namespace gdn
