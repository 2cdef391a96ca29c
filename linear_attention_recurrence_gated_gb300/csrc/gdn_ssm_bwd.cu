// Selective state space scan, backward pass (gdn_ssm.cuh has the recurrence).  With
// ds = dy silu(gate), G_t the gradient of h_t and g what a token passes to the one before,
//
//   G_t = g_{t+1} + c_t ds_t,  dc_t = sum_ch ds h_t,  db_t = sum_ch delta x G_t,
//   q = sum_s b G_t,  dx = delta q + D_skip ds,  g_t = exp(delta A) G_t,
//   w = g_t h_{t-1},  ddelta = x q + sum_s A w,  dA += delta w,
//   ddt = ddelta sigmoid(dt + dt_bias),  dgate = dy s silu'(gate),  dA_log = A dA
//
// The states of a token are needed in the reverse order of their making.  One launch
// runs the scan forward and keeps every kL-th state; the next takes the tiles of kL
// tokens from the last to the first, makes a tile's states again from the kept one and goes
// through them backward: they wait in tensor memory, 16 columns a token, which leaves
// shared memory and registers for three CTAs an SM.  12 multiply-adds and two
// exponentials an element there, 3 and one in the first (7 where sequences are cut along
// time: it leaves each segment's gradient of its start from zero too, by running products
// of the decays).  Sums over a CTA's channels (db, dc) and over tokens (dA_log, dD_skip,
// ddt_bias) are left in the workspace and added up in a fixed order by the last launch:
// results are bitwise reproducible.
//
// [4, 4096, 1280], S = 16, bf16 with a gate: 557 us; the launches 147, 405 and 10.  367
// instructions a token and 32 channels in the second: 136 of them the products and
// exponentials, some 80 the sums over lanes, the rest inputs, softplus, the gate and their
// gradients.  The multiply-adds' pipe is busy for 40 %, issue 51 %.  (States in shared
// memory, two CTAs an SM: 763 us in all; in tensor memory 603; inputs and kept states by
// asynchronous copies 554; lifts by tiles, for their accuracy, 561; the first two loops over
// a tile unrolled whole 554, the third too 563; the rows of a short tile before its tokens 557.)
#include "gdn_ptx.cuh"
#include "gdn_ssm.cuh"

namespace gdn {
gdn_status pass_states(const float *from, float *to, size_t bytes, cudaStream_t s);

namespace ssm {
namespace {

constexpr int kL = 8;   // tokens from one kept state to the next, and of a tile

struct BwdParams : Params {
  const void *dy;
  const float *dhT;
  void *dx, *ddt, *db, *dc, *dgate;
  float *dA_log, *dD_skip, *ddt_bias, *dh0;
  float *seg_y;      // [slot][D][S] gradient that a segment passes to the one before
  float *ckpt;       // [tokens / kL][D][S] kept states (of later segments: from zero)
  float *ckpt_d;     // [tokens / kL][D] sum of delta since the segment's start
  float *part_bc;    // [block][token][G][2][S]
  float *part_w;     // [gridDim.y][D S + 2 D] sums for dA, dD_skip, ddt_bias
  float *own_w;      // [CTA][2][16][thread] a thread's sums for them so far
  int32_t G, parts;
  __host__ __device__ int64_t rows() const {
    return seq.cu ? seq.seq_len : seq.seq_len * seq.num_seqs;
  }
};

// The place of the state before token t (a multiple of kL, > 0) of a sequence that begins
// at token `start`: floor(start / kL) + t / kL - 1, never that of another sequence.
__device__ __forceinline__ int64_t kept(int64_t start, int64_t t) { return start / kL + t / kL - 1; }

// The inputs of tiles of TT tokens, eight channels (or states of b, c) a thread at a time.
template <typename T, int S, int TT, bool GRAD>
struct Inputs {
  static constexpr int CB = Geo<S>::CB, VB = CB / 8, RT = kThreads / VB;
  static constexpr int NV = (TT + RT - 1) / RT;
  static constexpr int NBC = 2 * TT * S / 8, NB = (NBC + kThreads - 1) / kThreads;
  Raw8<T> x[NV], dt[NV], dy[GRAD ? NV : 1], gate[GRAD ? NV : 1], bc[NB];
  __device__ __forceinline__ void fetch(const BwdParams &p, int64_t first, int cnt, int group,
                                        int vch, bool von) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int row = tid / VB + i * RT;
      x[i].zero();
      dt[i].zero();
      if (GRAD) {
        dy[i].zero();
        gate[i].zero();
      }
      if (!von || row >= cnt) continue;
      const int64_t at = first + row;
      x[i].load(static_cast<const T *>(p.x) + at * p.sx + vch);
      dt[i].load(static_cast<const T *>(p.dt) + at * p.sdt + vch);
      if (GRAD) {
        dy[i].load(static_cast<const T *>(p.dy) + at * p.D + vch);
        if (p.gate) gate[i].load(static_cast<const T *>(p.gate) + at * p.sg + vch);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int idx = tid + i * kThreads, row = idx % (NBC / 2) / (S / 8), v = idx % (S / 8);
      bc[i].zero();
      if (idx >= NBC || row >= cnt) continue;
      if (idx < NBC / 2)
        bc[i].load(static_cast<const T *>(p.b) + (first + row) * p.sb + group * S + 8 * v);
      else if (GRAD)
        bc[i].load(static_cast<const T *>(p.c) + (first + row) * p.sc + group * S + 8 * v);
    }
  }
  // delta, delta x and ds of the tile, to shared memory
  __device__ __forceinline__ void form(const BwdParams &p, int cnt, int vch, bool von, float *sd,
                                       float *su, float *ss) const {
    const int tid = threadIdx.x, vec = tid % VB;
    uint64_t bias[4];
    load8(p.dt_bias, vch, von, bias);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int row = tid / VB + i * RT;
      if (row >= TT) continue;
      uint64_t v[4], d[4];
      steps_of(dt[i], bias, p.softplus, d);
      if (row >= cnt)   // tokens that do not exist leave the states as they are
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = 0ull;
      pairs_of(x[i], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = mul2(d[j], v[j]);
      put8(sd + row * CB + 8 * vec, d);
      put8(su + row * CB + 8 * vec, v);
      if (GRAD) {
        pairs_of(dy[i], d);
        if (p.gate) {
          pairs_of(gate[i], v);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = mul2(d[j], mul2(v[j], sigmoid2(v[j])));
        }
        put8(ss + row * CB + 8 * vec, d);
      }
    }
  }
};

template <int S> constexpr int kKeepTile = S < 32 ? S : 32;   // tokens of a tile of the first launch

// First launch: the kept states, and of segments their end state, sum of delta and
// gradient from zero.
template <typename T, int S, bool CUT>
__global__ void __launch_bounds__(kThreads, !CUT ? 4 : sizeof(T) == 2 ? 3 : 2)
gdn_ssm_keep_kernel(const BwdParams p) {
  constexpr int TT = kKeepTile<S>, CB = Geo<S>::CB;
  constexpr int LS = Run<S>::LS, CPT = Run<S>::CPT, NP = Run<S>::NP;
  static_assert(TT % kL == 0 && kChunkTokens % TT == 0, "tiles of whole runs of kL tokens");
  using In = Inputs<T, S, TT, CUT>;
  extern __shared__ __align__(16) float smem[];
  float *sd = smem, *su = sd + TT * CB, *sbc = su + TT * CB, *ss = sbc + (CUT ? 2 : 1) * TT * S;
  const int tid = threadIdx.x;
  const int group = blockIdx.x / p.blocks, cb = blockIdx.x % p.blocks, slot = blockIdx.y;
  const int first_ch = group * p.Dg + cb * CB, end_ch = (group + 1) * p.Dg;
  const int sl = tid % LS, cl = tid / LS * CPT, swap = S == 64 ? sl >> 1 : 0;
  const bool on = first_ch + cl < end_ch;
  const int64_t own = (int64_t)first_ch * S + 16 * tid;   // its elements of [D][S]
  let_second();
  lin::Span s;
  if (!lin::span_of(p.seq, slot, 0, s)) return;
  const int64_t D = p.D, state = D * S, begin = s.start - s.seg * p.seq.seg_len;
  const int64_t off = s.seg * p.seq.seg_len;   // the segment's first token in its sequence
  const bool last = s.seg == s.count - 1;
  // tokens up to the last kept state, or all where what follows needs the end
  const bool whole = CUT && s.count > 1;
  const int64_t len = whole ? s.len : s.len > 0 ? (s.len - 1) / kL * kL : 0;
  if (len == 0) return;

  uint64_t A[8], h[8], P[CUT ? 8 : 1], Y[CUT ? 8 : 1];
  rates16(p.A_log + own, on, A);
  load16(s.seg == 0 && p.h0 ? p.h0 + s.n * state + own : nullptr, on, h);
  if constexpr (CUT)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      P[i] = pk(1.f, 1.f);
      Y[i] = 0ull;
    }
  const int vec = tid % In::VB, vch = first_ch + 8 * vec;
  const bool von = vch < end_ch;

  float sums[CPT] = {};
  const auto keep = [&](int64_t t) {
    const int64_t at = kept(begin, off + t);
    store16(p.ckpt + at * state + own, on, h);
    if (CUT && s.seg > 0 && on && sl == 0)
#pragma unroll
      for (int k = 0; k < CPT; ++k) p.ckpt_d[at * D + first_ch + cl + k] = sums[k];
  };
  In in;
  in.fetch(p, s.start, (int)(len < TT ? len : TT), group, vch, von);
  for (int64_t t0 = 0; t0 < len; t0 += TT) {
    const int cnt = (int)(len - t0 < TT ? len - t0 : TT);
    in.form(p, cnt, vch, von, sd, su, ss);
#pragma unroll
    for (int i = 0; i < In::NB; ++i) {
      const int idx = tid + i * kThreads;
      if (idx >= (CUT ? In::NBC : In::NBC / 2)) continue;
      uint64_t v[4];
      pairs_of(in.bc[i], v);
      if (S == 64 && (idx & 4)) {   // see pairs()
        const uint64_t w[4] = {v[2], v[3], v[0], v[1]};
        put8(sbc + 8 * idx, w);
      } else {
        put8(sbc + 8 * idx, v);
      }
    }
    __syncthreads();
    if (t0 + TT < len)
      in.fetch(p, s.start + t0 + TT, (int)(len - t0 - TT < TT ? len - t0 - TT : TT), group, vch, von);
    for (int r = 0; r < cnt; r += kL) {
      if (t0 + r > 0) {
        keep(t0 + r);
        if constexpr (CUT)   // the product so far, from the sum: kL factors' roundings at most
#pragma unroll
          for (int k = 0; k < CPT; ++k)
#pragma unroll
            for (int i = 0; i < NP; ++i)
              P[k * NP + i] = ex2_pair(mul2(pk(sums[k], sums[k]), A[k * NP + i]));
      }
      float part[CPT] = {};
      uint64_t lift[2];
      lifts16<CPT>(A, sd + r * CB + cl, lift);
#pragma unroll
      for (int t = r; t < r + kL; ++t) {   // (tokens past the last: zeros)
        uint64_t d[CPT], u[CPT], y[CPT], b2[NP], c2[NP];
        twice<CPT>(sd + t * CB + cl, d);
        twice<CPT>(su + t * CB + cl, u);
        pairs<NP>(sbc + t * S + 16 * sl, swap, b2);
        if constexpr (CUT) {
          twice<CPT>(ss + t * CB + cl, y);
          pairs<NP>(sbc + TT * S + t * S + 16 * sl, swap, c2);
        }
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const int e = k * NP + i;
            const uint64_t a = decay(d[k], A[e], lift[e / 4]);
            h[e] = fma2(a, h[e], mul2(u[k], b2[i]));
            if constexpr (CUT) {
              P[e] = mul2(P[e], a);
              Y[e] = fma2(P[e], mul2(c2[i], y[k]), Y[e]);
            }
          }
          float lo, hi;
          unpk(d[k], lo, hi);
          part[k] += lo;
        }
      }
#pragma unroll
      for (int k = 0; k < CPT; ++k) sums[k] += part[k];
    }
    __syncthreads();
  }
  if (!whole) {   // the last kept state comes behind the last token that was run
    keep(len);
    return;
  }
  if (!last) store16(p.seg_x + slot * state + own, on, h);
  if constexpr (CUT) store16(p.seg_y + slot * state + own, on, Y);
  if (on && sl == 0)
#pragma unroll
    for (int k = 0; k < CPT; ++k) p.seg_d[(int64_t)slot * D + first_ch + cl + k] = sums[k];
}
template <int S, bool CUT>
constexpr size_t keep_smem() {
  constexpr int TT = kKeepTile<S>;
  return 4u * (TT * Geo<S>::CB * (CUT ? 3 : 2) + (CUT ? 2 : 1) * TT * S);
}

// v[8]: four values of db and four of dc of a lane's states, summed over the warp's CL
// groups of channels.  A lane keeps 8 / CL of them (one for CL of 8 and 16), from `first`.
template <int CL, int LS>
__device__ __forceinline__ int sum_groups(float (&v)[8], int grp) {
  constexpr uint32_t kAll = 0xffffffffu;
  int first = 0;
#pragma unroll
  for (int n = 4, bit = 1; bit < CL; n /= 2, bit *= 2) {
    const bool up = grp & bit;
    if (n >= 1) {
#pragma unroll
      for (int i = 0; i < (n ? n : 1); ++i) {
        const float give = up ? v[i] : v[i + n], mine = up ? v[i + n] : v[i];
        v[i] = mine + __shfl_xor_sync(kAll, give, bit * LS);
      }
      first += up ? n : 0;
    } else {
      v[0] += __shfl_xor_sync(kAll, v[0], bit * LS);
    }
  }
  return first;
}

// Shared memory of the second launch, in floats.
template <typename T, int S>
struct Bwd {
  static constexpr int CB = Geo<S>::CB, VB = CB / 8, RT = kThreads / VB, TILE = kL * CB, OWN = 16 * kThreads;
  static constexpr int NV = (kL + RT - 1) / RT;             // a thread's vectors of x, dt, dy, gate
  static constexpr int NBC = 2 * kL * S / 8, NB = (NBC + kThreads - 1) / kThreads;   // ... of b and c
  static constexpr int VEC = kThreads * 8 * sizeof(T) / 4;  // a vector of every thread
  static constexpr int D = 0, U = D + TILE, E = U + TILE;   // delta; delta x, later q; ds, later sum A w
  static constexpr int Y = E + TILE, BC = Y + TILE;         // c . h; b and c, each value twice
  static constexpr int RED = BC + 4 * kL * S;               // the warps' sums for db and dc
  static constexpr int START = RED + 4 * kL * 2 * S;        // a thread's states at the segment's start
  static constexpr int SUM = START + OWN;                   // ... sums for dD_skip and ddt_bias
  static constexpr int KEPT = SUM + OWN;                    // ... kept states of the next tile
  static constexpr int RAW = KEPT + OWN;                    // inputs of this tile and the next
  static constexpr int TILE_RAW = (4 * NV + NB) * VEC;
  static constexpr size_t kFloats = RAW + 2 * TILE_RAW + 4; // (and the place in tensor memory)
  static constexpr int kFit = 228 * 1024 / (4 * kFloats + 1024);   // (1 KB a CTA is the system's)
  static constexpr int kCtas = kFit < 3 ? kFit : 3;                // an SM
};
constexpr uint32_t kColumns = 16 * kL;   // of tensor memory: a thread's 16 values for each token

// 16 bytes from global to shared memory, zeros where there are none.
__device__ __forceinline__ void copy16(void *to, const void *from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(there ? 16 : 0)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void copy_vec(Raw8<T> *to, const T *from, bool there) {
  copy16(to, from, there);
  if constexpr (sizeof(T) == 4)
    copy16(reinterpret_cast<float *>(to) + 4, reinterpret_cast<const float *>(from) + 4, there);
}

// Second launch: tiles from the last token to the first.
template <typename T, int S, bool GATE>
__global__ void __launch_bounds__(kThreads, Bwd<T, S>::kCtas)
gdn_ssm_grad_kernel(const BwdParams p) {
  using B = Bwd<T, S>;
  constexpr int CB = B::CB, LS = Geo<S>::LS, CL = Geo<S>::CL;
  extern __shared__ __align__(16) float smem[];
  float *sd = smem + B::D, *su = smem + B::U, *ss = smem + B::E, *sy = smem + B::Y, *sbc = smem + B::BC;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = blockIdx.x / p.blocks, cb = blockIdx.x % p.blocks;
  const int first_ch = group * p.Dg + cb * CB, end_ch = (group + 1) * p.Dg;
  const int sl = lane % LS, grp = lane / LS, cl = warp * CL + grp;
  const Own own{first_ch + 4 * cl, 4 * sl, first_ch + 4 * cl < end_ch};
  const int64_t D = p.D, state = D * S;

  uint32_t *place = reinterpret_cast<uint32_t *>(smem + B::kFloats - 4);
  if (warp == 0) ptx::tmem_alloc((uint32_t)__cvta_generic_to_shared(place), kColumns);
  __syncthreads();
  const uint32_t columns = *place, mine = columns + ((uint32_t)(warp * 32) << 16);

  // a thread's 16 values: in tensor memory ...
  const auto store_tm = [&](int t, const uint64_t (&a)[2][4]) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r[2 * i] = (uint32_t)a[i >> 2][i & 3];
      r[2 * i + 1] = (uint32_t)(a[i >> 2][i & 3] >> 32);
    }
    ptx::tmem_st16(mine + 16 * t, r);
  };
  const auto load_tm = [&](int t, uint32_t (&r)[16]) { ptx::tmem_ld16(mine + 16 * t, r); };
  // ... and in shared memory, four float4, a row of threads each
  const auto put16 = [&](float *at, const uint64_t (&a)[2][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<ulonglong2 *>(at)[i * kThreads + tid] =
          make_ulonglong2(a[i >> 1][2 * (i & 1)], a[i >> 1][2 * (i & 1) + 1]);
  };
  const auto get16 = [&](const float *at, uint64_t (&a)[2][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ulonglong2 v = reinterpret_cast<const ulonglong2 *>(at)[i * kThreads + tid];
      a[i >> 1][2 * (i & 1)] = v.x;
      a[i >> 1][2 * (i & 1) + 1] = v.y;
    }
  };

  uint64_t A[2][4], dA[2][4], g[2][4], h[2][4];
  load_rates<S>(p.A_log, own, A);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) dA[k][j] = 0ull;
  put16(smem + B::SUM, dA);
  const int vec = tid % B::VB, vch = first_ch + 8 * vec;
  const bool von = vch < end_ch;
  // The inputs of a tile, and the states kept before it, on their way to shared memory;
  // every thread waits for its own.  A tile of fewer than kL tokens begins at row `lead`
  // (rows before it do not exist): behind its last token there is no step of zero that a
  // last state that is not finite would turn into a part of dA.
  const auto raw = [&](int64_t tile, int i) {
    return reinterpret_cast<Raw8<T> *>(smem + B::RAW + (tile & 1) * B::TILE_RAW + i * B::VEC) + tid;
  };
  const auto fetch = [&](int64_t tile, int64_t first, int lead, const float *kept_at) {
#pragma unroll
    for (int i = 0; i < B::NV; ++i) {
      const int row = tid / B::VB + i * B::RT;
      const bool there = von && row >= lead && (B::NV * B::RT == kL || row < kL);
      const int64_t at = there ? first + row - lead : 0;
      const int c = there ? vch : 0;
      copy_vec(raw(tile, 4 * i), static_cast<const T *>(p.x) + at * p.sx + c, there);
      copy_vec(raw(tile, 4 * i + 1), static_cast<const T *>(p.dt) + at * p.sdt + c, there);
      copy_vec(raw(tile, 4 * i + 2), static_cast<const T *>(p.dy) + at * D + c, there);
      if (GATE) copy_vec(raw(tile, 4 * i + 3), static_cast<const T *>(p.gate) + at * p.sg + c, there);
    }
#pragma unroll
    for (int i = 0; i < B::NB; ++i) {
      const int idx = tid + i * kThreads, row = idx % (B::NBC / 2) / (S / 8), v = idx % (S / 8);
      const bool there = idx < B::NBC && row >= lead;
      const int64_t at = there ? first + row - lead : 0;
      const T *from = idx < B::NBC / 2 ? static_cast<const T *>(p.b) + at * p.sb
                                       : static_cast<const T *>(p.c) + at * p.sc;
      copy_vec(raw(tile, 4 * B::NV + i), from + group * S + 8 * v, there);
    }
    if (kept_at)
#pragma unroll
      for (int i = 0; i < 4; ++i)   // channel i of the thread's four
        copy16(smem + B::KEPT + 4 * (i * kThreads + tid),
               own.on ? kept_at + (int64_t)(own.ch + i) * S + own.st : p.A_log, own.on);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // A thread's sums, for dA and for dD_skip and ddt_bias, run over 16 tiles at most; then
  // they join those before, in the workspace.
  int tiles_summed = 0;
  bool joined = false;
  float *before_sums = p.own_w + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * B::OWN;
  const auto joint = [&](const float *at, uint64_t (&a)[2][4]) {
    if (!joined) return;
    uint64_t b[2][4];
    get16(at, b);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) a[k][j] = add2(a[k][j], b[k][j]);
  };
  const auto flush = [&] {
    joint(before_sums, dA);
    put16(before_sums, dA);
    uint64_t some[2][4];
    get16(smem + B::SUM, some);
    joint(before_sums + B::OWN, some);
    put16(before_sums + B::OWN, some);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) dA[k][j] = 0ull;
    put16(smem + B::SUM, dA);
    joined = true;
    tiles_summed = 0;
  };
  wait_first();
  let_second();   // the sums' CTAs, as these leave room

  for (int slot = blockIdx.y; slot < p.seq.slots; slot += gridDim.y) {
    lin::Span s;
    if (!lin::span_of(p.seq, slot, 0, s)) continue;
    const int64_t begin = s.start - s.seg * p.seq.seg_len, off = s.seg * p.seq.seg_len;
    const int64_t tiles = (s.len + kL - 1) / kL;
    const auto kept_at = [&](int64_t tile) {
      return tile ? p.ckpt + kept(begin, off + tile * kL) * state : nullptr;
    };
    if (tiles > 0)
      fetch(tiles - 1, s.start + (tiles - 1) * kL, (int)(tiles * kL - s.len), kept_at(tiles - 1));
    // the gradient that comes from behind the segment, and the state at its start
    load_own<S>(p.dhT ? p.dhT + s.n * state : nullptr, own, g);
    for (int i = s.count - 1; i > s.seg; --i)
      join<S>(g, A, p.seg_y, p.seg_d, slot - s.seg + i, p.D, own);
    if (p.dh0 && s.seg == 0 && s.count > 1) {   // (not through the segment's hundreds of roundings)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k][j] = g[k][j];
      join<S>(h, A, p.seg_y, p.seg_d, slot, p.D, own);
      store_own<S>(p.dh0 + s.n * state, own, h);
    }
    if (s.seg == 0) {
      load_own<S>(p.h0 ? p.h0 + s.n * state : nullptr, own, h);
    } else {
      load_own<S>(p.seg_x + (int64_t)(slot - s.seg) * state, own, h);
      for (int i = 1; i < s.seg; ++i)
        join<S>(h, A, p.seg_x, p.seg_d, slot - s.seg + i, p.D, own);
    }
    put16(smem + B::START, h);

    for (int64_t tile = tiles - 1; tile >= 0; --tile) {
      const int64_t t0 = tile * kL;
      const int cnt = (int)(s.len - t0 < kL ? s.len - t0 : kL), lead = kL - cnt;
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      // delta, delta x and ds of the tile; tokens that do not exist are zeros, which leave
      // states and gradients as they are
      uint64_t bias[4], skip[4];
      load8(p.dt_bias, vch, von, bias);
#pragma unroll
      for (int i = 0; i < B::NV; ++i) {
        const int row = tid / B::VB + i * B::RT;
        if (row >= kL) continue;
        uint64_t v[4], d[4];
        steps_of(*raw(tile, 4 * i + 1), bias, p.softplus, d);
        if (row < lead) d[0] = d[1] = d[2] = d[3] = 0ull;
        pairs_of(*raw(tile, 4 * i), v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul2(d[j], v[j]);
        put8(sd + row * CB + 8 * vec, d);
        put8(su + row * CB + 8 * vec, v);
        pairs_of(*raw(tile, 4 * i + 2), d);
        if constexpr (GATE) {
          pairs_of(*raw(tile, 4 * i + 3), v);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = mul2(d[j], mul2(v[j], sigmoid2(v[j])));
        }
        put8(ss + row * CB + 8 * vec, d);
      }
#pragma unroll
      for (int i = 0; i < B::NB; ++i) {
        const int idx = tid + i * kThreads;
        if (idx >= B::NBC) continue;
        float v[8];
        raw(tile, 4 * B::NV + i)->get(v);
        store_twice<S>(sbc, idx, v);
      }
      // the state before the tile
      if (tile == 0) {
        get16(smem + B::START, h);
      } else {
        float v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 f = *reinterpret_cast<const float4 *>(smem + B::KEPT + 4 * (i * kThreads + tid));
          v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
        }
        if (s.seg == 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) h[k][j] = pk(v[2 * k][j], v[2 * k + 1][j]);
        } else {   // kept from zero: and what the segment's start has become
          get16(smem + B::START, h);
          const float4 sum = own.on ? *reinterpret_cast<const float4 *>(
                                          p.ckpt_d + kept(begin, off + t0) * D + own.ch)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
          const uint64_t past[2] = {pk(sum.x, sum.y), pk(sum.z, sum.w)};
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              h[k][j] = fma2(ex2_pair(mul2(past[k], A[k][j])), h[k][j], pk(v[2 * k][j], v[2 * k + 1][j]));
        }
      }
      __syncthreads();
      if (tile > 0) fetch(tile - 1, s.start + t0 - kL, 0, kept_at(tile - 1));
      uint64_t lift[2];
      lifts4(A, sd + lead * CB + 4 * cl, lift);
      // the tile's states
#pragma unroll
      for (int t = 0; t < kL; ++t) {
        store_tm(t, h);
        const Pairs d = lds2(sd + t * CB + 4 * cl), u = lds2(su + t * CB + 4 * cl);
        const uint64_t dd[2] = {d.a, d.b}, uu[2] = {u.a, u.b};
        uint64_t bb[4], cc[4], y[2];
        load_twice<S>(sbc, t, 0, sl, bb);
        if constexpr (GATE) load_twice<S>(sbc, t, 1, sl, cc);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[k][j] = fma2(decay(dd[k], A[k][j], lift[k]), h[k][j], mul2(uu[k], bb[j]));
            if constexpr (GATE) y[k] = j ? fma2(cc[j], h[k][j], y[k]) : mul2(cc[j], h[k][j]);
          }
        if constexpr (GATE) {
          float v[4];
          unpk(y[0], v[0], v[1]);
          unpk(y[1], v[2], v[3]);
          sum_channels<LS>(v, sl);
          store_channels<LS>(sy + t * CB + 4 * cl, v, sl);
          __syncwarp();
        }
      }
      ptx::tmem_wait_st();
      // and backward through them
      uint32_t ahead[16];
      load_tm(kL - 1, ahead);
#pragma unroll 4
      for (int t = kL - 1; t >= 0; --t) {
        const Pairs d = lds2(sd + t * CB + 4 * cl), u = lds2(su + t * CB + 4 * cl),
                    e = lds2(ss + t * CB + 4 * cl);
        const uint64_t dd[2] = {d.a, d.b}, uu[2] = {u.a, u.b}, ee[2] = {e.a, e.b};
        uint64_t bb[4], cc[4], before[2][4], db[4], dc[4], q[2], aw[2];
        load_twice<S>(sbc, t, 0, sl, bb);
        load_twice<S>(sbc, t, 1, sl, cc);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          before[i >> 2][i & 3] = ((uint64_t)ahead[2 * i + 1] << 32) | ahead[2 * i];
        __syncwarp();   // delta x and ds of this token are read: q and sum A w take their place
        if (t > 0) load_tm(t - 1, ahead);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t G = fma2(cc[j], ee[k], g[k][j]);
            dc[j] = k ? fma2(ee[k], h[k][j], dc[j]) : mul2(ee[k], h[k][j]);
            db[j] = k ? fma2(uu[k], G, db[j]) : mul2(uu[k], G);
            q[k] = j ? fma2(bb[j], G, q[k]) : mul2(bb[j], G);
            g[k][j] = mul2(decay(dd[k], A[k][j], lift[k]), G);
            const uint64_t w = mul2(g[k][j], before[k][j]);
            aw[k] = j ? fma2(A[k][j], w, aw[k]) : mul2(A[k][j], w);
            dA[k][j] = fma2(dd[k], w, dA[k][j]);
            h[k][j] = before[k][j];
          }
        float v[4], r[8];
        unpk(q[0], v[0], v[1]);
        unpk(q[1], v[2], v[3]);
        sum_channels<LS>(v, sl);
        store_channels<LS>(su + t * CB + 4 * cl, v, sl);
        unpk(aw[0], v[0], v[1]);
        unpk(aw[1], v[2], v[3]);
        sum_channels<LS>(v, sl);
        store_channels<LS>(ss + t * CB + 4 * cl, v, sl);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          r[j] = total(db[j]);
          r[4 + j] = total(dc[j]);
        }
        const int first = sum_groups<CL, LS>(r, grp);
        float *red = smem + B::RED + (warp * kL + t) * 2 * S;
        constexpr int KEEP = CL >= 8 ? 1 : 8 / CL;
        if (CL <= 8 || grp < 8)
#pragma unroll
          for (int i = 0; i < KEEP; ++i) {
            const int id = first + i;   // 0-3: db of its states, 4-7: dc
            red[(id >> 2) * S + 4 * sl + (id & 3)] = r[i];
          }
        __syncwarp();
      }
      __syncthreads();
      // db and dc of this CTA's channels, four values a thread
      for (int i = 4 * tid; i < cnt * 2 * S; i += 4 * kThreads) {
        const int row = i / (2 * S), at = i % (2 * S);
        const float *red = smem + B::RED + (lead + row) * 2 * S + at;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
          const float4 v = *reinterpret_cast<const float4 *>(red + w * kL * 2 * S);
          sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
        }
        *reinterpret_cast<float4 *>(
            p.part_bc + (((int64_t)cb * p.rows() + s.start + t0 + row) * p.G + group) * 2 * S + at) = sum;
      }
      uint64_t sums[2][4];   // for dD_skip and ddt_bias
      load8(p.dt_bias, vch, von, bias);
      load8(p.d_skip, vch, von, skip);
      get16(smem + B::SUM, sums);
#pragma unroll
      for (int i = 0; i < B::NV; ++i) {
        const int row = tid / B::VB + i * B::RT;
        if (!von || row < lead || (B::NV * B::RT > kL && row >= kL)) continue;
        const int64_t out = (s.start + t0 + row - lead) * D + vch;
        const int at = row * CB + 8 * vec;
        uint64_t xv[4], yv[4], qv[4], v[4], o[4];
        Raw8<T> r;
        pairs_of(*raw(tile, 4 * i), xv);
        pairs_of(*raw(tile, 4 * i + 2), yv);
        if constexpr (GATE) {
          uint64_t gv[4];
          pairs_of(*raw(tile, 4 * i + 3), gv);
          take8(sy + at, v);
          if (p.d_skip)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = fma2(skip[j], xv[j], v[j]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // silu'(g) = sg (1 + g (1 - sg))
            const uint64_t sg = sigmoid2(gv[j]), one = pk(1.f, 1.f);
            const uint64_t slope = mul2(sg, fma2(gv[j], fma2(sg, pk(-1.f, -1.f), one), one));
            o[j] = mul2(mul2(yv[j], v[j]), slope);
            yv[j] = mul2(yv[j], mul2(gv[j], sg));
          }
          set_pairs(r, o);
          r.store(static_cast<T *>(p.dgate) + out);
        }
        take8(sd + at, v);
        take8(su + at, qv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[j] = fma2(v[j], qv[j], mul2(skip[j], yv[j]));
          sums[0][j] = fma2(yv[j], xv[j], sums[0][j]);
        }
        set_pairs(r, o);
        r.store(static_cast<T *>(p.dx) + out);
        take8(ss + at, v);
        uint64_t tv[4];
        pairs_of(*raw(tile, 4 * i + 1), tv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // (rates carry log2 e)
          o[j] = fma2(xv[j], qv[j], mul2(pk(0.6931471805599453f, 0.6931471805599453f), v[j]));
          if (p.softplus) o[j] = mul2(o[j], softplus_slope2<T>(add2(tv[j], bias[j])));
          sums[1][j] = add2(sums[1][j], o[j]);
        }
        set_pairs(r, o);
        r.store(static_cast<T *>(p.ddt) + out);
      }
      put16(smem + B::SUM, sums);
      if (++tiles_summed == 16) flush();
      __syncthreads();
    }
    if (p.dh0 && s.count == 1) store_own<S>(p.dh0 + s.n * state, own, g);
  }

  // this CTA's sums over its tokens
  joint(before_sums, dA);
  float *part = p.part_w + (int64_t)blockIdx.y * (state + 2 * D);
  store_own<S>(part, own, dA);
  uint64_t sums[2][4];
  get16(smem + B::SUM, sums);
  joint(before_sums + B::OWN, sums);
  __syncthreads();
  float *sum = smem;   // [2][rows of threads][CB]: 2048 floats
  static_assert(2 * B::RT * CB <= B::START, "room for the sums");
#pragma unroll
  for (int which = 0; which < 2; ++which)
    put8(sum + (which * B::RT + tid / B::VB) * CB + 8 * vec, sums[which]);
  __syncthreads();
  for (int i = tid; i < 2 * CB; i += kThreads) {
    const int which = i / CB, ch = i % CB;
    if (first_ch + ch >= end_ch) continue;
    float r = 0.f;
    for (int k = 0; k < B::RT; ++k) r += sum[(which * B::RT + k) * CB + ch];
    part[state + which * D + first_ch + ch] = r;
  }
  if (warp == 0) ptx::tmem_dealloc(columns, kColumns);
}

// Third launch: the sums over blocks of channels, and behind them those over the tokens of
// the second launch's CTAs.
template <typename T>
__global__ void __launch_bounds__(256)
gdn_ssm_sum_kernel(const BwdParams p, int S, int64_t bc_blocks) {
  wait_first();
  if (blockIdx.x < bc_blocks) {   // four values a thread
    const int64_t per = (int64_t)p.G * 2 * S, n = p.rows() * per;
    const int64_t i0 = (int64_t)blockIdx.x * 1024, i = i0 + 4 * threadIdx.x;
    if (p.seq.cu) {   // rows of a sequence whose offsets are bad stay as they are
      const Sequences q{p.seq.cu, p.seq.status, p.seq.seq_len, p.seq.num_seqs};
      const int64_t row = (i < n ? i : n - 1) / per;
      const int64_t first = (i0 + 4 * (threadIdx.x & ~31)) / per;
      int at = q.find(first < p.rows() ? first : p.rows() - 1);
      while (at + 1 < p.seq.num_seqs && p.seq.cu[at + 1] <= row) ++at;
      int64_t start, len;
      if (!q.bounds(at, start, len) || row < start || row >= start + len) return;
    }
    if (i >= n) return;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int b = 0; b < p.blocks; ++b) {
      const float4 v = *reinterpret_cast<const float4 *>(p.part_bc + b * n + i);
      sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
    }
    const int64_t row = i / per;
    const int r = (int)(i - row * per), grp = r / (2 * S), which = r / S % 2, st = r % S;
    Raw4<T> out;
    const uint64_t v[2] = {pk(sum.x, sum.y), pk(sum.z, sum.w)};
    out.set(v);
    out.store(static_cast<T *>(which ? p.dc : p.db) + (row * p.G + grp) * S + st);
    return;
  }
  // 32 of the weights' sums, shared by eight warps
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t state = (int64_t)p.D * S, n = state + 2 * p.D;
  const int64_t i = (blockIdx.x - bc_blocks) * 32 + lane;
  float sum = 0.f;
  if (i < n)
#pragma unroll 4
    for (int k = warp; k < p.parts; k += 8) sum += p.part_w[k * n + i];
  red[warp][lane] = sum;
  __syncthreads();
  if (warp || i >= n) return;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) sum += red[w][lane];
  if (i < state) {
    if (p.dA_log) p.dA_log[i] = -expf(p.A_log[i]) * sum;
  } else if (i < state + p.D) {
    if (p.dD_skip) p.dD_skip[i - state] = sum;
  } else if (p.ddt_bias) {
    p.ddt_bias[i - state - p.D] = sum;
  }
}

// The arrays of the workspace behind the status word, in floats.
struct Layout {
  size_t x, y, d, ckpt, ckpt_d, bc, w, own, total;
};
Layout layout(int64_t rows, int64_t D, int64_t S, int64_t groups, int64_t blocks, int64_t parts,
              const lin::Plan &pl) {
  const auto round = [](size_t n) { return (n + 3) / 4 * 4; };
  const size_t state = (size_t)(D * S), slots = pl.seg_len ? (size_t)pl.slots : 0;
  Layout l;
  l.x = 0;
  l.y = l.x + slots * state;
  l.d = l.y + slots * state;
  l.ckpt = l.d + slots * D;
  l.ckpt_d = l.ckpt + (size_t)(rows / kL) * state;
  l.bc = l.ckpt_d + (slots ? (size_t)(rows / kL) * D : 0);
  l.w = l.bc + round((size_t)blocks * rows * groups * 2 * S);
  l.own = l.w + (size_t)parts * (state + 2 * D);
  l.total = l.own + (size_t)parts * groups * blocks * 2 * 16 * kThreads;
  return l;
}
constexpr double kFirst = 0.5;
// CTAs of the second launch over the slots: at most as many as three an SM, and one more
// round of them
int64_t parts_of(int64_t slots, int64_t blocks) {
  const int64_t most = (6 * kSMs + blocks - 1) / blocks;
  return slots < most ? slots : most;
}
// CTAs an SM that the plan counts on: those of the second launch (Bwd::kCtas), but two for
// fp32 with S = 8, of which one fits.  (Planned with one, fp32, S 8: [8, 1024, 2560] 927 us,
// [1, 16384, 1280] 660, [4, 4096, 2560] 1166, [2, 2048, 1024] 158, [3, 3000, 512] 165; with
// two 592, 619, 1115, 166, 185.)
constexpr int plan_ctas(bool wide, int S) { return wide || S == 8 ? 2 : 3; }

// The workspace of a call in any form that it may take (storage types, and uncut).
size_t workspace_bytes_of(int32_t num_seqs, int32_t seq_len, bool packed, int32_t channels,
                          int32_t d_state, int32_t groups) {
  const int64_t blocks = channel_blocks(channels / groups, d_state), all = blocks * groups;
  const int64_t rows = packed ? seq_len : (int64_t)num_seqs * seq_len;
  size_t most = 0;
  for (const auto &one : {plan(num_seqs, seq_len, packed, all, 2, kFirst),
                          plan(num_seqs, seq_len, packed, all, 3, kFirst),
                          lin::Plan{0, num_seqs}}) {
    const size_t n = layout(rows, channels, d_state, groups, blocks, parts_of(one.slots, all),
                            one).total;
    most = n > most ? n : most;
  }
  return kStatusBytes + 4 * most;
}

template <typename T, int S>
cudaError_t launch_s(const BwdParams &p, int groups, cudaStream_t stream) {
  const dim3 grid(groups * p.blocks, p.seq.slots);
  cudaError_t err;
  if (p.seq.seg_len) {
    constexpr size_t kBytes = keep_smem<S, true>();
    err = allow_smem<gdn_ssm_keep_kernel<T, S, true>>(kBytes);
    if (err != cudaSuccess) return err;
    gdn_ssm_keep_kernel<T, S, true><<<grid, kThreads, kBytes, stream>>>(p);
  } else {
    constexpr size_t kBytes = keep_smem<S, false>();
    err = allow_smem<gdn_ssm_keep_kernel<T, S, false>>(kBytes);
    if (err != cudaSuccess) return err;
    gdn_ssm_keep_kernel<T, S, false><<<grid, kThreads, kBytes, stream>>>(p);
  }
  err = taken(cudaGetLastError());
  if (err != cudaSuccess) return err;
  const dim3 tiles(groups * p.blocks, p.parts);
  constexpr size_t kGrad = 4 * Bwd<T, S>::kFloats;
  static_assert(Bwd<T, S>::kCtas * (kGrad + 1024) <= 228 * 1024, "CTAs that fit an SM");
  static_assert(Bwd<T, S>::kCtas == (sizeof(T) == 4 && S == 8 ? 1 : plan_ctas(sizeof(T) == 4, S)),
                "what the plan's comment says of them");
  if (p.gate) {
    err = allow_smem<gdn_ssm_grad_kernel<T, S, true>>(kGrad);
    if (err == cudaSuccess)
      err = launch_beside(gdn_ssm_grad_kernel<T, S, true>, tiles, kThreads, kGrad, stream, p);
  } else {
    err = allow_smem<gdn_ssm_grad_kernel<T, S, false>>(kGrad);
    if (err == cudaSuccess)
      err = launch_beside(gdn_ssm_grad_kernel<T, S, false>, tiles, kThreads, kGrad, stream, p);
  }
  if (err != cudaSuccess) return err;
  const int64_t bc = (p.rows() * groups * 2 * S + 1023) / 1024;
  const int64_t w = ((int64_t)p.D * (S + 2) + 31) / 32;
  if (bc + w > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_beside(gdn_ssm_sum_kernel<T>, dim3((unsigned)(bc + w)), 256, 0, stream, p, S, bc);
}
template <typename T>
cudaError_t launch_t(const BwdParams &p, int S, int groups, cudaStream_t stream) {
  switch (S) {
    case 8: return launch_s<T, 8>(p, groups, stream);
    case 16: return launch_s<T, 16>(p, groups, stream);
    case 32: return launch_s<T, 32>(p, groups, stream);
    default: return launch_s<T, 64>(p, groups, stream);
  }
}

}  // namespace
}  // namespace ssm
}  // namespace gdn

extern "C" {

size_t gdn_ssm_bwd_workspace_size(int32_t num_seqs, int32_t seq_len, int32_t channels,
                                  int32_t d_state, int32_t groups) {
  using namespace gdn::ssm;
  if (!some_sizes(num_seqs, seq_len, channels, d_state, groups)) return 0;
  const size_t dense = workspace_bytes_of(num_seqs, seq_len, false, channels, d_state, groups);
  const size_t packed = workspace_bytes_of(num_seqs, seq_len, true, channels, d_state, groups);
  return dense > packed ? dense : packed;
}
size_t gdn_ssm_bwd_packed_workspace_size(int32_t num_seqs, int32_t total_tokens, int32_t channels,
                                         int32_t d_state, int32_t groups) {
  using namespace gdn::ssm;
  if (!some_sizes(num_seqs, total_tokens, channels, d_state, groups)) return 0;
  return workspace_bytes_of(num_seqs, total_tokens, true, channels, d_state, groups);
}

gdn_status gdn_ssm_bwd(const void *x, const void *dt, const float *A_log, const void *b,
                       const void *c, const float *D_skip, const void *gate, const float *dt_bias,
                       const float *initial_state, const int32_t *cu_seqlens, const void *d_y,
                       const float *d_final_state, void *dx, void *ddt, float *dA_log, void *db,
                       void *dc, float *dD_skip, void *dgate, float *ddt_bias,
                       float *d_initial_state, int32_t batch, int32_t seq_len, int32_t channels,
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
  const size_t ds_bytes = (size_t)channels * d_state * 4, ch_bytes = (size_t)channels * 4;
  cudaStream_t s = (cudaStream_t)stream;
  if (seq_len == 0) {   // no tokens: the weights' gradients are zero, the states' pass through
    const gdn_status r = pass_states(d_final_state, d_initial_state, z.state, s);
    if (r != GDN_OK) return r;
    for (const auto &w : {Range{dA_log, ds_bytes}, Range{dD_skip, ch_bytes},
                          Range{ddt_bias, ch_bytes}})
      if (w.p && taken(cudaMemsetAsync(const_cast<void *>(w.p), 0, w.n, s)) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
  }
  if (!strides_of(z, x_stride, dt_stride, b_stride, c_stride, gate_stride))
    return GDN_ERR_INVALID_ARG;
  if (!x || !dt || !A_log || !b || !c || !d_y || !dx || !ddt || !db || !dc)
    return GDN_ERR_INVALID_ARG;
  if ((gate != nullptr) != (dgate != nullptr)) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {x, dt, A_log, b, c, D_skip, gate, dt_bias, initial_state, cu_seqlens, d_y,
                        d_final_state, dx, ddt, dA_log, db, dc, dD_skip, dgate, ddt_bias,
                        d_initial_state, workspace};
  if (!all_aligned(ptrs)) return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kStatusBytes) return GDN_ERR_WORKSPACE;

  const size_t wide = z.rows * channels * z.e, thin = z.rows * z.gs * z.e;
  const Range outs[] = {{dx, wide}, {ddt, wide}, {db, thin}, {dc, thin}, {dgate, wide},
                        {dA_log, ds_bytes}, {dD_skip, ch_bytes}, {ddt_bias, ch_bytes},
                        {d_initial_state, z.state}};
  const Range ins[] = {{workspace, workspace_bytes},
                       {x, span_bytes(z.rows, z.sx, z.D, z.e)},
                       {dt, span_bytes(z.rows, z.sdt, z.D, z.e)},
                       {b, span_bytes(z.rows, z.sb, z.gs, z.e)},
                       {c, span_bytes(z.rows, z.sc, z.gs, z.e)},
                       {gate, span_bytes(z.rows, z.sg, z.D, z.e)},
                       {A_log, ds_bytes}, {D_skip, ch_bytes}, {dt_bias, ch_bytes},
                       {cu_seqlens, (size_t)(num_seqs + 1) * 4}, {d_y, wide},
                       {initial_state, z.state}, {d_final_state, z.state}};
  if (!apart(outs, ins)) return GDN_ERR_INVALID_ARG;
  for (int i = 1; i < 13; ++i)
    if (overlaps(ins[0], ins[i])) return GDN_ERR_INVALID_ARG;

  BwdParams p{};
  p.x = x; p.dt = dt; p.b = b; p.c = c; p.gate = gate; p.dy = d_y;
  p.A_log = A_log; p.d_skip = D_skip; p.dt_bias = dt_bias;
  p.h0 = initial_state; p.dhT = d_final_state;
  p.dx = dx; p.ddt = ddt; p.db = db; p.dc = dc; p.dgate = dgate;
  p.dA_log = dA_log; p.dD_skip = dD_skip; p.ddt_bias = ddt_bias; p.dh0 = d_initial_state;
  p.sx = z.sx; p.sdt = z.sdt; p.sb = z.sb; p.sc = z.sc; p.sg = z.sg;
  p.D = channels;
  p.G = groups;
  p.Dg = channels / groups;
  p.blocks = channel_blocks(p.Dg, d_state);
  p.softplus = flags & GDN_DT_SOFTPLUS;
  p.seq.cu = cu_seqlens;
  p.seq.status = static_cast<DeviceStatus *>(workspace);
  p.seq.seq_len = seq_len;
  p.seq.num_seqs = num_seqs;
  const int64_t all = (int64_t)groups * p.blocks;
  auto pl = plan(num_seqs, seq_len, cu_seqlens != nullptr, all,
                 plan_ctas(dtype == GDN_F32, d_state), kFirst);
  Layout l;
  for (;;) {   // uncut where the workspace is too small for the segments
    p.parts = (int32_t)parts_of(pl.slots, all);
    l = layout((int64_t)z.rows, channels, d_state, groups, p.blocks, p.parts, pl);
    if (4 * l.total <= workspace_bytes - kStatusBytes) break;
    if (!pl.seg_len) return GDN_ERR_WORKSPACE;
    pl = {0, num_seqs};
  }
  p.seq.seg_len = pl.seg_len;
  p.seq.slots = pl.slots;
  float *ws = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kStatusBytes);
  p.seg_x = ws + l.x;
  p.seg_y = ws + l.y;
  p.seg_d = ws + l.d;
  p.ckpt = ws + l.ckpt;
  p.ckpt_d = ws + l.ckpt_d;
  p.part_bc = ws + l.bc;
  p.part_w = ws + l.w;
  p.own_w = ws + l.own;
  const cudaError_t err = dtype == GDN_F32 ? launch_t<float>(p, d_state, groups, s)
                                           : launch_t<__nv_bfloat16>(p, d_state, groups, s);
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
