// Linear attention with a decay for each head on the CUDA cores: the scan of
// gdn_lin.cuh in fp32, for fp32 storage and for head sizes without a
// tensor-core form.
//
// One CTA owns NV value columns of one (sequence, head) and walks its chunks of
// 64 tokens.  A chunk's e rows are loaded in the scan's order (the last token first
// backward in time), so that both directions are, with rows i, j of the tile:
//   P_ij = lam^(i-j) (a_i.b_j) for j <= i, else 0
//   o_i  = lam^(i+1) S^T a_i + sum_j P_ij c_j      (lam^i       backward)
//   S   <- lam^e S + sum_j lam^(e-1-j) b_j c_j^T   (lam^(e-j)   backward)
// The four products are fp32 fused multiply-adds on 4 x 4 register tiles: two
// 16-byte shared loads for every sixteen of them, so the fp32 pipes bound it (a
// chunk of 64 x 64 x 64 takes 4 x 2^18 of them, eight times what its bytes cost).
// [8, 2048, 16 heads, 64/64] takes 385 us, its backward pass 883, [4, 2048, 16, 128/128]
// 725 and 1647: the fp32 pipes are busy 45 % of the time and an instruction is issued
// in 66 % of the cycles (the rest waits for shared memory).  Small calls are latency:
// [1, 256, 2, 32/32], four chunks cut apart, takes 12 us on the device (28 uncut).
// P and its product skip what the mask leaves out, in blocks of 16 rows and columns.
// S stays in registers and is put into shared memory once a chunk.  Products beyond the
// mask are left out and rows past the sequence's end are never loaded, so nothing that
// lies there (an infinity, a NaN of a later token or of the next sequence) reaches a
// result.
#include "gdn_lin.cuh"
#include "gdn_launch.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kThreads = 256;
constexpr int kC = 64;        // tokens per chunk
constexpr int kPd = kC + 4;   // row of P

// floats of shared memory: A, B [64][da + 4], V [64][NV], P [64][68], S [da][NV],
// lam^0 .. lam^64; for the states alone B and V twice
__host__ __device__ constexpr size_t smem_floats(int da, int nv, bool states) {
  return 2 * (size_t)kC * (da + 4) + kC * nv + (states ? kC * nv : kC * kPd + da * nv) + kC + 4;
}

// Rows 0 .. 63 of a tile (cols values each, rows `stride` apart in memory) into
// shared memory, backwards from row e - 1 with `flip`, rows from e on as zeros; fp32
// by asynchronous copies.
template <typename T>
__device__ __forceinline__ void load_tile(float *to, int ld, const T *from, int64_t stride, int cols,
                                          int e, bool flip) {
  const int per = cols / 4;
  for (int x = threadIdx.x; x < kC * per; x += kThreads) {
    const int i = x / per, k = 4 * (x % per);
    float *dst = to + i * ld + k;
    const T *src = from + (i < e ? (flip ? e - 1 - i : i) * stride + k : 0);
    if constexpr (sizeof(T) == 4) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(dst)),
                   "l"(src), "r"(i < e ? 16 : 0)
                   : "memory");
    } else {
      uint2 v = make_uint2(0, 0);
      if (i < e) v = *reinterpret_cast<const uint2 *>(src);
      *reinterpret_cast<float4 *>(dst) =
          make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                      __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
    }
  }
}
__device__ __forceinline__ void loads_done() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

__device__ __forceinline__ float4 at4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
// acc[u][.] += x[u][.] . y rows: rows u of x (4 values of the sum's index each)
// times 4 rows of y
__device__ __forceinline__ void mul44(float (&acc)[4][4], const float4 (&x)[4], const float4 (&y)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      acc[u][0] = fmaf(xs[k], y[k].x, acc[u][0]);
      acc[u][1] = fmaf(xs[k], y[k].y, acc[u][1]);
      acc[u][2] = fmaf(xs[k], y[k].z, acc[u][2]);
      acc[u][3] = fmaf(xs[k], y[k].w, acc[u][3]);
    }
  }
}

__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                             *reinterpret_cast<const uint32_t *>(&b));
}

// NV value columns a CTA; the state's rows are held RT groups of four a pass, MK
// passes.  Where that takes fewer threads than there are (small heads), JS lanes
// share a tile of the state, each summing every JS-th token; they add up once a
// chunk.  STATES: the first launch of a split along time (the state increments
// alone).
template <typename T, int NV, int RT, int MK, bool STATES>
__global__ void __launch_bounds__(kThreads, 2)
gdn_lin_simt_kernel(const Params p) {
  if (STATES) let_second();
  extern __shared__ __align__(16) float sm[];
  constexpr int CG = NV / 4, RG = kThreads / CG;   // column and row groups of o
  constexpr int JS = RG / RT;
  const Scan &s = p.scan[blockIdx.z % p.num_scans];
  const int z = blockIdx.z / p.num_scans, h = blockIdx.y, col0 = blockIdx.x * NV;
  const bool second = !STATES && p.seg_len;   // (a CTA ends after the first launch in any case)
  if (col0 >= s.dc) {  // (the scans of a launch may have fewer tiles)
    if (second) wait_first();
    return;
  }
  const int tid = threadIdx.x, H = p.num_heads, da = s.da, dc = s.dc, ld = da + 4;
  const bool rev = s.reverse != 0;
  float *lam = sm, *B = lam + kC + 4, *V = B + kC * ld, *A = V + kC * NV, *P = A + kC * ld,
        *S = P + kC * kPd, *B2 = A, *V2 = B2 + kC * ld;   // (states alone: B and V twice)

  Span span;
  if (!span_of(p, z, h, span)) {
    if (second) wait_first();
    return;
  }
  const int64_t start = span.start, len = span.len;
  const int64_t unit = (int64_t)span.n * H + h;
  // the segment whose end is the sequence's, in the scan's direction
  const bool last = span.seg == (rev ? 0 : span.count - 1);
  const int64_t x_unit = ((int64_t)(blockIdx.z % p.num_scans) * p.slots + z) * H + h;  // of seg_x
  if (STATES && last) {
    if (keeps_copy(p, s))
      for (int i = tid; i < da * NV; i += kThreads) {
        const int j = col0 + i % NV;
        const int64_t at = (int64_t)(i / NV) * dc + j;
        if (j < dc) p.seg_x[x_unit * da * dc + at] = s.s_in[unit * da * dc + at];
      }
    return;
  }
  float *const s_out = STATES ? p.seg_x + x_unit * da * dc
                              : s.s_out && last ? s.s_out + unit * da * dc : nullptr;
  const float rate = p.log_decay[h];
  for (int i = tid; i <= kC; i += kThreads) lam[i] = i ? expf(rate * (float)i) : 1.f;

  const int rg = tid / CG, c0 = 4 * (tid % CG);   // of o
  // S: rows 4 rs + 4 RT m .. + 3, columns cs .. + 3, tokens js, js + JS, ...
  const int js = tid % JS, cs = 4 * (tid / JS % CG), rs = tid / (JS * CG);
  float st[MK][4][4];
#pragma unroll
  for (int m = 0; m < MK; ++m)
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int x = 0; x < 4; ++x) st[m][u][x] = 0.f;
  const auto add_state = [&](const float *from, float f) {  // st <- f st + [da][dc] rows of it
#pragma unroll
    for (int m = 0; m < MK; ++m)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = 4 * (rs + RT * m) + u;
        if (row < da) {
          const float4 y = at4(from + (int64_t)row * dc + col0 + cs);
          st[m][u][0] = fmaf(f, st[m][u][0], y.x);
          st[m][u][1] = fmaf(f, st[m][u][1], y.y);
          st[m][u][2] = fmaf(f, st[m][u][2], y.z);
          st[m][u][3] = fmaf(f, st[m][u][3], y.w);
        }
      }
  };
  const T *a = static_cast<const T *>(s.a) + (int64_t)h * da;
  const T *b = static_cast<const T *>(s.b) + (int64_t)h * da;
  const T *c = static_cast<const T *>(s.c) + (int64_t)h * dc + col0;
  T *o = static_cast<T *>(s.o) + (int64_t)h * dc + col0;

  const int64_t nc = (len + kC - 1) / kC;
  const auto token = [&](int64_t step) { return start + (rev ? nc - 1 - step : step) * kC; };
  const auto rows = [&](int64_t step) {
    const int64_t left = start + len - token(step);
    return (int)(left < kC ? left : kC);
  };
  const auto load_a = [&](int64_t step) {
    load_tile(A, ld, a + token(step) * s.sa, s.sa, da, rows(step), rev);
  };
  const auto load_b = [&](int64_t step, float *to) {
    load_tile(to, ld, b + token(step) * s.sb, s.sb, da, rows(step), rev);
  };
  const auto load_v = [&](int64_t step, float *to) {
    load_tile(to, NV, c + token(step) * s.sc, s.sc, NV, rows(step), rev);
  };
  if (nc > 0) {
    if (!STATES) load_a(0);
    load_b(0, B);
    load_v(0, V);
  }
  if (!STATES && js == 0) {
    if (second) wait_first();
    if (s.s_in && s.s_in_t) {
#pragma unroll
      for (int m = 0; m < MK; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = 4 * (rs + RT * m);
          if (row < da) {
            const float4 y = at4(s.s_in + unit * da * dc + (int64_t)(col0 + cs + x) * da + row);
            st[m][0][x] = y.x;
            st[m][1][x] = y.y;
            st[m][2][x] = y.z;
            st[m][3][x] = y.w;
          }
        }
    } else if (s.s_in) {
      add_state(keeps_copy(p, s)
                    ? p.seg_x + (x_unit + (int64_t)(span.count - 1 - span.seg) * H) * da * dc
                    : s.s_in + unit * da * dc,
                0.f);
    }
    // the segments before this one, in order
    for (int k = rev ? span.count - 1 : 0; k != span.seg; k += rev ? -1 : 1) {
      const int64_t length = k == span.count - 1 ? span.total - k * p.seg_len : p.seg_len;
      add_state(p.seg_x + (x_unit + (int64_t)(k - span.seg) * H) * da * dc,
                length ? expf(rate * (float)length) : 1.f);
    }
  }
  // every lane of a tile gets its sum; the first keeps it
  const auto join = [&]() {
    if constexpr (JS > 1)
#pragma unroll
      for (int m = 0; m < MK; ++m)
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int off = 1; off < JS; off <<= 1)
              st[m][u][x] += __shfl_xor_sync(0xffffffffu, st[m][u][x], off);
  };
  // Every tile's next load hides behind the products that it is not in: A behind the
  // state's update and P V, B behind P V, V behind A S and P of the next chunk.
  constexpr int U = kC / RG;
  for (int64_t step = 0; step < nc; ++step) {
    const int64_t tok = token(step);
    const int e = rows(step);
    const bool more = step + 1 < nc;
    float acc[4][4] = {};
    if (!STATES) {  // the state that this chunk reads
      join();
#pragma unroll
      for (int m = 0; m < MK; ++m)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = 4 * (rs + RT * m) + u;
          if (row < da && u % JS == js) store4(S + row * NV + cs, st[m][u]);
        }
    }
    loads_done();
    if (STATES && more) {  // into the other B and V
      load_b(step + 1, B2);
      load_v(step + 1, V2);
    }
    if (!STATES) {
      if (step) load_v(step, V);
      // o: rows rg + RG u (NV 32: two of them), columns c0 .. + 3
#pragma unroll 2
      for (int k = 0; k < da; k += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x[u] = at4(A + (rg + RG * (u % U)) * ld + k);
          y[u] = at4(S + (k + u) * NV + c0);
        }
        if constexpr (U == 4) {
          mul44(acc, x, y);
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              acc[u][0] = fmaf(xs[q], y[q].x, acc[u][0]);
              acc[u][1] = fmaf(xs[q], y[q].y, acc[u][1]);
              acc[u][2] = fmaf(xs[q], y[q].z, acc[u][2]);
              acc[u][3] = fmaf(xs[q], y[q].w, acc[u][3]);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = rg + RG * u;
        const float f = i < e ? lam[rev ? i : i + 1] : 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[u][x] *= f;
      }
      {  // P: rows i = tid / 16 + 16 u, columns j = tid % 16 + 16 w
        const int i0 = tid >> 4, j0 = tid & 15;
        float pij[4][4] = {};
#pragma unroll 2
        for (int k = 0; k < da; k += 4) {
          float4 x[4], y[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            x[u] = at4(A + (i0 + 16 * u) * ld + k);
            y[u] = at4(B + (j0 + 16 * u) * ld + k);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              if (w > u) continue;  // (beyond the mask)
              pij[u][w] = fmaf(x[u].x, y[w].x, pij[u][w]);
              pij[u][w] = fmaf(x[u].y, y[w].y, pij[u][w]);
              pij[u][w] = fmaf(x[u].z, y[w].z, pij[u][w]);
              pij[u][w] = fmaf(x[u].w, y[w].w, pij[u][w]);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int i = i0 + 16 * u, j = j0 + 16 * w;
            P[i * kPd + j] = i >= j ? pij[u][w] * lam[i - j] : 0.f;
          }
      }
      loads_done();
      if (more) load_a(step + 1);
    }
    // S <- lam^e S + sum_j b_j (w_j c_j)^T
    const float le = STATES || js == 0 ? lam[e] : 0.f;   // (joined: the first lane's)
#pragma unroll
    for (int m = 0; m < MK; ++m)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x) st[m][u][x] *= le;
#pragma unroll 4
    for (int j = js; j < e; j += JS) {
      const float w = lam[rev ? e - j : e - 1 - j];
      float4 v = at4(V + j * NV + cs);
      v.x *= w;
      v.y *= w;
      v.z *= w;
      v.w *= w;
#pragma unroll
      for (int m = 0; m < MK; ++m) {
        const int row = 4 * (rs + RT * m);
        if (row < da) {
          const float4 x = at4(B + j * ld + row);
          const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            st[m][u][0] = fmaf(xs[u], v.x, st[m][u][0]);
            st[m][u][1] = fmaf(xs[u], v.y, st[m][u][1]);
            st[m][u][2] = fmaf(xs[u], v.z, st[m][u][2]);
            st[m][u][3] = fmaf(xs[u], v.w, st[m][u][3]);
          }
        }
      }
    }
    if (!STATES) {
      __syncthreads();
      if (more) load_b(step + 1, B);
#pragma unroll
      for (int b16 = 0; b16 < kC; b16 += 16) {
        if (b16 >= e) break;
#pragma unroll 2
        for (int j = b16; j < b16 + 16; j += 4) {
          float4 y[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) y[u] = at4(V + (j + u) * NV + c0);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (RG * (u + 1) <= b16) continue;  // (beyond the mask)
            const bool edge = RG * u < b16 + 16;   // the mask runs through this block
            const float4 x = at4(P + (rg + RG * u) * kPd + j);
            const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              // left out, not multiplied by zero: a later value may not be finite
              if (edge && j + q > rg + RG * u) continue;
              acc[u][0] = fmaf(xs[q], y[q].x, acc[u][0]);
              acc[u][1] = fmaf(xs[q], y[q].y, acc[u][1]);
              acc[u][2] = fmaf(xs[q], y[q].z, acc[u][2]);
              acc[u][3] = fmaf(xs[q], y[q].w, acc[u][3]);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = rg + RG * u;
        if (i < e) store4(o + (tok + (rev ? e - 1 - i : i)) * ((int64_t)H * dc) + c0, acc[u]);
      }
    }
    if (STATES) {
      float *const b2 = B, *const v2 = V;
      B = B2, V = V2, B2 = b2, V2 = v2;
    }
  }
  join();
  if (s_out == nullptr) return;
#pragma unroll
  for (int m = 0; m < MK; ++m)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = 4 * (rs + RT * m) + u;
      if (row < da && u % JS == js) store4(s_out + (int64_t)row * dc + col0 + cs, st[m][u]);
    }
}

template <typename T, int NV, int RT, int MK, bool STATES>
cudaError_t run(const Params &p, int da, int dc, cudaStream_t stream) {
  const size_t bytes = smem_floats(da, NV, STATES) * 4;
  constexpr auto kernel = gdn_lin_simt_kernel<T, NV, RT, MK, STATES>;
  const cudaError_t err = allow_smem<kernel>(bytes);
  if (err != cudaSuccess) return err;
  const dim3 grid((dc + NV - 1) / NV, p.num_heads, p.slots * p.num_scans);
  if (!STATES && p.seg_len) return launch_beside(kernel, grid, kThreads, bytes, stream, p);
  kernel<<<grid, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, int NV, int RT, int MK>
cudaError_t run_split(const Params &p, int da, int dc, cudaStream_t stream) {
  if (p.seg_len) {
    const cudaError_t err = run<T, NV, RT, MK, true>(p, da, dc, stream);
    if (err != cudaSuccess) return err;
  }
  return run<T, NV, RT, MK, false>(p, da, dc, stream);
}

template <typename T>
cudaError_t launch_t(const Params &p, cudaStream_t stream) {
  int da = 0, dc = 0;
  bool wide = true;   // every scan in tiles of 64 columns
  for (int i = 0; i < p.num_scans; ++i) {
    da = p.scan[i].da > da ? p.scan[i].da : da;
    dc = p.scan[i].dc > dc ? p.scan[i].dc : dc;
    wide = wide && p.scan[i].dc % 64 == 0;
  }
  // 64 value columns a CTA share P twice as widely where the tiles fit (da <= 128):
  // [4, 1024, 16 heads] 64/64 102 us against 145 with 32 columns, [1, 1024, 4] 24 / 26;
  // 128/128 375 / 352 (one CTA a SM instead of two), its backward pass 856 / 1041
  wide = wide && da <= 128;
  Params on = p;
  split(on, dc / (wide ? 64 : 32), kSimtWidth, kC, 0.4, 0.4);
  if (wide)
    return da <= 32   ? run_split<T, 64, 8, 1>(on, da, dc, stream)
           : da <= 64 ? run_split<T, 64, 16, 1>(on, da, dc, stream)
                      : run_split<T, 64, 16, 2>(on, da, dc, stream);
  return da <= 32    ? run_split<T, 32, 8, 1>(on, da, dc, stream)
         : da <= 64  ? run_split<T, 32, 16, 1>(on, da, dc, stream)
         : da <= 128 ? run_split<T, 32, 32, 1>(on, da, dc, stream)
                     : run_split<T, 32, 32, 2>(on, da, dc, stream);
}

}  // namespace

cudaError_t launch_simt(const Params &p, gdn_dtype dtype, cudaStream_t stream) {
  return dtype == GDN_F32 ? launch_t<float>(p, stream) : launch_t<__nv_bfloat16>(p, stream);
}

}  // namespace lin
}  // namespace gdn
