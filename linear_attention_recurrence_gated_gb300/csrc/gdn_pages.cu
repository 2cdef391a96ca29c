// Pages of a state cache: copy, fork, free and compact.
//
// A pool holds num_pages pages of page_bytes.  Row r of the table owns
// counts[r] pages, table[r][0 .. counts[r] - 1]: shared snapshots first, the
// row's own current page last (entries past the count are -1 and never read).
// refs[p] is the number of rows that hold page p; a page with refs 0 is free.
//
// The bookkeeping of a call is a few thousand small integers with an order in
// it (the i-th new page is the i-th lowest free one), so one CTA does it with
// block-wide prefix sums and writes a list of page copies; the copies, which
// are the traffic (2 page_bytes each), run on the whole GPU in a second
// launch.  Every decision depends on the arguments alone, never on the order
// in which threads arrive: counters are only added to, and where two jobs name
// one row the first in the list wins.
//
// Measured: 192 forks of 256 KB pages (101 MB) 18 us on the device, of which 15 are the
// copies at the copy bandwidth and 3 the bookkeeping's chain of dependent loads; freeing
// 160 rows and compacting (303 of 1536 pages moved, 159 MB) 34 us, 23 of them copies.
#include <stdint.h>

#include "gdn_internal.cuh"
#include "gdn_launch.cuh"

namespace gdn {
namespace pages {
namespace {

constexpr int kPlan = 1024;   // threads of the bookkeeping CTA
constexpr int kCopy = 256;    // threads of a copying CTA
constexpr int kZero = -2;     // source of a page that is filled with zeros

struct Params {
  uint8_t *pool;
  int64_t page_bytes;
  int32_t num_pages, num_rows, max_pages, n;
  const int32_t *table, *counts, *refs;
  int32_t *table_out, *counts_out, *refs_out;
  const int32_t *a, *b;        // fork: parents, children; copy: sources, targets; free: rows
  int32_t *out;                // fork: the new pages; compact: the number of live pages
  DeviceStatus *status;
  int32_t *num_jobs;           // workspace
  int2 *jobs;                  // (source, target) of each copy; target < 0: none
  int32_t *tmp0, *tmp1, *tmp2;
};

__device__ __forceinline__ void bad(const Params &p, int i, uint32_t code, uint32_t site) {
  report(p.status, code, (uint32_t)i, 0u, site);
}

// Exclusive prefix sum of v over the CTA's threads; `total` gets the sum.
__device__ __forceinline__ int block_scan(int v, int &total, int *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();  // the last scan's reads are done
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < kPlan / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += y;
    }
    if (lane < kPlan / 32) warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[kPlan / 32 - 1];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
}

// The bookkeeping into its new tensors (those updated in place stay): 16 bytes at a
// time, the loads of all three ahead of the stores, one latency of memory for them.
__device__ __forceinline__ void copy_bookkeeping(const Params &p) {
  int32_t *const to[3] = {p.table_out, p.counts_out, p.refs_out};
  const int32_t *const from[3] = {p.table, p.counts, p.refs};
  const int64_t n[3] = {(int64_t)p.num_rows * p.max_pages, p.num_rows, p.num_pages};
  int64_t most = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (to[k] != from[k] && n[k] > most) most = n[k];
  for (int64_t i = threadIdx.x; 4 * i < most; i += kPlan) {
    int4 x[3];
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (to[k] != from[k] && 4 * i + 4 <= n[k]) x[k] = reinterpret_cast<const int4 *>(from[k])[i];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (to[k] == from[k]) continue;
      if (4 * i + 4 <= n[k])
        reinterpret_cast<int4 *>(to[k])[i] = x[k];
      else
        for (int64_t j = 4 * i; j < n[k]; ++j) to[k][j] = from[k][j];
    }
  }
}

// tmp0: count of the job's parent, -1 for a job that is left out (num jobs);
// tmp1: the job that owns a child row (num_rows); tmp2: the lowest free pages.
__global__ void __launch_bounds__(kPlan) fork_plan_kernel(const Params p) {
  let_second();
  __shared__ int warp_sums[kPlan / 32];
  const int tid = threadIdx.x, n = p.n, R = p.num_rows, M = p.max_pages;
  copy_bookkeeping(p);
  for (int i = tid; i < n; i += kPlan) {
    const int c = p.b[i];
    if (c >= 0 && c < R) p.tmp1[c] = INT32_MAX;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlan) {
    const int c = p.b[i];
    if (c >= 0 && c < R) atomicMin(&p.tmp1[c], i);
  }
  __syncthreads();
  int need_all = 0;
  for (int i0 = 0; i0 < n; i0 += kPlan) {
    const int i = i0 + tid;
    int cnt = -1;  // left out
    if (i < n) {
      const int par = p.a[i], c = p.b[i];
      bool ok = par >= -1 && par < R && c >= 0 && c < R && p.tmp1[c] == i;
      if (ok) {
        const int held = p.counts[c], have = par < 0 ? 0 : p.counts[par];
        // a new row (parent -1) or a child starts empty; a row that is its own
        // parent grows by a page
        ok = have >= 0 && have <= M && (par == c ? held < M : held == 0);
        for (int m = 0; ok && m < have; ++m) {
          const int pg = p.table[(int64_t)par * M + m];
          ok = pg >= 0 && pg < p.num_pages && p.refs[pg] > 0;
        }
        if (ok) cnt = have;
      }
      if (!ok) bad(p, i, GDN_ERR_DEVICE_CHECK, 0u);
      p.tmp0[i] = cnt;
    }
    int total;
    const int need = i < n && (cnt > 0 || (cnt == 0 && p.a[i] < 0));
    const int at = block_scan(need, total, warp_sums) + need_all;
    if (i < n) p.out[i] = need ? at : -1;  // the job's rank, for now
    need_all += total;
  }
  // the lowest free pages, as many as are needed
  int found = 0;
  for (int p0 = 0; p0 < p.num_pages && found < need_all; p0 += kPlan) {
    const int pg = p0 + tid;
    const int free = pg < p.num_pages && p.refs[pg] <= 0;
    int total;
    const int at = block_scan(free, total, warp_sums) + found;
    if (free && at < n) p.tmp2[at] = pg;
    found += total;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlan) {
    const int rank = p.out[i], cnt = p.tmp0[i], par = p.a[i], c = p.b[i];
    int2 job = make_int2(-1, -1);
    int page = -1;
    if (rank >= 0) {
      if (rank < found) {
        page = p.tmp2[rank];
        const bool grow = par == c;
        const int len = grow ? cnt + 1 : cnt < 1 ? 1 : cnt;  // pages of the child
        int32_t *row = p.table_out + (int64_t)c * M;
        const int32_t *from = p.table + (int64_t)(par < 0 ? 0 : par) * M;
        job = make_int2(par < 0 ? kZero : from[cnt - 1], page);
        if (!grow)
          for (int m = 0; m < M; ++m) {
            const int pg = m < len - 1 ? from[m] : -1;
            row[m] = pg;
            if (pg >= 0) atomicAdd(&p.refs_out[pg], 1);
          }
        row[len - 1] = page;
        p.refs_out[page] = 1;
        p.counts_out[c] = len;
      } else {
        bad(p, i, GDN_ERR_NO_PAGES, 0u);
      }
    }
    p.out[i] = page;
    p.jobs[i] = job;
  }
  if (tid == 0) *p.num_jobs = n;
}

__global__ void __launch_bounds__(kPlan) copy_plan_kernel(const Params p) {
  let_second();
  for (int i = threadIdx.x; i < p.n; i += kPlan) {
    const int s = p.a[i], d = p.b[i];
    const bool ok = s >= 0 && s < p.num_pages && d >= 0 && d < p.num_pages;
    if (!ok) bad(p, i, GDN_ERR_DEVICE_CHECK, 0u);
    p.jobs[i] = ok && s != d ? make_int2(s, d) : make_int2(-1, -1);
  }
  if (threadIdx.x == 0) *p.num_jobs = p.n;
}

// Pages four at a time: one latency for all.  `use(m, page)` for each of `cnt` entries.
template <typename F>
__device__ __forceinline__ void four_at_a_time(const int32_t *row, int cnt, F use) {
  for (int m0 = 0; m0 < cnt; m0 += 4) {
    int pg[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) pg[k] = m0 + k < cnt ? row[m0 + k] : -1;
    use(m0, pg);
  }
}

// Two passes: what breaks a rule is judged by the arguments as they came, before any of
// them changes, so that a job is left out whole and whatever the others do.  The jobs go
// to the last threads, which have the least to copy.  tmp0: the jobs' counts, -1 for one
// that is left out.
__global__ void __launch_bounds__(kPlan) free_kernel(const Params p) {
  const int R = p.num_rows, M = p.max_pages, first = kPlan - 1 - (int)threadIdx.x;
  for (int i = first; i < p.n; i += kPlan) {
    const int r = p.a[i];
    const bool there = r >= 0 && r < R;
    const int cnt = there ? p.counts[r] : -1;
    bool ok = cnt >= 0 && cnt <= M;
    if (ok)
      four_at_a_time(p.table + (int64_t)r * M, cnt, [&](int m0, const int (&pg)[4]) {
        int held[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          held[k] = pg[k] >= 0 && pg[k] < p.num_pages ? p.refs[pg[k]] : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) ok = ok && (m0 + k >= cnt || held[k] > 0);
      });
    if (!ok) bad(p, i, GDN_ERR_DEVICE_CHECK, 0u);
    p.tmp0[i] = ok ? cnt : -1;
  }
  copy_bookkeeping(p);
  __syncthreads();
  for (int i = first; i < p.n; i += kPlan) {
    if (p.tmp0[i] < 0) continue;
    const int r = p.a[i];
    const int cnt = atomicExch(&p.counts_out[r], 0);   // a row listed twice is freed once
    int32_t *row = p.table_out + (int64_t)r * M;
    four_at_a_time(row, cnt, [&](int m0, const int (&pg)[4]) {
      int held[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) held[k] = m0 + k < cnt ? atomicSub(&p.refs_out[pg[k]], 1) : 1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (m0 + k < cnt) row[m0 + k] = -1;
        if (held[k] <= 0) {   // held by more rows than it counts: it stays at zero
          atomicAdd(&p.refs_out[pg[k]], 1);
          bad(p, i, GDN_ERR_DEVICE_CHECK, 0u);
        }
      }
    });
  }
}

// tmp0: the new number of every page, -1 for a free one; tmp1: the free pages below the
// live count, ascending.  The k-th live page above it moves to the k-th of them.
__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const Params p) {
  let_second();
  __shared__ int warp_sums[kPlan / 32];
  const int tid = threadIdx.x, P = p.num_pages;
  constexpr int kHeld = 4;   // blocks of pages whose counts stay in registers
  int held[kHeld], mine = 0, live;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int pg = k * kPlan + tid;
    held[k] = pg < P ? p.refs[pg] : 0;
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k) mine += held[k] > 0;
  for (int pg = kHeld * kPlan + tid; pg < P; pg += kPlan) mine += p.refs[pg] > 0;
  block_scan(mine, live, warp_sums);
  int holes = 0, moves = 0;
  const auto block = [&](int p0, int r) {
    const int pg = p0 + tid;
    const int hole = pg < live && r <= 0, move = pg >= live && pg < P && r > 0;
    int total;
    const int at = block_scan(hole | (move << 16), total, warp_sums);
    if (hole) p.tmp1[holes + (at & 0xffff)] = pg;
    if (move) p.jobs[moves + (at >> 16)] = make_int2(pg, r);
    if (pg < P) {
      p.tmp0[pg] = r > 0 ? pg : -1;
      if (p.refs_out != p.refs) p.refs_out[pg] = r;
    }
    holes += total & 0xffff;
    moves += total >> 16;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (k * kPlan < P) block(k * kPlan, held[k]);
  for (int p0 = kHeld * kPlan; p0 < P; p0 += kPlan) block(p0, p0 + tid < P ? p.refs[p0 + tid] : 0);
  __syncthreads();
  for (int k = tid; k < moves; k += kPlan) {  // as many holes as moves
    const int2 m = p.jobs[k];
    const int to = p.tmp1[k];
    p.jobs[k] = make_int2(m.x, to);
    p.tmp0[m.x] = to;
    p.refs_out[to] = m.y;
    p.refs_out[m.x] = 0;
  }
  if (tid == 0) {
    *p.num_jobs = moves;
    *p.out = live;
  }
}

// Copies the pages of the list (and, for compact, rewrites the table).
__global__ void __launch_bounds__(kCopy) copy_pages_kernel(const Params p, int pieces,
                                                            int64_t piece_bytes, bool rewrite) {
  wait_first();  // the bookkeeping is done
  if (rewrite) {
    const int64_t all = (int64_t)p.num_rows * p.max_pages;
    for (int64_t i = (int64_t)blockIdx.x * kCopy + threadIdx.x; i < all;
         i += (int64_t)gridDim.x * kCopy) {
      const int r = (int)(i / p.max_pages), m = (int)(i % p.max_pages);
      const bool held = m < p.counts[r];
      const int pg = held ? p.table[i] : -1;
      const int to = pg >= 0 && pg < p.num_pages ? p.tmp0[pg] : -1;
      // a number out of range, or of a free page, where another may have moved to
      if (held && to < 0) bad(p, r, GDN_ERR_DEVICE_CHECK, 0u);
      p.table_out[i] = to;
    }
  }
  const int64_t work = (int64_t)*p.num_jobs * pieces;
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int2 job = p.jobs[w / pieces];
    if (job.y < 0) continue;
    const int64_t at = (w % pieces) * piece_bytes;
    const int64_t left = p.page_bytes - at, bytes = left < piece_bytes ? left : piece_bytes;
    uint4 *to = reinterpret_cast<uint4 *>(p.pool + (int64_t)job.y * p.page_bytes + at);
    const int n = (int)(bytes / 16);
    if (job.x == kZero) {
      for (int i = threadIdx.x; i < n; i += kCopy) to[i] = make_uint4(0, 0, 0, 0);
    } else {
      const uint4 *from =
          reinterpret_cast<const uint4 *>(p.pool + (int64_t)job.x * p.page_bytes + at);
      int i = threadIdx.x;
      for (; i + 7 * kCopy < n; i += 8 * kCopy) {  // eight loads on their way
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __ldcs(from + i + k * kCopy);
#pragma unroll
        for (int k = 0; k < 8; ++k) to[i + k * kCopy] = x[k];
      }
      for (; i < n; i += kCopy) to[i] = from[i];
    }
  }
}

// The copies start beside the bookkeeping and wait for its end (programmatic
// dependent launch: the wait is the hardware's), which hides their launch.
cudaError_t launch_copies(const Params &p, int64_t most, bool rewrite, cudaStream_t stream) {
  const int64_t piece = 32768;
  const int64_t pieces = (p.page_bytes + piece - 1) / piece;
  const int64_t want = most * pieces;
  const int grid = (int)(want < 1 ? 1 : want < 152 * 8 ? want : 152 * 8);
  return launch_beside(copy_pages_kernel, dim3(grid), kCopy, 0, stream, p, (int)pieces, piece, rewrite);
}

bool aligned16(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }
struct Range {
  const void *p;
  size_t n;
};
bool overlaps(const Range &a, const Range &b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
// Outputs overlap neither inputs nor one another, but outs[i] may be ins[i]
// itself for i < in_place.
template <int NI, int NO>
bool clash(const Range (&ins)[NI], const Range (&outs)[NO], int in_place) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (!(i == j && i < in_place && outs[i].p == ins[j].p) && overlaps(outs[i], ins[j]))
        return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Status record, copy count, then jobs and three lists.
size_t workspace_bytes_for(int64_t pages, int64_t rows, int64_t n) {
  const size_t most = (size_t)(pages > n ? pages : n);
  return kStatusBytes + 256 + align256(most * 8) + align256(most * 4) +
         align256((size_t)(pages > rows ? pages : rows) * 4) + align256(most * 4);
}
void carve(Params &p, void *workspace) {
  const size_t most = (size_t)(p.num_pages > p.n ? p.num_pages : p.n);
  const size_t rows = (size_t)(p.num_pages > p.num_rows ? p.num_pages : p.num_rows);
  uint8_t *w = static_cast<uint8_t *>(workspace);
  p.status = reinterpret_cast<DeviceStatus *>(w);
  w += kStatusBytes;
  p.num_jobs = reinterpret_cast<int32_t *>(w);
  w += 256;
  p.jobs = reinterpret_cast<int2 *>(w);
  w += align256(most * 8);
  p.tmp0 = reinterpret_cast<int32_t *>(w);
  w += align256(most * 4);
  p.tmp1 = reinterpret_cast<int32_t *>(w);
  w += align256(rows * 4);
  p.tmp2 = reinterpret_cast<int32_t *>(w);
}

gdn_status check(int32_t num_pages, int32_t num_rows, int32_t max_pages, int32_t n,
                 int64_t page_bytes, const void *ws, size_t ws_bytes) {
  if (num_pages <= 0 || num_rows < 0 || max_pages <= 0 || n < 0 || page_bytes <= 0)
    return GDN_ERR_INVALID_ARG;
  if (page_bytes % 16) return GDN_ERR_UNSUPPORTED;
  if (num_pages > (1 << 24) || num_rows > (1 << 24) || n > (1 << 24)) return GDN_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < workspace_bytes_for(num_pages, num_rows, n)) return GDN_ERR_WORKSPACE;
  if (!aligned16(ws)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

}  // namespace
}  // namespace pages
}  // namespace gdn

extern "C" {

size_t gdn_pages_workspace_size(int32_t num_pages, int32_t num_rows, int32_t n) {
  if (num_pages <= 0 || num_rows < 0 || n < 0) return 0;
  return gdn::pages::workspace_bytes_for(num_pages, num_rows, n);
}

gdn_status gdn_pages_copy(void *pool, int64_t page_bytes, int32_t num_pages, const int32_t *src,
                          const int32_t *dst, int32_t n, void *workspace, size_t workspace_bytes,
                          void *stream) {
  using namespace gdn;
  using namespace gdn::pages;
  const gdn_status st = check(num_pages, 0, 1, n, page_bytes, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  if (n == 0) return GDN_OK;
  if (!pool || !src || !dst) return GDN_ERR_INVALID_ARG;
  if (!aligned16(pool) || !aligned16(src) || !aligned16(dst)) return GDN_ERR_INVALID_ARG;
  const Range pool_r = {pool, (size_t)num_pages * page_bytes}, ws = {workspace, workspace_bytes};
  for (const Range &r : {Range{src, (size_t)n * 4}, Range{dst, (size_t)n * 4}})
    if (overlaps(pool_r, r) || overlaps(ws, r)) return GDN_ERR_INVALID_ARG;
  if (overlaps(pool_r, ws)) return GDN_ERR_INVALID_ARG;
  Params p{};
  p.pool = static_cast<uint8_t *>(pool);
  p.page_bytes = page_bytes;
  p.num_pages = num_pages;
  p.n = n;
  p.a = src;
  p.b = dst;
  carve(p, workspace);
  copy_plan_kernel<<<1, kPlan, 0, (cudaStream_t)stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  return launch_copies(p, n, false, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_pages_fork(void *pool, int64_t page_bytes, int32_t num_pages, const int32_t *table,
                          const int32_t *counts, const int32_t *refs, int32_t num_rows,
                          int32_t max_pages, const int32_t *parents, const int32_t *children,
                          int32_t n, int32_t *fresh, int32_t *table_out, int32_t *counts_out,
                          int32_t *refs_out, void *workspace, size_t workspace_bytes,
                          void *stream) {
  using namespace gdn;
  using namespace gdn::pages;
  const gdn_status st =
      check(num_pages, num_rows, max_pages, n, page_bytes, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  if (num_rows == 0 && n > 0) return GDN_ERR_INVALID_ARG;
  if (!pool || !refs || !refs_out) return GDN_ERR_INVALID_ARG;
  if (num_rows > 0 && (!table || !counts || !table_out || !counts_out)) return GDN_ERR_INVALID_ARG;
  if (n > 0 && (!parents || !children || !fresh)) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {pool, table, counts, refs, parents, children, fresh, table_out, counts_out,
                        refs_out};
  for (const void *q : ptrs)
    if (q && !aligned16(q)) return GDN_ERR_INVALID_ARG;
  const size_t b_t = (size_t)num_rows * max_pages * 4, b_r = (size_t)num_rows * 4,
               b_p = (size_t)num_pages * 4, b_n = (size_t)n * 4;
  const Range ins[] = {{table, b_t}, {counts, b_r}, {refs, b_p}, {parents, b_n}, {children, b_n}};
  const Range outs[] = {{table_out, b_t}, {counts_out, b_r}, {refs_out, b_p}, {fresh, b_n},
                        {pool, (size_t)num_pages * page_bytes}, {workspace, workspace_bytes}};
  if (clash(ins, outs, 3)) return GDN_ERR_INVALID_ARG;
  Params p{};
  p.pool = static_cast<uint8_t *>(pool);
  p.page_bytes = page_bytes;
  p.num_pages = num_pages; p.num_rows = num_rows; p.max_pages = max_pages; p.n = n;
  p.table = table; p.counts = counts; p.refs = refs;
  p.table_out = table_out; p.counts_out = counts_out; p.refs_out = refs_out;
  p.a = parents; p.b = children; p.out = fresh;
  carve(p, workspace);
  fork_plan_kernel<<<1, kPlan, 0, (cudaStream_t)stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  if (n == 0) return GDN_OK;
  return launch_copies(p, n, false, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_pages_free(const int32_t *table, const int32_t *counts, const int32_t *refs,
                          int32_t num_pages, int32_t num_rows, int32_t max_pages,
                          const int32_t *rows, int32_t n, int32_t *table_out, int32_t *counts_out,
                          int32_t *refs_out, void *workspace, size_t workspace_bytes,
                          void *stream) {
  using namespace gdn;
  using namespace gdn::pages;
  const gdn_status st = check(num_pages, num_rows, max_pages, n, 16, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  if (num_rows == 0 && n > 0) return GDN_ERR_INVALID_ARG;
  if (!refs || !refs_out || (n > 0 && !rows)) return GDN_ERR_INVALID_ARG;
  if (num_rows > 0 && (!table || !counts || !table_out || !counts_out)) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {table, counts, refs, rows, table_out, counts_out, refs_out};
  for (const void *q : ptrs)
    if (q && !aligned16(q)) return GDN_ERR_INVALID_ARG;
  const size_t b_t = (size_t)num_rows * max_pages * 4, b_r = (size_t)num_rows * 4,
               b_p = (size_t)num_pages * 4;
  const Range ins[] = {{table, b_t}, {counts, b_r}, {refs, b_p}, {rows, (size_t)n * 4}};
  const Range outs[] = {{table_out, b_t}, {counts_out, b_r}, {refs_out, b_p},
                        {workspace, workspace_bytes}};
  if (clash(ins, outs, 3)) return GDN_ERR_INVALID_ARG;
  Params p{};
  p.num_pages = num_pages; p.num_rows = num_rows; p.max_pages = max_pages; p.n = n;
  p.table = table; p.counts = counts; p.refs = refs;
  p.table_out = table_out; p.counts_out = counts_out; p.refs_out = refs_out;
  p.a = rows;
  carve(p, workspace);
  free_kernel<<<1, kPlan, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_pages_compact(void *pool, int64_t page_bytes, int32_t num_pages,
                             const int32_t *table, const int32_t *counts, const int32_t *refs,
                             int32_t num_rows, int32_t max_pages, int32_t *num_live,
                             int32_t *table_out, int32_t *refs_out, void *workspace,
                             size_t workspace_bytes, void *stream) {
  using namespace gdn;
  using namespace gdn::pages;
  const gdn_status st =
      check(num_pages, num_rows, max_pages, 0, page_bytes, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  if (!pool || !refs || !num_live || !refs_out) return GDN_ERR_INVALID_ARG;
  if (num_rows > 0 && (!table || !counts || !table_out)) return GDN_ERR_INVALID_ARG;
  const void *ptrs[] = {pool, table, counts, refs, num_live, table_out, refs_out};
  for (const void *q : ptrs)
    if (q && !aligned16(q)) return GDN_ERR_INVALID_ARG;
  const size_t b_t = (size_t)num_rows * max_pages * 4, b_p = (size_t)num_pages * 4;
  const Range ins[] = {{table, b_t}, {refs, b_p}, {counts, (size_t)num_rows * 4}};
  const Range outs[] = {{table_out, b_t}, {refs_out, b_p}, {num_live, 4},
                        {pool, (size_t)num_pages * page_bytes}, {workspace, workspace_bytes}};
  if (clash(ins, outs, 2)) return GDN_ERR_INVALID_ARG;
  Params p{};
  p.pool = static_cast<uint8_t *>(pool);
  p.page_bytes = page_bytes;
  p.num_pages = num_pages; p.num_rows = num_rows; p.max_pages = max_pages;
  p.table = table; p.counts = counts; p.refs = refs;
  p.table_out = table_out; p.refs_out = refs_out;
  p.out = num_live;
  carve(p, workspace);
  compact_plan_kernel<<<1, kPlan, 0, (cudaStream_t)stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  return launch_copies(p, num_pages / 2 + 1, true, (cudaStream_t)stream) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

}  // extern "C"
