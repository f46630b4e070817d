// Rows sorted by expert and back: the sort of a caller's selection, the rows
// in expert order, their gate-weighted sum per token, and the gradients.
//
// With pair p = (token t, expert e, gate g) and r(p) its row in expert order,
//   permute         rows[r(p)] = x[t], padding rows 0
//   its gradient    dx[t]      = sum_p drows[r(p)]
//   unpermute       out[t]     = sum_p g_p rows[r(p)]
//   its gradients   drows[r(p)] = g_p dout[t],  dg_p = <dout[t], rows[r(p)]>
// All of it is bound by bytes: each row is moved once, and each token's row is
// read once however many experts it goes to.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "moe.h"
#include "moe_internal.h"
#include "rows.cuh"

namespace moe {
namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// ----------------------------------------------------------------- sort
// The choices (t, k) are sorted by expert, stably, in chunks of 1024 ITERS.
// Inside a chunk each warp takes 32 ITERS consecutive choices and ranks 32 at a
// time: lanes with the same expert find each other with match_any, and a
// per-warp histogram in shared memory carries the count from one step to the
// next.  The warps' histograms are then summed in order, which gives each
// choice its rank among the chunk's choices of its expert.  One chunk needs
// one launch; more chunks leave their histograms in the workspace for a second
// launch, whose blocks each add up the chunks before theirs (nchunks * E
// values, a few KB) instead of waiting for a scan of their own.
//
// All of it is latency: short chunks (2 steps) where that leaves few of them,
// long ones (8) for many choices, where every block of the second launch reads
// all the histograms.  16384 x 8 choices over 128 experts: 11 us, with long
// chunks 18.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kShort = 2, kLong = 8;                        // steps of a chunk
constexpr int64_t kMostShort = 128 * kSortThreads * kShort;  // choices up to which chunks are short
constexpr int kScatter = kSortThreads;                      // choices per block of the second launch
inline int sort_steps(int64_t P) { return P <= kMostShort ? kShort : kLong; }

struct SortArgs {
  int64_t P;  // T * K choices
  int T, K, E, nchunks, chunk;  // chunk: choices of one
  const int* topk_idx;
  const float* topk_gate;
  int* tok_ptr;
  int* pair_expert;
  float* pair_gate;
  int* pair_row;
  int* pair_slot;  // nullable
  int* counts;
  int* offsets;
  int* row_tok;
  float* row_gate;
  int* tile_expert;
  int64_t P_max, R_max;
  int* hist;        // [nchunks, E]
  uint32_t* local;  // [P] rank in the chunk | kept choices before it in the chunk << 16
};

// Over the block's 1024 threads: the exclusive sums of `v`, and the totals of v,
// p and k, in one pass over the barriers.
struct BlockSums {
  int before, v, p, k;
};
__device__ __forceinline__ BlockSums block_sums(int v, int p, int k, int (*warp_sums)[kSortWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
    p += __shfl_xor_sync(0xffffffffu, p, o);
    k += __shfl_xor_sync(0xffffffffu, k, o);
  }
  if (lane == 31) warp_sums[0][warp] = x;
  if (lane == 0) warp_sums[1][warp] = p, warp_sums[2][warp] = k;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[0][lane], q = warp_sums[1][lane], r = warp_sums[2][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
      q += __shfl_xor_sync(0xffffffffu, q, o);
      r += __shfl_xor_sync(0xffffffffu, r, o);
    }
    warp_sums[0][lane] = s;
    if (lane == 0) warp_sums[1][0] = q, warp_sums[2][0] = r;
  }
  __syncthreads();
  return {x - v + (warp > 0 ? warp_sums[0][warp - 1] : 0), warp_sums[0][kSortWarps - 1], warp_sums[1][0],
          warp_sums[2][0]};
}

// The parts of a routing that no choice owns: padding rows and the tails
// past the used rows and pairs (token -1, gate 0), each tile's expert, counts
// and offsets.  off and cnt: shared arrays [E + 1] and [E].  Called by every
// block of the launch; the work is spread over all their warps.
__device__ __forceinline__ void fill_rest(const SortArgs& a, const int* off, const int* cnt, int64_t pairs) {
  const int lane = threadIdx.x & 31;
  const int64_t gw = (int64_t)blockIdx.x * kSortWarps + (threadIdx.x >> 5);
  const int64_t nw = (int64_t)gridDim.x * kSortWarps;
  for (int64_t e = gw; e < a.E; e += nw) {
    for (int r = off[e] + cnt[e] + lane; r < off[e + 1]; r += 32) {
      a.row_tok[r] = -1;
      a.row_gate[r] = 0.f;
    }
    for (int i = off[e] / kTile + lane; i < off[e + 1] / kTile; i += 32) a.tile_expert[i] = (int)e;
  }
  const int64_t g = gw * 32 + lane, n = nw * 32;
  const int64_t used = off[a.E];
  for (int64_t r = used + g; r < a.R_max; r += n) {
    a.row_tok[r] = -1;
    a.row_gate[r] = 0.f;
  }
  for (int64_t i = used / kTile + g; i < a.R_max / kTile; i += n) a.tile_expert[i] = -1;
  for (int64_t p = pairs + g; p < a.P_max; p += n) {
    a.pair_row[p] = -1;
    a.pair_expert[p] = -1;
    a.pair_gate[p] = 0.f;
    if (a.pair_slot) a.pair_slot[p] = -1;
  }
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e <= a.E; e += kSortThreads) {
      a.offsets[e] = off[e];
      if (e < a.E) a.counts[e] = cnt[e];
    }
    if (threadIdx.x == 0) a.tok_ptr[a.T] = (int)pairs;
  }
}

// choice i < 2^31 with gate g; `before`: kept choices before it
__device__ __forceinline__ void scatter_choice(const SortArgs& a, uint32_t i, int e, float g, int row, int64_t before) {
  const int t = (int)(i / (uint32_t)a.K);
  const uint32_t slot = i - (uint32_t)t * (uint32_t)a.K;
  if (slot == 0) a.tok_ptr[t] = (int)before;
  if (e < 0) return;
  a.pair_row[before] = row;
  a.pair_expert[before] = e;
  a.pair_gate[before] = g;
  if (a.pair_slot) a.pair_slot[before] = (int)slot;
  a.row_tok[row] = t;
  a.row_gate[row] = g;
}

// Dynamic shared memory: uint16 hist[32][E] (E rounded up to even), then, in
// the one-launch form, int off[E + 1] and cnt[E].
template <bool ONE, int ITERS>
__global__ void __launch_bounds__(kSortThreads) sort_rank_kernel(const SortArgs a) {
  pdl_wait();
  extern __shared__ __align__(16) uint8_t smem_sort[];
  __shared__ int warp_sums[3][kSortWarps];
  __shared__ int warp_kept[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E, Es = (E + 1) & ~1;
  uint16_t* hist = reinterpret_cast<uint16_t*>(smem_sort);
  // ONE: every block ranks all choices, and places and fills its share
  const int64_t first = ONE ? 0 : (int64_t)blockIdx.x * (kSortThreads * ITERS);
  const int64_t left = a.P - first;
  const int warps = (int)min((int64_t)kSortWarps, (left + 32 * ITERS - 1) / (32 * ITERS));  // those with choices
  for (int i = threadIdx.x; i < Es * warps / 2; i += kSortThreads) reinterpret_cast<uint32_t*>(hist)[i] = 0u;
  const int64_t i0 = first + warp * (32 * ITERS) + lane;
  int e[ITERS];
  float gate[ITERS];
  uint32_t rk[ITERS];
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int64_t i = i0 + it * 32;
    const int v = i < a.P ? __ldg(a.topk_idx + i) : -1;
    e[it] = (unsigned)v < (unsigned)E ? v : -1;
    gate[it] = ONE && i < a.P ? __ldg(a.topk_gate + i) : 0.f;
  }
  __syncthreads();
  uint16_t* mine = hist + warp * Es;
  uint32_t kept = 0;
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    rk[it] = 0;
    if (i0 - lane + it * 32 >= a.P) continue;  // the whole warp
    const unsigned same = __match_any_sync(0xffffffffu, e[it]);
    const unsigned live = __ballot_sync(0xffffffffu, e[it] >= 0);
    const unsigned below = (1u << lane) - 1;
    const uint32_t h = e[it] >= 0 ? mine[e[it]] : 0u;
    __syncwarp();
    if (e[it] >= 0 && (same & below) == 0) mine[e[it]] = (uint16_t)(h + __popc(same));
    __syncwarp();
    rk[it] = (h + __popc(same & below)) | (kept + __popc(live & below)) << 16;
    kept += __popc(live);
  }
  if (lane == 0) warp_kept[warp] = (int)kept;
  __syncthreads();
  int count = 0;  // thread x < E: expert x's choices of the chunk
  if (threadIdx.x < E) {
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const int v = hist[w * Es + threadIdx.x];
      hist[w * Es + threadIdx.x] = (uint16_t)count;
      count += v;
    }
  }
  uint32_t kept0 = 0;
  for (int w = 0; w < warp; ++w) kept0 += warp_kept[w];
  __syncthreads();
  if constexpr (!ONE) {
    if (threadIdx.x < E) a.hist[(size_t)blockIdx.x * E + threadIdx.x] = count;
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      const int64_t i = i0 + it * 32;
      if (i >= a.P) continue;
      const uint32_t base = e[it] >= 0 ? mine[e[it]] : 0u;
      a.local[i] = rk[it] + base + (kept0 << 16);
    }
  } else {
    int* off = reinterpret_cast<int*>(smem_sort + (size_t)Es * kSortWarps * 2);
    int* cnt = off + E + 1;
    const BlockSums sum = block_sums((count + kTile - 1) / kTile * kTile, count, 0, warp_sums);
    if (threadIdx.x < E) {
      off[threadIdx.x] = sum.before;
      cnt[threadIdx.x] = count;
    }
    if (threadIdx.x == 0) off[E] = sum.v;
    __syncthreads();
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      const int64_t i = i0 + it * 32;
      if (i >= a.P || warp % gridDim.x != blockIdx.x) continue;
      const int x = e[it];
      const int row = x >= 0 ? off[x] + mine[x] + (int)(rk[it] & 0xffffu) : -1;
      scatter_choice(a, (uint32_t)i, x, gate[it], row, (int64_t)kept0 + (rk[it] >> 16));
    }
    fill_rest(a, off, cnt, sum.p);
  }
}

__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const SortArgs a) {
  pdl_wait();
  extern __shared__ __align__(16) uint8_t smem_sort[];
  __shared__ int warp_sums[3][kSortWarps];
  const int E = a.E;
  int* off = reinterpret_cast<int*>(smem_sort);  // [E + 1]
  int* cnt = off + E + 1;                        // [E]
  int* base = cnt + E;                           // [E] first row of this chunk's choices of the expert
  const int64_t i = (int64_t)blockIdx.x * kScatter + threadIdx.x;  // this thread's choice
  const bool live = i < a.P;
  const int v = live ? __ldg(a.topk_idx + i) : -1;
  const float gate = live ? __ldg(a.topk_gate + i) : 0.f;
  const uint32_t local = live ? __ldg(a.local + i) : 0u;
  const int chunk = (int)((int64_t)blockIdx.x * kScatter / a.chunk);
  // column sums of the histograms, before this chunk and in all: several threads
  // per expert where there are few experts, so that the loads are in flight together
  int cols = 32;
  while (cols < E) cols <<= 1;
  const int parts = kSortThreads / cols, part = threadIdx.x / cols, col = threadIdx.x & (cols - 1);
  int before = 0, count = 0;
  if (col < E) {
    const int* h = a.hist + col;
#pragma unroll 16
    for (int c = part; c < a.nchunks; c += parts) {
      const int v = __ldg(h + (size_t)c * E);
      before += c < chunk ? v : 0;
      count += v;
    }
  }
  int* sum = base;  // [2][1024], then base
  sum[threadIdx.x] = before;
  sum[kSortThreads + threadIdx.x] = count;
  __syncthreads();
  if (threadIdx.x < cols) {
    for (int p = 1; p < parts; ++p) {
      before += sum[p * cols + threadIdx.x];
      count += sum[kSortThreads + p * cols + threadIdx.x];
    }
  } else {
    before = count = 0;
  }
  const BlockSums all = block_sums((count + kTile - 1) / kTile * kTile, count, before, warp_sums);
  if (threadIdx.x < E) {
    off[threadIdx.x] = all.before;
    cnt[threadIdx.x] = count;
    base[threadIdx.x] = all.before + before;
  }
  if (threadIdx.x == 0) off[E] = all.v;
  __syncthreads();
  if (live) {
    const int e = (unsigned)v < (unsigned)E ? v : -1;
    scatter_choice(a, (uint32_t)i, e, gate, e >= 0 ? base[e] + (int)(local & 0xffffu) : -1,
                   (int64_t)all.k + (local >> 16));
  }
  fill_rest(a, off, cnt, all.p);
}

cudaError_t launch_sort(SortArgs a, cudaStream_t s) {
  const int Es = (a.E + 1) & ~1;
  const size_t hist = (size_t)Es * kSortWarps * 2, seg = (size_t)(2 * a.E + 1) * 4;
  // limits set for the largest E, so that they are set once
  constexpr int kMost = 1024 * kSortWarps * 2 + 2049 * 4;
  const bool brief = a.chunk == kSortThreads * kShort;
  auto rank = a.nchunks <= 1 ? sort_rank_kernel<true, kShort>
                             : brief ? sort_rank_kernel<false, kShort> : sort_rank_kernel<false, kLong>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(rank), kMost);
  if (e != cudaSuccess) return e;
  // as many blocks as the rows to fill need (one alone took 10.4 us for 64 x 8
  // choices over 256 experts, 33280 rows, 5.5 with the work spread)
  const int64_t fill = std::max<int64_t>(1, std::min<int64_t>(32, cdiv(a.R_max, 2 * kSortThreads)));
  if (a.nchunks <= 1) return launch_pdl(rank, dim3((unsigned)fill), dim3(kSortThreads), hist + seg, s, a);
  e = launch_pdl(rank, dim3((unsigned)a.nchunks), dim3(kSortThreads), hist, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(sort_scatter_kernel, dim3((unsigned)std::max(fill, cdiv(a.P, kScatter))), dim3(kSortThreads),
                    (size_t)(2 * a.E + 1 + 2 * kSortThreads) * 4, s, a);
}

// ----------------------------------------------------------------- rows
// Rows move in 16-byte pieces, one per thread: blockDim.x pieces of blockDim.y
// tokens, grid.y column parts, so that a few tokens of a wide row still fill
// the machine and no thread divides to find its place.
//
// Where a base, a width or a stride is not a multiple of 16 bytes
// (ALIGNED = false), a row starts anywhere inside a 16-byte window.  Pieces
// are then cut at the windows of the row that is written, so that stores stay
// whole, and a piece of a row that is read comes from the two windows it lies
// in, shifted together (load16_any).  Pieces whose windows could reach outside
// their row are left out: those elements, at most 2 V - 2 at each end, go one
// by one to the lanes of one extra warp.  Nothing outside a row is read or
// written.  (One element per thread took 48.7 us, and pieces with their ends
// taken in place 45.2 us, where this takes 17.5 us: gradient of 5003 tokens of
// 1001 fp16 values, 6 choices each.)
struct Shape2 {
  dim3 block;
  unsigned parts;
};
Shape2 row_shape(int64_t pieces) {
  const int64_t parts = std::max<int64_t>(1, cdiv(pieces, 256));
  const int64_t x = std::max<int64_t>(32, cdiv(cdiv(pieces, parts), 32) * 32);
  return {dim3((unsigned)x, (unsigned)(256 / x)), (unsigned)parts};
}
// Threads of a row of `width` elements, V to a piece: unaligned rows have one
// piece more and their last 32 threads are the warp of the ends.
template <int V, bool ALIGNED>
__host__ __device__ __forceinline__ int row_threads(int64_t width) {
  return ALIGNED ? (int)(width / V) : (int)(((width + 2 * V - 2) / V + 31) / 32 * 32 + 32);
}

constexpr int kPadSplit = 4;  // blocks that share an expert's padding rows

// How a row that is written is cut: piece c holds elements
// [c V - h, c V - h + V); pieces lo .. hi - 1 are whole, with all windows of
// any row at another alignment inside the row; the elements below head_end and
// from tail on are the ends.
template <typename T>
struct Cut {
  int h, lo, hi;
  int head_end, tail;
};
template <typename T, bool ALIGNED>
__device__ __forceinline__ Cut<T> cut_row(const T* written, int width) {
  constexpr int V = kVec<T>;
  Cut<T> c;
  if (ALIGNED) {
    c.h = 0;
    c.lo = 0;
    c.hi = width / V;
    c.head_end = 0;
    c.tail = width;
    return c;
  }
  c.h = (int)(reinterpret_cast<uintptr_t>(written) & 15u) / (int)sizeof(T);
  c.lo = (V - 1 + c.h + V - 1) / V;             // first with c V - h >= V - 1
  const int room = width - 2 * V + 1 + c.h;     // last with c V - h + 2 V - 1 <= width
  c.hi = room < 0 ? 0 : room / V + 1;
  if (c.hi <= c.lo) c.hi = c.lo, c.head_end = c.tail = width;
  else c.head_end = c.lo * V - c.h, c.tail = c.hi * V - c.h;
  return c;
}
// the row's i-th end element
template <typename T>
__device__ __forceinline__ int end_elem(const Cut<T>& c, int i) {
  return i < c.head_end ? i : i - c.head_end + c.tail;
}
template <typename T>
__device__ __forceinline__ int num_ends(const Cut<T>& c, int width) { return c.head_end + width - c.tail; }
template <typename T>
__device__ __forceinline__ void store_piece(T* p, const Piece<T>& v) {
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&v);
}

// A thread's part of a row, `at` its place among the row's threads: calls
// piece(first element) for a whole piece, or one(element) for each end element.
template <typename T, bool ALIGNED, typename FPiece, typename FOne>
__device__ __forceinline__ void for_part(const T* written, int width, int at, FPiece piece, FOne one) {
  constexpr int V = kVec<T>;
  const Cut<T> c = cut_row<T, ALIGNED>(written, width);
  if constexpr (ALIGNED) {
    if (at < c.hi) piece(at * V);
  } else {
    const int ends_at = row_threads<V, false>(width) - 32;
    if (at < ends_at) {
      if (at >= c.lo && at < c.hi) piece(at * V - c.h);
    } else {
      const int n = num_ends(c, width);
      for (int i = at - ends_at; i < n; i += 32) one(end_elem(c, i));
    }
  }
}

// T: an integer of the element's size (bits are moved)
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(256) permute_kernel(int T_, unsigned tok_blocks, int width,
                                                      const int* __restrict__ tok_ptr,
                                                      const int* __restrict__ pair_row,
                                                      const int* __restrict__ offsets,
                                                      const int* __restrict__ counts, const T* __restrict__ src,
                                                      int64_t ld_src, T* __restrict__ rows, int64_t ld_rows) {
  pdl_wait();
  const int at = (int)(blockIdx.y * blockDim.x + threadIdx.x);
  if (at >= row_threads<kVec<T>, ALIGNED>(width)) return;
  if (blockIdx.x >= tok_blocks) {  // zeros into the padding rows of one expert
    const int b = (int)(blockIdx.x - tok_blocks);
    const int e = b / kPadSplit;
    const int end = __ldg(offsets + e + 1);
    Piece<T> zero;
    *reinterpret_cast<uint4*>(&zero) = make_uint4(0u, 0u, 0u, 0u);
    for (int r = __ldg(offsets + e) + __ldg(counts + e) + threadIdx.y + blockDim.y * (b % kPadSplit); r < end;
         r += blockDim.y * kPadSplit) {
      T* row = rows + (int64_t)r * ld_rows;
      for_part<T, ALIGNED>(row, width, at, [&](int e0) { store_piece(row + e0, zero); }, [&](int i) { row[i] = T(0); });
    }
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= T_) return;
  const int p0 = __ldg(tok_ptr + t), p1 = __ldg(tok_ptr + t + 1);
  const T* x = src + t * ld_src;
  if constexpr (ALIGNED) {  // the token's piece is read once
    const Piece<T> v = load_piece<T, true>(x + at * kVec<T>);
    for (int p = p0; p < p1; ++p) store_piece(rows + (int64_t)__ldg(pair_row + p) * ld_rows + at * kVec<T>, v);
  } else {  // each destination cuts it at its own windows; the repeated reads hit L1
    for (int p = p0; p < p1; ++p) {
      T* row = rows + (int64_t)__ldg(pair_row + p) * ld_rows;
      for_part<T, false>(row, width, at, [&](int e0) { store_piece(row + e0, load_piece<T, false>(x + e0)); },
                         [&](int i) { row[i] = x[i]; });
    }
  }
}

// acc += sum over N pairs from p on of (gate) * their rows' pieces, all N
// loads in flight before the first is used.
template <typename T, bool ALIGNED, bool GATE, int N>
__device__ __forceinline__ void add_pairs(float (&acc)[kVec<T>], int p, const int* __restrict__ pair_row,
                                          const float* __restrict__ pair_gate, const T* __restrict__ rows,
                                          int64_t ld_rows) {
  const T* from[N];
  Piece<T> v[N];
  float g[N];
#pragma unroll
  for (int j = 0; j < N; ++j) from[j] = rows + (int64_t)__ldg(pair_row + p + j) * ld_rows;
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = load_piece<T, ALIGNED>(from[j]);
#pragma unroll
  for (int j = 0; j < N; ++j) g[j] = GATE ? __ldg(pair_gate + p + j) : 1.f;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i)
      acc[i] = GATE ? fmaf(g[j], to_float(v[j].x[i]), acc[i]) : acc[i] + to_float(v[j].x[i]);
}

// out[t] = sum over the token's pairs of (gate) * rows[row], fp32 sums in
// pair order, rounded once.
template <typename T, bool ALIGNED, bool GATE>
__global__ void __launch_bounds__(256, 4) unpermute_kernel(int T_, int width, const int* __restrict__ tok_ptr,
                                                        const int* __restrict__ pair_row,
                                                        const float* __restrict__ pair_gate,
                                                        const T* __restrict__ rows, int64_t ld_rows,
                                                        T* __restrict__ out, int64_t ld_out) {
  pdl_wait();
  const int at = (int)(blockIdx.y * blockDim.x + threadIdx.x);
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= T_ || at >= row_threads<kVec<T>, ALIGNED>(width)) return;
  T* o = out + t * ld_out;
  const int p0 = __ldg(tok_ptr + t), p1 = __ldg(tok_ptr + t + 1);
  for_part<T, ALIGNED>(
      o, width, at,
      [&](int e0) {
        const T* from = rows + e0;
        int p = p0;
        float acc[kVec<T>];
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) acc[i] = 0.f;
        constexpr int kMost = ALIGNED ? 8 : 4;  // an unaligned piece is two loads
        for (; p + kMost <= p1; p += kMost) add_pairs<T, ALIGNED, GATE, kMost>(acc, p, pair_row, pair_gate, from, ld_rows);
        if (kMost > 4 && p + 4 <= p1) {
          add_pairs<T, ALIGNED, GATE, 4>(acc, p, pair_row, pair_gate, from, ld_rows);
          p += 4;
        }
        if (p + 2 <= p1) {
          add_pairs<T, ALIGNED, GATE, 2>(acc, p, pair_row, pair_gate, from, ld_rows);
          p += 2;
        }
        if (p < p1) add_pairs<T, ALIGNED, GATE, 1>(acc, p, pair_row, pair_gate, from, ld_rows);
        Piece<T> v;
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) v.x[i] = from_float<T>(acc[i]);
        store_piece(o + e0, v);
      },
      [&](int i) {
        float acc = 0.f;
#pragma unroll 4
        for (int p = p0; p < p1; ++p) {
          const float v = to_float(rows[(int64_t)__ldg(pair_row + p) * ld_rows + i]);
          acc = GATE ? fmaf(__ldg(pair_gate + p), v, acc) : acc + v;
        }
        o[i] = from_float<T>(acc);
      });
}

// One warp per pair: drows[r] = g dout[t] and dg = <dout[t], rows[r]>, the
// row's products summed in fp32 (per lane, then over the lanes in a fixed
// order).  A token's pairs are neighbours, so its dout row comes from DRAM
// once.  The blocks past the pairs zero the padding rows and the gate
// gradients of dropped choices.  A pair's slot is the one its sort wrote; in a
// routing without these, a token with K pairs has them in slot order, and one
// with fewer has them in the order of topk_idx's choices inside [0, E).
struct UnpermuteBwdArgs {
  int64_t T, P_max;
  int width, E, K;
  unsigned pair_blocks, pad_blocks;
  const int *tok_ptr, *pair_row, *row_tok, *offsets, *counts, *topk_idx;
  const int* pair_slot;  // nullable
  const float* pair_gate;
  float *pair_dgate, *topk_dgate;  // each nullable
  int64_t ld_dout, ld_rows, ld_drows;
};
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(256, 4) unpermute_bwd_kernel(const UnpermuteBwdArgs a, const T* __restrict__ dout,
                                                               const T* __restrict__ rows, T* __restrict__ drows) {
  pdl_wait();
  constexpr int V = kVec<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x >= a.pair_blocks + a.pad_blocks) {
    const int64_t step = (int64_t)(gridDim.x - a.pair_blocks - a.pad_blocks) * 256;
    for (int64_t t = (int64_t)(blockIdx.x - a.pair_blocks - a.pad_blocks) * 256 + threadIdx.x; t < a.T; t += step) {
      const int p0 = __ldg(a.tok_ptr + t), p1 = __ldg(a.tok_ptr + t + 1);
      if (p1 - p0 == a.K) continue;
      unsigned kept = 0;
      if (a.pair_slot) {
        for (int p = p0; p < p1; ++p) kept |= 1u << (__ldg(a.pair_slot + p) & 31);
      } else {
        for (int k = 0; k < a.K; ++k)
          if ((unsigned)__ldg(a.topk_idx + t * a.K + k) < (unsigned)a.E) kept |= 1u << k;
      }
      for (int k = 0; k < a.K; ++k)
        if (!(kept >> k & 1)) a.topk_dgate[t * a.K + k] = 0.f;
    }
    return;
  }
  if (blockIdx.x >= a.pair_blocks) {
    const int b = (int)(blockIdx.x - a.pair_blocks);
    const int e = b / kPadSplit;
    const int end = __ldg(a.offsets + e + 1);
    Piece<T> zero;
    *reinterpret_cast<uint4*>(&zero) = make_uint4(0u, 0u, 0u, 0u);
    for (int r = __ldg(a.offsets + e) + __ldg(a.counts + e) + 8 * (b % kPadSplit) + warp; r < end;
         r += 8 * kPadSplit) {
      T* row = drows + (int64_t)r * a.ld_drows;
      for (int at = lane; at < row_threads<V, ALIGNED>(a.width); at += 32)
        for_part<T, ALIGNED>(row, a.width, at, [&](int e0) { store_piece(row + e0, zero); },
                             [&](int i) { row[i] = from_float<T>(0.f); });
    }
    return;
  }
  const int64_t p = (int64_t)blockIdx.x * 8 + warp;
  if (p >= __ldg(a.tok_ptr + a.T)) return;
  const int64_t r = __ldg(a.pair_row + p);
  const int t = __ldg(a.row_tok + r);
  const float g = __ldg(a.pair_gate + p);
  const T* d = dout + (int64_t)t * a.ld_dout;
  const T* y = rows + r * a.ld_rows;
  T* o = drows + r * a.ld_drows;
  float dot = 0.f;
  const Cut<T> cut = cut_row<T, ALIGNED>(o, a.width);
  constexpr int kAhead = 2;
  for (int c0 = cut.lo + lane; c0 < cut.hi; c0 += 32 * kAhead) {
    Piece<T> dv[kAhead], yv[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (c0 + 32 * u < cut.hi) {
        const int e0 = (c0 + 32 * u) * V - cut.h;
        yv[u] = load_piece<T, ALIGNED>(y + e0);
        dv[u] = load_piece<T, ALIGNED>(d + e0);
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (c0 + 32 * u < cut.hi) {
        Piece<T> w;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float x = to_float(dv[u].x[i]);
          dot = fmaf(x, to_float(yv[u].x[i]), dot);
          w.x[i] = from_float<T>(g * x);
        }
        store_piece(o + (c0 + 32 * u) * V - cut.h, w);
      }
  }
  if constexpr (!ALIGNED) {
    const int n = num_ends(cut, a.width);
    for (int i = lane; i < n; i += 32) {
      const int k = end_elem(cut, i);
      const float x = to_float(d[k]);
      dot = fmaf(x, to_float(y[k]), dot);
      o[k] = from_float<T>(g * x);
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
  if (a.pair_dgate && lane == 0) a.pair_dgate[p] = dot;
  if (a.topk_dgate) {
    const int p0 = __ldg(a.tok_ptr + t);
    int slot = (int)p - p0;
    if (a.pair_slot) {
      slot = __ldg(a.pair_slot + p);
    } else if (__ldg(a.tok_ptr + t + 1) - p0 != a.K) {
      const int v = lane < a.K ? __ldg(a.topk_idx + (int64_t)t * a.K + lane) : -1;
      unsigned kept = __ballot_sync(0xffffffffu, (unsigned)v < (unsigned)a.E);
      for (int j = slot; j > 0; --j) kept &= kept - 1;
      slot = __ffs(kept) - 1;
    }
    if (lane == 0 && (unsigned)slot < (unsigned)a.K) a.topk_dgate[(int64_t)t * a.K + slot] = dot;
  }
}

// ----------------------------------------------------------------- launches
template <typename T, bool ALIGNED>
cudaError_t launch_permute_rows(int64_t T_, int E, int64_t width, const moe_routing* rt, const void* src,
                                int64_t ld_src, void* rows, int64_t ld_rows, cudaStream_t s) {
  const Shape2 sh = row_shape(row_threads<kVec<T>, ALIGNED>(width));
  const unsigned tok_blocks = (unsigned)cdiv(T_, sh.block.y);
  return launch_pdl(permute_kernel<T, ALIGNED>, dim3(tok_blocks + (unsigned)(E * kPadSplit), sh.parts), sh.block, 0, s,
                    (int)T_, tok_blocks, (int)width, (const int*)rt->tok_ptr, (const int*)rt->pair_row,
                    (const int*)rt->offsets, (const int*)rt->counts, static_cast<const T*>(src), ld_src,
                    static_cast<T*>(rows), ld_rows);
}

bool whole_pieces(const void* const* ptrs, int n_ptrs, const int64_t* elems, int n_elems, int64_t esize) {
  for (int i = 0; i < n_ptrs; ++i)
    if (reinterpret_cast<uintptr_t>(ptrs[i]) % 16) return false;
  for (int i = 0; i < n_elems; ++i)
    if (elems[i] * esize % 16) return false;
  return true;
}

template <typename T, bool ALIGNED, bool GATE>
cudaError_t launch_unpermute_one(int64_t T_, int64_t width, const moe_routing* rt, const void* rows, int64_t ld_rows,
                                 void* out, int64_t ld_out, cudaStream_t s) {
  const Shape2 sh = row_shape(row_threads<kVec<T>, ALIGNED>(width));
  return launch_pdl(unpermute_kernel<T, ALIGNED, GATE>, dim3((unsigned)cdiv(T_, sh.block.y), sh.parts), sh.block, 0, s,
                    (int)T_, (int)width, (const int*)rt->tok_ptr, (const int*)rt->pair_row, (const float*)rt->pair_gate,
                    static_cast<const T*>(rows), ld_rows, static_cast<T*>(out), ld_out);
}

template <typename T, bool GATE>
cudaError_t launch_unpermute(int64_t T_, int64_t width, const moe_routing* rt, const void* rows, int64_t ld_rows,
                             void* out, int64_t ld_out, cudaStream_t s) {
  const void* ptrs[] = {rows, out};
  const int64_t elems[] = {width, ld_rows, ld_out};
  if (whole_pieces(ptrs, 2, elems, 3, sizeof(T)))
    return launch_unpermute_one<T, true, GATE>(T_, width, rt, rows, ld_rows, out, ld_out, s);
  return launch_unpermute_one<T, false, GATE>(T_, width, rt, rows, ld_rows, out, ld_out, s);
}

template <typename T>
cudaError_t launch_unpermute_bwd(UnpermuteBwdArgs a, const void* dout, const void* rows, void* drows,
                                 cudaStream_t s) {
  const void* ptrs[] = {dout, rows, drows};
  const int64_t elems[] = {a.width, a.ld_dout, a.ld_rows, a.ld_drows};
  a.pair_blocks = (unsigned)cdiv(a.P_max, 8);
  a.pad_blocks = (unsigned)(a.E * kPadSplit);
  const unsigned extra = a.topk_dgate ? (unsigned)std::min<int64_t>(148, cdiv(a.T, 256)) : 0;
  const dim3 grid(a.pair_blocks + a.pad_blocks + extra);
  if (whole_pieces(ptrs, 3, elems, 4, sizeof(T)))
    return launch_pdl(unpermute_bwd_kernel<T, true>, grid, dim3(256), 0, s, a, static_cast<const T*>(dout),
                      static_cast<const T*>(rows), static_cast<T*>(drows));
  return launch_pdl(unpermute_bwd_kernel<T, false>, grid, dim3(256), 0, s, a, static_cast<const T*>(dout),
                    static_cast<const T*>(rows), static_cast<T*>(drows));
}

// ----------------------------------------------------------------- argument checks
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t elem_size(moe_dtype t) {
  switch (t) {
    case MOE_BF16:
    case MOE_F16: return 2;
    case MOE_F32: return 4;
    case MOE_E4M3: return 1;
  }
  return 0;
}

// The arrays of a routing that the row movement reads.
bool rows_routing_ok(const moe_routing* rt) {
  if (!rt) return false;
  const void* req[] = {rt->tok_ptr, rt->pair_row, rt->pair_gate, rt->counts, rt->offsets, rt->row_tok};
  for (const void* q : req)
    if (!q || !aligned16(q)) return false;
  return true;
}
moe_status check_rows(int64_t T, int32_t E, moe_dtype type, int64_t width, const moe_routing* rt) {
  const int64_t es = elem_size(type);
  if (es == 0) return MOE_ERR_INVALID_ARG;
  if (T < 0 || width < 1 || !rows_routing_ok(rt)) return MOE_ERR_INVALID_ARG;
  if (E < 1 || E > 1024 || T >= (int64_t(1) << 31) - 4096 || width > (int64_t(1) << 20)) return MOE_ERR_UNSUPPORTED;
  if (rt->P_max < 0 || rt->P_max >= (int64_t(1) << 31) || rt->R_max >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
// A row tensor: a base aligned to its elements and a stride of at least a row.
bool rows_ok(const void* p, int64_t ld, int64_t width, moe_dtype type) {
  return p && ld >= width && reinterpret_cast<uintptr_t>(p) % (uintptr_t)elem_size(type) == 0;
}

moe_status sort_plan(int64_t T, int32_t E, int32_t K, int64_t* P, int64_t* R, size_t* ws) {
  if (T < 0 || E < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  constexpr int64_t kMostPairs = (int64_t(1) << 31) - 4096 * 1024;
  if (E > 1024 || K > 32 || T >= kMostPairs || T * (int64_t)K >= kMostPairs) return MOE_ERR_UNSUPPORTED;
  *P = T * K;
  *R = cdiv(*P + (int64_t)(kTile - 1) * std::min<int64_t>(E, *P), kTile) * kTile;
  const int64_t chunks = cdiv(*P, kSortThreads * sort_steps(*P));
  *ws = chunks <= 1 ? 0 : align256((size_t)chunks * E * sizeof(int)) + align256((size_t)*P * sizeof(uint32_t));
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

#define MOE_TRY_CUDA(...)                                                               \
  do {                                                                                  \
    const cudaError_t moe_e_ = (__VA_ARGS__);                                           \
    if (moe_e_ != cudaSuccess) return api_cuda_failed(moe_e_, "moe_move.cu", __LINE__); \
  } while (0)

extern "C" {

moe_status moe_sort_sizes(int64_t T, int32_t E, int32_t K, int64_t* P_max, int64_t* R_max, size_t* ws_bytes) {
  if (!P_max || !R_max || !ws_bytes) return MOE_ERR_INVALID_ARG;
  return sort_plan(T, E, K, P_max, R_max, ws_bytes);
}

moe_status moe_sort_pairs(int64_t T, int32_t E, int32_t K, const moe_routing* rt, void* ws, size_t ws_bytes,
                          void* stream) {
  ApiRange api_range("moe_sort_pairs");
  int64_t P, R;
  size_t need;
  moe_status st = sort_plan(T, E, K, &P, &R, &need);
  if (st != MOE_OK) return st;
  if (!rows_routing_ok(rt)) return MOE_ERR_INVALID_ARG;
  const void* req[] = {rt->pair_expert, rt->row_gate, rt->tile_expert};
  for (const void* q : req)
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(rt->pair_slot)) return MOE_ERR_INVALID_ARG;
  if (P > 0 && (!rt->topk_idx || !rt->topk_gate || (reinterpret_cast<uintptr_t>(rt->topk_idx) & 3u) ||
                (reinterpret_cast<uintptr_t>(rt->topk_gate) & 3u)))
    return MOE_ERR_INVALID_ARG;
  if (rt->P_max < P || rt->R_max < R || rt->R_max % kTile != 0) return MOE_ERR_INVALID_ARG;
  if (rt->R_max >= (int64_t(1) << 31) || rt->P_max >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (need > 0 && !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  SortArgs a;
  a.P = P;
  a.T = (int)T;
  a.K = K;
  a.E = E;
  a.chunk = kSortThreads * sort_steps(P);
  a.nchunks = (int)cdiv(P, a.chunk);
  a.topk_idx = rt->topk_idx;
  a.topk_gate = rt->topk_gate;
  a.tok_ptr = rt->tok_ptr;
  a.pair_expert = rt->pair_expert;
  a.pair_gate = rt->pair_gate;
  a.pair_row = rt->pair_row;
  a.pair_slot = rt->pair_slot;
  a.counts = rt->counts;
  a.offsets = rt->offsets;
  a.row_tok = rt->row_tok;
  a.row_gate = rt->row_gate;
  a.tile_expert = rt->tile_expert;
  a.P_max = rt->P_max;
  a.R_max = rt->R_max;
  a.hist = static_cast<int*>(ws);
  a.local = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + align256((size_t)a.nchunks * E * sizeof(int)));
  ProfScope ps(s, "sort_pairs");
  MOE_TRY_CUDA(launch_sort(a, s));
  return MOE_OK;
}

moe_status moe_permute(int64_t T, int32_t E, const moe_routing* rt, moe_dtype type, int64_t width, const void* src,
                       int64_t ld_src, void* rows, int64_t ld_rows, void* stream) {
  ApiRange api_range("moe_permute");
  const moe_status st = check_rows(T, E, type, width, rt);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!rows_ok(src, ld_src, width, type) || !rows_ok(rows, ld_rows, width, type)) return MOE_ERR_INVALID_ARG;
  const int64_t es = elem_size(type);
  const void* ptrs[] = {src, rows};
  const int64_t elems[] = {width, ld_src, ld_rows};
  const bool whole = whole_pieces(ptrs, 2, elems, 3, es);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope ps(s, "permute");
  if (whole)  // in bytes: the pieces are the same whatever the type
    MOE_TRY_CUDA(launch_permute_rows<uint8_t, true>(T, E, width * es, rt, src, ld_src * es, rows, ld_rows * es, s));
  else if (es == 4)
    MOE_TRY_CUDA(launch_permute_rows<uint32_t, false>(T, E, width, rt, src, ld_src, rows, ld_rows, s));
  else if (es == 2)
    MOE_TRY_CUDA(launch_permute_rows<uint16_t, false>(T, E, width, rt, src, ld_src, rows, ld_rows, s));
  else
    MOE_TRY_CUDA(launch_permute_rows<uint8_t, false>(T, E, width, rt, src, ld_src, rows, ld_rows, s));
  return MOE_OK;
}

static moe_status sum_rows(bool gate, int64_t T, int32_t E, const moe_routing* rt, moe_dtype type, int64_t width,
                           const void* rows, int64_t ld_rows, void* out, int64_t ld_out, cudaStream_t s) {
  const moe_status st = check_rows(T, E, type, width, rt);
  if (st != MOE_OK) return st;
  if (type == MOE_E4M3) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!rows_ok(rows, ld_rows, width, type) || !rows_ok(out, ld_out, width, type)) return MOE_ERR_INVALID_ARG;
  ProfScope ps(s, gate ? "unpermute" : "permute_bwd");
  switch (type) {
    case MOE_BF16:
      MOE_TRY_CUDA(gate ? launch_unpermute<__nv_bfloat16, true>(T, width, rt, rows, ld_rows, out, ld_out, s)
                        : launch_unpermute<__nv_bfloat16, false>(T, width, rt, rows, ld_rows, out, ld_out, s));
      break;
    case MOE_F16:
      MOE_TRY_CUDA(gate ? launch_unpermute<__half, true>(T, width, rt, rows, ld_rows, out, ld_out, s)
                        : launch_unpermute<__half, false>(T, width, rt, rows, ld_rows, out, ld_out, s));
      break;
    default:
      MOE_TRY_CUDA(gate ? launch_unpermute<float, true>(T, width, rt, rows, ld_rows, out, ld_out, s)
                        : launch_unpermute<float, false>(T, width, rt, rows, ld_rows, out, ld_out, s));
  }
  return MOE_OK;
}

moe_status moe_permute_bwd(int64_t T, int32_t E, const moe_routing* rt, moe_dtype type, int64_t width,
                           const void* drows, int64_t ld_drows, void* dsrc, int64_t ld_dsrc, void* stream) {
  ApiRange api_range("moe_permute_bwd");
  return sum_rows(false, T, E, rt, type, width, drows, ld_drows, dsrc, ld_dsrc, static_cast<cudaStream_t>(stream));
}

moe_status moe_unpermute(int64_t T, int32_t E, const moe_routing* rt, moe_dtype type, int64_t width, const void* rows,
                         int64_t ld_rows, void* out, int64_t ld_out, void* stream) {
  ApiRange api_range("moe_unpermute");
  return sum_rows(true, T, E, rt, type, width, rows, ld_rows, out, ld_out, static_cast<cudaStream_t>(stream));
}

moe_status moe_unpermute_bwd(int64_t T, int32_t E, int32_t K, const moe_routing* rt, moe_dtype type, int64_t width,
                             const void* dout, int64_t ld_dout, const void* rows, int64_t ld_rows, void* drows,
                             int64_t ld_drows, float* pair_dgate, float* topk_dgate, void* stream) {
  ApiRange api_range("moe_unpermute_bwd");
  const moe_status st = check_rows(T, E, type, width, rt);
  if (st != MOE_OK) return st;
  if (type == MOE_E4M3) return MOE_ERR_UNSUPPORTED;
  if (topk_dgate && (K < 1 || K > 32)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!rows_ok(dout, ld_dout, width, type) || !rows_ok(rows, ld_rows, width, type) ||
      !rows_ok(drows, ld_drows, width, type))
    return MOE_ERR_INVALID_ARG;
  if (topk_dgate && !rt->topk_idx && !rt->pair_slot) return MOE_ERR_INVALID_ARG;
  if (!aligned16(rt->pair_slot)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  UnpermuteBwdArgs a;
  a.T = T;
  a.width = (int)width;
  a.P_max = rt->P_max;
  a.E = E;
  a.K = topk_dgate ? K : 0;
  a.tok_ptr = rt->tok_ptr;
  a.pair_row = rt->pair_row;
  a.row_tok = rt->row_tok;
  a.offsets = rt->offsets;
  a.counts = rt->counts;
  a.topk_idx = rt->topk_idx;
  a.pair_slot = rt->pair_slot;
  a.pair_gate = rt->pair_gate;
  a.pair_dgate = pair_dgate;
  a.topk_dgate = topk_dgate;
  a.ld_dout = ld_dout;
  a.ld_rows = ld_rows;
  a.ld_drows = ld_drows;
  ProfScope ps(s, "unpermute_bwd");
  switch (type) {
    case MOE_BF16: MOE_TRY_CUDA(launch_unpermute_bwd<__nv_bfloat16>(a, dout, rows, drows, s)); break;
    case MOE_F16: MOE_TRY_CUDA(launch_unpermute_bwd<__half>(a, dout, rows, drows, s)); break;
    default: MOE_TRY_CUDA(launch_unpermute_bwd<float>(a, dout, rows, drows, s));
  }
  return MOE_OK;
}

}  // extern "C"
