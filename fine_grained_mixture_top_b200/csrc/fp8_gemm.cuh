// Matrix products of E4M3 codes with one fp32 scale per block of 128 along the
// summed dimension:
//
//   C[m, n] = sum_b sA[b, m] sB[.] (sum_{k in block b} A[m, k] B[n, k])
//
// A has a scale per row and block; B one per 128 x 128 block (weights), or one
// per row and block like A (BROWS: the weight gradient, whose operands are both
// quantized along the tokens).  The tensor core sums one block at a time into
// a TMEM slot; the epilogue warps read the slot, multiply by the block's scales
// and add to fp32 accumulators that stay in their registers for the whole tile.
// So no more than 128 products are ever summed in the tensor core, whose fp8
// sums hold fewer bits than fp32, and C is rounded once, to bf16.
//
// Two kernels: tiles of 256 x 256 on pairs of CTAs, and tiles of 128 columns with
// the operands exchanged where there are few rows.  All waits are bounded
// (mbar_wait, mbar_wait_cl).
#pragma once
#include <cuda.h>

#include "ptx.cuh"

namespace moe {

enum Fp8Mode : int { FP8_DENSE = 0, FP8_GROUPED = 1, FP8_DW = 2 };

struct Fp8Params {
  CUtensorMap tmA, tmB;  // [planes, rows, K] bytes, boxes of 128 rows x 128
  CUtensorMap tmC;       // [planes, rows, N] bf16, boxes of 32 rows x 64
  const float* sA;       // [K / 128, ldsA]
  const float* sB;       // BROWS: [K / 128, ldsB]; else [planes, nb, kb]
  int64_t ldsA, ldsB, ldc;
  __nv_bfloat16* C;
  const int* offsets;  // [E + 1] first row (GROUPED) or k (DW) of each expert, multiples of 128
  int E, M, N, nb, kb;     // nb, kb: 128-blocks of N and of the summed dimension
  int mode;
  int mt, nt;              // tiles of M (not GROUPED: from offsets) and N
  int tok_boxes, split;    // few rows: 32s of tokens per tile, CTAs that share a tile
  DevStatus st;
};

constexpr int kFp8Bk = 128;                // summed elements (bytes) per stage
constexpr int kFp8Box = 128 * kFp8Bk;      // one operand box: 128 rows x 128 bytes
constexpr int kFp8Group = 16;              // M tiles side by side in the tile order

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tmap), "r"(src),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
// D[tmem] (+)= A * B, E4M3 operands in shared memory, fp32 D.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor for kind::f8f6f4, E4M3 A and B (K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_f8(int N, int M) {
  return (1u << 4)                      // D format f32
         | (0u << 7) | (0u << 10)       // A, B format E4M3
         | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// 16-byte chunk `c` of 128-byte line `line` under the 128-byte swizzle
__device__ __forceinline__ uint32_t fp8_sw128(int line, int c) { return (uint32_t)(line * 128 + ((c ^ (line & 7)) << 4)); }

// Wait for the TMEM loads issued so far, tied to the registers of two of them,
// so that no use of these can be moved in front of the wait.
__device__ __forceinline__ void tc_wait_ld_pair(uint32_t (&a)[32], uint32_t (&b)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(a[16]), "+r"(a[17]), "+r"(a[18]), "+r"(a[19]), "+r"(a[20]), "+r"(a[21]), "+r"(a[22]), "+r"(a[23]),
                 "+r"(a[24]), "+r"(a[25]), "+r"(a[26]), "+r"(a[27]), "+r"(a[28]), "+r"(a[29]), "+r"(a[30]), "+r"(a[31])
               :
               : "memory");
  asm volatile(""
               : "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]),
                 "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15]),
                 "+r"(b[16]), "+r"(b[17]), "+r"(b[18]), "+r"(b[19]), "+r"(b[20]), "+r"(b[21]), "+r"(b[22]), "+r"(b[23]),
                 "+r"(b[24]), "+r"(b[25]), "+r"(b[26]), "+r"(b[27]), "+r"(b[28]), "+r"(b[29]), "+r"(b[30]), "+r"(b[31])
               :
               : "memory");
}

// acc += 32 columns of a block's sums times the scales.  BROWS, with its product
// per value besides the FMA, computes two values per instruction (weight gradient
// of 131072 rows over 128 experts, 1536 x 512: 180 us, one at a time 186); for the
// FMA alone the moves into register pairs cost more than that saves (65536 rows x
// 2048 x 2048 over 16 experts: 335 us one at a time, 355 in pairs).
__device__ __forceinline__ uint64_t pack2f(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
template <bool BROWS>
__device__ __forceinline__ void add_columns(float* acc, const uint32_t (&v)[32], float s, const float* cols) {
  if constexpr (!BROWS) {
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = fmaf(__uint_as_float(v[j]), s, acc[j]);
  } else {
    const uint64_t s2 = pack2f(s, s);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint64_t w = reinterpret_cast<const uint64_t*>(cols)[j];
      const uint64_t x = pack2f(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
      uint64_t f, a = pack2f(acc[2 * j], acc[2 * j + 1]);
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(f) : "l"(w), "l"(s2));
      asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(x), "l"(f));
      asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[2 * j]), "=f"(acc[2 * j + 1]) : "l"(a));
    }
  }
}
// One block's sums: acc += TMEM slot (128 columns of this thread's row) times
// the scales; s: the row's scale (!BROWS: times the block's), cols: shared
// memory with the 128 column scales (BROWS).  Beside running MMAs a TMEM load
// takes some 250 clocks whatever its width, and a wait is for all loads in
// flight, so the slot comes in two rounds of two 32-column loads.  mid() runs
// under the second round; done() is called once the slot has been read.
template <bool BROWS, typename Mid, typename Done>
__device__ __forceinline__ void add_block(float (&acc)[128], uint32_t taddr, float s, const float* cols, Mid mid,
                                          Done done) {
  uint32_t v0[32], v1[32];
  tmem_ld32(taddr, v0);
  tmem_ld32(taddr + 32, v1);
  tc_wait_ld_pair(v0, v1);
  add_columns<BROWS>(acc, v0, s, cols);
  tmem_ld32(taddr + 64, v0);
  add_columns<BROWS>(acc + 32, v1, s, cols + 32);
  tmem_ld32(taddr + 96, v1);
  mid();
  tc_wait_ld_pair(v0, v1);
  done();
  add_columns<BROWS>(acc + 64, v0, s, cols + 64);
  add_columns<BROWS>(acc + 96, v1, s, cols + 96);
}

// A load that is issued where it is written (the compiler would move it down to
// its use, behind a barrier wait, and expose its latency).
__device__ __forceinline__ float load_now(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
// The scales an epilogue thread needs, loaded one block ahead: its row's, and
// the block's (!BROWS) or this lane's four of the 128 columns' (BROWS).  The
// pointers step from block to block.  (Fetched six blocks ahead through shared
// memory, by the warp itself or by one of its own with barriers, they cost as
// much or more: it is not their latency that counts, some 20 ns of a block's 615.)
template <bool BROWS>
struct BlockScales {
  const float *a, *b;
  float sa, sb, col[BROWS ? 4 : 1];
  // e, k0, m, n: the tile's expert and first k, this thread's row, this half's first column
  __device__ __forceinline__ void start(const Fp8Params& p, int e, int k0, int m, int n) {
    const int kb0 = k0 / kFp8Bk;
    a = p.sA + (int64_t)kb0 * p.ldsA + min(m, p.M - 1);
    b = BROWS ? p.sB + (int64_t)kb0 * p.ldsB + n + (threadIdx.x & 31)
              : p.sB + ((int64_t)(p.mode == FP8_GROUPED ? e : 0) * p.nb + min(n / 128, p.nb - 1)) * p.kb;
  }
  // BROWS: columns from this half's first one to the last
  __device__ __forceinline__ void load(int64_t step_a, int64_t step_b, int left) {
    sa = load_now(a);
    a += step_a;
    if constexpr (BROWS) {
      left -= (int)(threadIdx.x & 31);
#pragma unroll
      for (int j = 0; j < 4; ++j) col[j] = 32 * j < left ? load_now(b + 32 * j) : 0.f;
    } else {
      sb = load_now(b);
    }
    b += step_b;
  }
  // the factor of the loaded block; BROWS: the column scales go to `cols`.  The two
  // buffers take turns: the lanes' last reads of this one lie before the slot's
  // first TMEM load, where the warp meets (sync.aligned).  (A warp barrier of its
  // own, or a third buffer, costs registers: 215 and 208 us where this takes 211
  // and 204, in turn, for the weight gradient named above.)
  __device__ __forceinline__ float take(float* cols) {
    if constexpr (BROWS) {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int j = 0; j < 4; ++j) cols[lane + 32 * j] = col[j];
      __syncwarp();
      return sa;
    }
    return sa * sb;
  }
};

// This thread's row of 128 columns from n0 on, rounded to bf16, into C: 64
// columns at a time through this warp's two staging buffers at stg (a box is 32
// rows x 128 bytes).  Nothing is staged before the tensor stores of the tile
// before have left both buffers; a box past the last column is not staged.
__device__ __forceinline__ void store_row(const Fp8Params& p, const float (&acc)[128], uint32_t stg, int plane,
                                          int row0, int n0) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int n = n0 + 64 * x;
    if (n >= p.N) continue;
    if (n + 64 > p.N && p.N % 8 != 0) {
      // a tensor store is clipped to whole 16-byte chunks: the box with a
      // ragged last chunk goes element by element
      const int r = row0 + lane;
      if (r < p.M) {
        __nv_bfloat16* c = p.C + ((int64_t)plane * p.M + r) * p.ldc + n;
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (n + j < p.N) c[j] = __float2bfloat16_rn(acc[x * 64 + j]);
      }
      continue;
    }
    const uint32_t buf = stg + x * 4096;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float* a = acc + x * 64 + j * 8;
      st_shared_v4(buf + fp8_sw128(lane, j), make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                        pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7])));
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && row0 < p.M) {
      tma_store_3d(&p.tmC, buf, n, row0, plane);
      bulk_commit();
    }
  }
}

// True in one lane of the (converged) warp, the same one each time.  Unlike a
// test of the lane number this keeps the guarded code warp-uniform for the
// compiler: descriptors and addresses stay in uniform registers, where the
// tensor and TMA instructions want them (77 clocks per MMA issued otherwise,
// which paced the whole kernel: 334 against 290 us for 65536 rows x 2048 x 2048
// over 16 experts).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// After a wait has run out no barrier tells when the copies and MMAs already
// issued are done.  They need microseconds: a CTA that has given up stays for
// 2^18 clocks, some 140 us, before it frees its TMEM and leaves.
__device__ __forceinline__ void settle(const volatile int* abort_flag) {
  if (*abort_flag == 0) return;
  const long long t0 = clock64();
  while (clock64() - t0 < (1 << 18)) __nanosleep(1000);
}

// ----------------------------------------------------------------- few rows
// The product with its operands exchanged, for few rows of A: the weights are
// the MMA's 128 rows and up to 128 rows of A ("tokens", 32 at a time) its
// columns, so that a tile of few tokens costs few columns in the tensor core, in
// TMEM and in the epilogue, and reads the weights at the rate of memory.
//
// Dense products only: tiles of 128 columns of C x 32 tok_boxes tokens, at most
// one per SM.  Where there are fewer than half as many, a cluster of `split` CTAs shares one, each
// summing its share of the blocks; their fp32 sums meet in distributed shared
// memory and are added in rank order.
//
// Warps: 0 TMA loads, 1 TMEM allocation and MMA issue, 2 .. 9 the epilogue (one
// column of C per thread, two warps per TMEM lane quarter, each with every other
// 32 tokens in its registers); four 128-column TMEM slots.
// The result leaves through shared memory ([token][column], so that global
// stores are coalesced).
struct Fp8SmallShape {
  static constexpr int kEpi = 8;
  static constexpr int kThreads = 32 * (2 + kEpi);
  static constexpr int kMaxReg = 168;  // three warps on a sub-partition's 16384 registers
  static constexpr int kSlots = 4;
  static constexpr int kMaxStages = 10;
  static constexpr int kScaleWarp = 2 * 64 * 4;    // two blocks' factors of a warp's tokens
  static constexpr int kTokBox = 32 * kFp8Bk;      // 32 tokens x 128 bytes
  static constexpr int kSumBox = 32 * 128 * 4;     // 32 tokens x 128 columns fp32
  static constexpr int kSide = kEpi * kScaleWarp + 1024;
  static __host__ __device__ constexpr int stage_bytes(int boxes) { return kFp8Box + boxes * kTokBox; }
  static __host__ __device__ constexpr int stages(int boxes) {
    const int n = (227 * 1024 - 1024 - kSide - boxes * kSumBox) / stage_bytes(boxes);
    return n < kMaxStages ? n : kMaxStages;
  }
  static __host__ __device__ constexpr int smem(int boxes) {
    return stages(boxes) * stage_bytes(boxes) + boxes * kSumBox + kSide + 1024;
  }
};
static_assert(Fp8SmallShape::stages(4) >= 4 && Fp8SmallShape::smem(4) <= 227 * 1024, "operand ring");

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// acc += 32 columns of a block's sums times their factors in shared memory.
__device__ __forceinline__ void add_scaled(float* acc, const uint32_t (&v)[32], const float* factors) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 w = reinterpret_cast<const float4*>(factors)[j];
    acc[4 * j] = fmaf(__uint_as_float(v[4 * j]), w.x, acc[4 * j]);
    acc[4 * j + 1] = fmaf(__uint_as_float(v[4 * j + 1]), w.y, acc[4 * j + 1]);
    acc[4 * j + 2] = fmaf(__uint_as_float(v[4 * j + 2]), w.z, acc[4 * j + 2]);
    acc[4 * j + 3] = fmaf(__uint_as_float(v[4 * j + 3]), w.w, acc[4 * j + 3]);
  }
}

struct Fp8SmallTile {
  int m0, n0, rows;  // first token, first column, tokens
};
__device__ __forceinline__ Fp8SmallTile fp8_small_tile(const Fp8Params& p, int id) {
  Fp8SmallTile t;
  const int m = id / p.nt;
  t.n0 = (id - m * p.nt) * 128;
  t.m0 = m * 32 * p.tok_boxes;
  t.rows = min(p.M - t.m0, 32 * p.tok_boxes);
  return t;
}

// The tile's sums (from RANKS CTAs' shared memory at address `at` of each,
// [token][128]) rounded and stored by all threads of each of the CTAs; a
// thread takes four columns of a token, and has all loads of several such pieces
// in flight (one after the other they cost 4 us of a 7 us product).
template <int RANKS>
__device__ __forceinline__ void fp8_small_store(const Fp8Params& p, const Fp8SmallTile& t, uint32_t at, int rank,
                                                int tid) {
  constexpr int U = RANKS >= 8 ? 1 : (RANKS >= 4 ? 2 : 4);
  const int n_pieces = t.rows * 32, stride = RANKS * Fp8SmallShape::kThreads;
  uint32_t from[RANKS];
#pragma unroll
  for (int r = 0; r < RANKS; ++r) from[r] = mapa_shared(at, r);
  for (int i0 = rank * Fp8SmallShape::kThreads + tid; i0 < n_pieces; i0 += U * stride) {
    float4 x[U][RANKS];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < RANKS; ++r)
        x[u][r] = ld_cluster_v4(from[r] + 16 * (uint32_t)min(i0 + u * stride, n_pieces - 1));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * stride;
      if (i >= n_pieces) break;
      float4 v = x[u][0];
#pragma unroll
      for (int r = 1; r < RANKS; ++r) v.x += x[u][r].x, v.y += x[u][r].y, v.z += x[u][r].z, v.w += x[u][r].w;
      const int m = i >> 5, n = t.n0 + 4 * (i & 31);
      __nv_bfloat16* c = p.C + (int64_t)(t.m0 + m) * p.ldc + n;
      if (n + 4 <= p.N) {
        *reinterpret_cast<uint2*>(c) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      } else {
        if (n < p.N) c[0] = __float2bfloat16_rn(v.x);
        if (n + 1 < p.N) c[1] = __float2bfloat16_rn(v.y);
        if (n + 2 < p.N) c[2] = __float2bfloat16_rn(v.z);
      }
    }
  }
}

// tmA: weights (boxes of 128 rows), tmB: tokens (boxes of 32 tok_boxes rows).
__global__ void __maxnreg__((Fp8SmallShape::kMaxReg)) fp8_gemm_small_kernel(const __grid_constant__ Fp8Params p) {
  using SH = Fp8SmallShape;
  constexpr int kTmemCols = 512;
  const int stage = SH::stage_bytes(p.tok_boxes), S = SH::stages(p.tok_boxes);

  extern __shared__ uint8_t smem_raw[];
  if (dynamic_smem_bytes() < (uint32_t)SH::smem(p.tok_boxes)) {  // all CTAs of a cluster leave alike
    if (threadIdx.x == 0) raise_status(p.st, ST_DEVICE_CHECK, 0x380);
    return;
  }
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int sum_offset = S * stage;
  const int scale_offset = sum_offset + p.tok_boxes * SH::kSumBox;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + scale_offset + SH::kEpi * SH::kScaleWarp);
  uint64_t* full = bars;
  uint64_t* empty = bars + SH::kMaxStages;
  uint64_t* slot_full = bars + 2 * SH::kMaxStages;
  uint64_t* slot_empty = slot_full + SH::kSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(slot_empty + SH::kSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot_empty + SH::kSlots + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = p.split;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < SH::kSlots; ++b) {
      mbar_init(&slot_full[b], 1);
      mbar_init(&slot_empty[b], SH::kEpi);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  const Fp8SmallTile t = fp8_small_tile(p, (int)blockIdx.x / split);
  // this CTA's share of the blocks
  const int kb0 = (int)((int64_t)p.kb * rank / split), nkb = (int)((int64_t)p.kb * (rank + 1) / split) - kb0;

  if (warp == 0) {
    int s = 0;
    uint32_t phase = 1;
    for (int kb = kb0; kb < kb0 + nkb; ++kb) {
      if (!mbar_wait(smem_u32(&empty[s]), phase, abort_flag, p.st, 0x381)) break;
      if (elect_one()) {
        const uint32_t bar = smem_u32(&full[s]), dst = base + s * stage;
        mbar_arrive_expect_tx(bar, (uint32_t)stage);
        tma_load_3d(dst, &p.tmA, bar, kb * kFp8Bk, t.n0, 0);
        tma_load_3d(dst + kFp8Box, &p.tmB, bar, kb * kFp8Bk, t.m0, 0);
      }
      __syncwarp();
      if (++s == S) s = 0, phase ^= 1;
    }
  } else if (warp == 1) {
    int s = 0;
    uint32_t phase = 0;
    const uint32_t idesc = idesc_f8(32 * p.tok_boxes, 128);
    for (int kb = 0; kb < nkb; ++kb) {
      const int b = kb % SH::kSlots;
      if (!mbar_wait(smem_u32(&slot_empty[b]), ((kb / SH::kSlots) & 1) ^ 1, abort_flag, p.st, 0x383) ||
          !mbar_wait(smem_u32(&full[s]), phase, abort_flag, p.st, 0x382))
        break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t a_s = base + s * stage;
        const uint64_t ad = smem_desc_sw128(a_s, 16, 1024), bd = smem_desc_sw128(a_s + kFp8Box, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kFp8Bk / 32; ++kk)
          tc_mma_f8(tmem + b * 128, ad + 2 * kk, bd + 2 * kk, idesc, kk > 0 ? 1u : 0u);
        tc_commit(smem_u32(&slot_full[b]));
        tc_commit(smem_u32(&empty[s]));
      }
      __syncwarp();
      if (++s == S) s = 0, phase ^= 1;
    }
  } else {
    const int ew = warp - 2;
    const int g = ew >> 2;   // its tokens: the 32s g and g + 2
    const int q = warp & 3;  // TMEM lane quarter: columns n0 + 32 q ..
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16) + 32 * g;
    float* cs = reinterpret_cast<float*>(smem + scale_offset + ew * SH::kScaleWarp);
    float* sums = reinterpret_cast<float*>(smem + sum_offset);
    const float* sb_p = p.sB + (int64_t)(t.n0 / 128) * p.kb + kb0;
    const float* sa_p = p.sA + (int64_t)kb0 * p.ldsA + t.m0 + 32 * g + lane;
    const int left = p.M - (t.m0 + 32 * g + lane);
    // a block's factors: the weights' block scale times this lane's tokens' scales
    float sb = 0.f, sa0 = 0.f, sa1 = 0.f;
    auto load_scales = [&] {
      sb = load_now(sb_p);
      sa0 = left > 0 ? load_now(sa_p) : 0.f;
      sa1 = left > 64 ? load_now(sa_p + 64) : 0.f;
      ++sb_p;
      sa_p += p.ldsA;
    };
    auto take_scales = [&](int kb) {
      float* f = cs + (kb & 1) * 64;
      f[lane] = sa0 * sb;
      f[32 + lane] = sa1 * sb;
      __syncwarp();
    };
    float acc[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0.f;
    load_scales();
    take_scales(0);
    if (nkb > 1) load_scales();
    for (int kb = 0; kb < nkb; ++kb) {
      const int b = kb % SH::kSlots;
      if (!mbar_wait(smem_u32(&slot_full[b]), (kb / SH::kSlots) & 1, abort_flag, p.st, 0x384)) break;
      tc_fence_after();
      uint32_t v0[32], v1[32];
      // (columns past the tile's tokens hold leftovers, whose sums are not stored)
      tmem_ld32(tq + b * 128, v0);
      tmem_ld32(tq + b * 128 + 64, v1);
      if (kb + 1 < nkb) take_scales(kb + 1);
      if (kb + 2 < nkb) load_scales();
      tc_wait_ld_pair(v0, v1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&slot_empty[b]));
      const float* f = cs + (kb & 1) * 64;
      add_scaled(acc, v0, f);
      add_scaled(acc + 32, v1, f + 32);
    }
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const int m = (i < 32 ? 32 * g : 64 + 32 * g - 32) + i;
      if (m < t.rows) sums[m * 128 + q * 32 + lane] = acc[i];
    }
  }

  settle(abort_flag);
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync();
  const uint32_t at = base + sum_offset;
  if (split == 1) fp8_small_store<1>(p, t, at, 0, threadIdx.x);
  else if (split == 2) fp8_small_store<2>(p, t, at, rank, threadIdx.x);
  else if (split == 4) fp8_small_store<4>(p, t, at, rank, threadIdx.x);
  else fp8_small_store<8>(p, t, at, rank, threadIdx.x);
  if (split > 1) cluster_sync();  // the other CTAs have read this one's sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ----------------------------------------------------------------- CTA pairs
// The same product on pairs of CTAs (cta_group::2): tiles of 256 rows x 256
// columns.  Each CTA loads its own 128 rows of A and half of B's columns, 32 KB
// per block where two single-CTA tiles of the same area load 48 KB each, and
// holds its 128 rows of the result: 128 columns in each of two epilogue
// warpgroups' registers.  TMEM holds two 256-column slots.
//
// What paces it, per block and CTA in short runs: 615 ns with everything; about
// 450 without the epilogue's arithmetic and the MMAs (32 KB of operands from L2:
// an SM fills its shared memory with 73 GB/s), 470 without the operand
// loads and that arithmetic (the MMAs, 512 clocks at the tensor core's peak), 510
// without the MMAs.  The three overlap through four operand stages and two slots.
// In long runs the power cap lowers the clock, and a block takes 735 ns.
//
// GROUPED: a tile is two consecutive 128-row tiles of one expert; where an
// expert's last tile is alone, the second CTA loads no A, lets its accumulator
// pass and stores nothing.  The M tiles of each expert in pairs are counted once
// per launch into shared memory (pair_start), and a tile finds its expert there.
//
// Warps: 0 TMA loads, 1 MMA issue (first CTA), 2 TMEM allocation, 3 idle (one
// warpgroup, which gives up most of its registers), 4 .. 11 the epilogue.
// Barriers: full[s] and slot_empty[b] are the first CTA's (both CTAs' loads and
// epilogues arrive there); empty[s] and slot_full[b] are each CTA's own, the
// MMA's commit arriving at both.  All four are signalled across the pair, so
// every wait acquires at cluster scope.
struct Fp8PairShape {
  static constexpr int kStage = 2 * kFp8Box;  // per CTA
  static constexpr int kSlots = 2;            // 256-column TMEM slots
  static constexpr int kEpi = 8;
  static constexpr int kStoreWarp = 8192;
  static constexpr int kScaleWarp = 2 * 128 * 4;  // BROWS: two blocks' column scales per warp
  static constexpr int kList = 1024 * 4;      // one entry per expert
  static constexpr int kStages = 4;
  static constexpr int kStoreOffset = kStages * kStage;
  static constexpr int kScaleOffset = kStoreOffset + kEpi * kStoreWarp;
  static constexpr int kListOffset = kScaleOffset + kEpi * kScaleWarp;
  static constexpr int kBarOffset = kListOffset + kList;
  static constexpr int kSmem = kBarOffset + 1024 + 1024;
  static constexpr int kThreads = 384;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// Arrive once on the barrier at this offset in both CTAs of the pair when the
// pair MMAs issued so far by this thread are done.
__device__ __forceinline__ void tc_commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct Fp8PairTile {
  int e, m0, n0, k0, nkb;
  bool both;  // the second CTA's rows exist
};
// The pair's tile of round r.  DW deals its tiles, experts by falling row count,
// back and forth, so that every pair gets much the same work (in expert order
// and always forward, the weight gradient of 131072 rows over 128 experts of
// uneven load took 304 us instead of 185).
__device__ __forceinline__ int fp8_turn(const Fp8Params& p, int r, int pair, int npairs) {
  return r * npairs + (p.mode == FP8_DW && (r & 1) ? npairs - 1 - pair : pair);
}
// Tile `id` (all lanes of a warp alike); list: in shared memory, pair_start
// (GROUPED) or the experts in the order of their tiles (DW).
__device__ __forceinline__ Fp8PairTile fp8_pair_tile(const Fp8Params& p, int id, int mt, const int* list) {
  Fp8PairTile t;
  int plane = 0;
  if (p.mode == FP8_DW) {
    plane = id / (mt * p.nt);
    id -= plane * (mt * p.nt);
    if (p.offsets) plane = list[plane];
  }
  constexpr int kGroup = kFp8Group / 2;
  const int per = kGroup * p.nt;
  const int g = id / per;
  const int rows = min(kGroup, mt - g * kGroup);
  const int in = id - g * per;
  const int n = in / rows;
  const int m = g * kGroup + in - n * rows;
  t.m0 = m * 256;
  t.n0 = n * 256;
  t.k0 = 0;
  t.nkb = p.kb;
  t.e = 0;
  t.both = t.m0 + 128 < p.M;
  if (p.mode == FP8_GROUPED) {
    // the last expert that starts at or before pair m: first among every 32nd, then inside that run
    const int lane = threadIdx.x & 31;
    const int far = 32 * lane < p.E ? list[32 * lane] : 0x7fffffff;
    const int run = 31 - __clz(__ballot_sync(0xffffffffu, far <= m));
    const int near = 32 * run + lane < p.E ? list[32 * run + lane] : 0x7fffffff;
    t.e = 32 * run + 31 - __clz(__ballot_sync(0xffffffffu, near <= m));
    const int row = __ldg(p.offsets + t.e) + 256 * (m - list[t.e]);
    t.m0 = row;
    t.both = row + 128 < __ldg(p.offsets + t.e + 1);
  }
  if (p.mode == FP8_DW) {
    t.e = plane;
    if (p.offsets) {
      t.k0 = __ldg(p.offsets + plane);
      t.nkb = (__ldg(p.offsets + plane + 1) - t.k0) / kFp8Bk;
    }
  }
  return t;
}

template <bool BROWS>
__global__ void __launch_bounds__(Fp8PairShape::kThreads, 1) __cluster_dims__(2, 1, 1)
    fp8_gemm_pair_kernel(const __grid_constant__ Fp8Params p) {
  using SH = Fp8PairShape;
  constexpr int S = SH::kStages;
  constexpr uint32_t kIdesc = idesc_f8(256, 256);
  constexpr int kTmemCols = 512;

  extern __shared__ uint8_t smem_raw[];
  if (dynamic_smem_bytes() < (uint32_t)SH::kSmem) {  // both CTAs of the pair leave alike
    if (threadIdx.x == 0) raise_status(p.st, ST_DEVICE_CHECK, 0x388);
    return;
  }
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SH::kBarOffset);
  uint64_t* full = bars;
  uint64_t* empty = bars + 8;
  uint64_t* slot_full = bars + 16;
  uint64_t* slot_empty = bars + 18;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 21);
  int* mt_slot = reinterpret_cast<int*>(bars + 22);
  int* list = reinterpret_cast<int*>(smem + SH::kListOffset);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool lead = rank == 0;
  auto lead_bar = [&](uint64_t* b) -> uint32_t { return mapa_shared(smem_u32(b), 0); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < SH::kSlots; ++b) {
      mbar_init(&slot_full[b], 1);
      mbar_init(&slot_empty[b], 2 * SH::kEpi);  // the epilogue warps of both CTAs
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
    tma_prefetch_desc(&p.tmC);
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  pdl_wait();
  if (p.mode == FP8_GROUPED && warp == 3) {  // pairs of M tiles before each expert
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int n = e < p.E ? ((__ldg(p.offsets + e + 1) - __ldg(p.offsets + e)) / 128 + 1) / 2 : 0;
      const int own = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n += y;
      }
      if (e < p.E) list[e] = before + n - own;
      before += __shfl_sync(0xffffffffu, n, 31);
    }
    if (lane == 0) *mt_slot = before;
  }
  if (p.mode == FP8_DW && p.offsets) {
    // experts by falling row count (ties: the lower one first), the same list in
    // every CTA: a bitonic sort of count << 10 | 1023 - expert
    int size = 32;
    while (size < p.E) size <<= 1;
    for (int e = threadIdx.x; e < size; e += SH::kThreads)
      list[e] = e < p.E ? min((__ldg(p.offsets + e + 1) - __ldg(p.offsets + e)) / kFp8Bk, (1 << 21) - 1) << 10 | (1023 - e)
                        : -1;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int i = threadIdx.x; i < size / 2; i += SH::kThreads) {
          const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
          const int a = list[lo], b = list[hi];
          if ((a < b) == ((lo & k) == 0)) list[lo] = b, list[hi] = a;
        }
        __syncthreads();
      }
    for (int e = threadIdx.x; e < p.E; e += SH::kThreads) list[e] = 1023 - (list[e] & 1023);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers initialised before any remote arrive or load
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int mt = p.mode == FP8_GROUPED ? *mt_slot : p.mt;
  const int tiles = mt * p.nt * (p.mode == FP8_DW ? p.E : 1);
  const int pair = (int)blockIdx.x >> 1, npairs = (int)gridDim.x >> 1;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      int it = 0;
      bool ok = true;
      for (int r = 0; ok; ++r) {
        const int id = fp8_turn(p, r, pair, npairs);
        if (id >= tiles) break;
        const Fp8PairTile t = fp8_pair_tile(p, id, mt, list);
        const int eb = p.mode == FP8_GROUPED ? t.e : 0;
        const bool a_too = lead || t.both;
        const uint32_t bytes = 2u * SH::kStage - (t.both ? 0u : (uint32_t)kFp8Box);
        const int m = t.m0 + 128 * (int)rank, n = t.n0 + 128 * (int)rank;
        for (int kb = 0; kb < t.nkb; ++kb, ++it) {
          const int s = it % S;
          if (!mbar_wait_cl(smem_u32(&empty[s]), ((it / S) & 1) ^ 1, abort_flag, p.st, 0x389)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            const uint32_t bar = lead_bar(&full[s]), dst = base + s * SH::kStage;
            if (lead) mbar_arrive_expect_tx(smem_u32(&full[s]), bytes);
            const int k = t.k0 + kb * kFp8Bk;
            if (a_too) tma_load_3d_pair(dst, &p.tmA, bar, k, m, 0);
            tma_load_3d_pair(dst + kFp8Box, &p.tmB, bar, k, n, eb);
          }
          __syncwarp();
        }
      }
    } else if (warp == 1 && lead) {
      int it = 0;
      bool ok = true;
      for (int r = 0; ok; ++r) {
        const int id = fp8_turn(p, r, pair, npairs);
        if (id >= tiles) break;
        const Fp8PairTile t = fp8_pair_tile(p, id, mt, list);
        for (int kb = 0; kb < t.nkb && ok; ++kb, ++it) {
          const int s = it % S;
          if (!mbar_wait_cl(smem_u32(&full[s]), (it / S) & 1, abort_flag, p.st, 0x38a)) {
            ok = false;
            break;
          }
          const int b = it % SH::kSlots;
          if (!mbar_wait_cl(smem_u32(&slot_empty[b]), ((it / SH::kSlots) & 1) ^ 1, abort_flag, p.st, 0x38b)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t a_s = base + s * SH::kStage;
            const uint64_t ad = smem_desc_sw128(a_s, 16, 1024), bd = smem_desc_sw128(a_s + kFp8Box, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < kFp8Bk / 32; ++kk)  // 32 bytes further along k: 2 in the descriptors' 16-byte units
              tc_mma_f8_pair(tmem + b * 256, ad + 2 * kk, bd + 2 * kk, kIdesc, kk > 0 ? 1u : 0u);
            tc_commit_both(smem_u32(&slot_full[b]));
            tc_commit_both(smem_u32(&empty[s]));
          }
          __syncwarp();
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int ew = warp - 4;
    const int h = ew >> 2;
    const int q = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t stg = base + SH::kStoreOffset + ew * SH::kStoreWarp;
    float* cs = reinterpret_cast<float*>(smem + SH::kScaleOffset + ew * SH::kScaleWarp);
    int it = 0;
    bool ok = true;
    auto wait_slot = [&](int i) {
      const int b = i % SH::kSlots;
      if (!mbar_wait_cl(smem_u32(&slot_full[b]), (i / SH::kSlots) & 1, abort_flag, p.st, 0x38c)) return false;
      tc_fence_after();
      return true;
    };
    auto release_slot = [&](int i) {  // read to the end: the next MMAs may have it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(lead_bar(&slot_empty[i % SH::kSlots]));
    };
    Fp8PairTile t = {};
    BlockScales<BROWS> sc;
    auto load_scales = [&] { sc.load(p.ldsA, BROWS ? p.ldsB : 1, p.N - t.n0 - 128 * h); };
    auto take_tile = [&](int id) {  // its first scales travel while the tile before it is stored
      t = fp8_pair_tile(p, id, mt, list);
      sc.start(p, t.e, t.k0, t.m0 + 128 * (int)rank + q * 32 + lane, t.n0 + 128 * h);
      if (t.nkb > 0) load_scales();
    };
    if (pair < tiles) take_tile(pair);
    for (int r = 0; ok && fp8_turn(p, r, pair, npairs) < tiles; ++r) {
      const int row0 = t.m0 + 128 * (int)rank + q * 32;
      const int n = t.n0 + 128 * h;
      const int plane = p.mode == FP8_DW ? t.e : 0;
      const bool mine = lead || t.both;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      if (mine) {
        float s = 0.f;
        if (t.nkb > 0) s = sc.take(cs);
        if (t.nkb > 1) load_scales();
        for (int kb = 0; kb < t.nkb; ++kb, ++it) {
          ok = wait_slot(it);
          if (!ok) break;
          const float s_now = s;
          add_block<BROWS>(
              acc, tq + (it % SH::kSlots) * 256 + h * 128, s_now, cs + (kb & 1) * 128,
              [&] {
                if (kb + 1 < t.nkb) s = sc.take(cs + (~kb & 1) * 128);
                if (kb + 2 < t.nkb) load_scales();
              },
              [&] { release_slot(it); });
        }
      } else {  // no rows here: only let the slots pass
        for (int kb = 0; kb < t.nkb && ok; ++kb, ++it) {
          ok = wait_slot(it);
          if (ok) release_slot(it);
        }
      }
      if (!ok) break;
      const int then = fp8_turn(p, r + 1, pair, npairs);
      if (then < tiles) take_tile(then);
      if (mine) store_row(p, acc, stg, plane, row0, n);
    }
    if (lane == 0) bulk_wait_all();
  }

  settle(abort_flag);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its pair may still arrive on its barriers
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace moe
