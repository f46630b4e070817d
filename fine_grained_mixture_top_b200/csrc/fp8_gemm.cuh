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
// A tile is 128 rows x (128 HALVES) columns; each half has four warps (one row
// per thread) and, of the four 128-column TMEM slots, takes every HALVES-th, so
// that the MMAs run ahead of the epilogue by 4 / HALVES blocks.
//
// Warps: 0 TMA loads (one lane), 1 TMEM allocation and MMA issue, 2 .. 2 + 4
// HALVES the epilogue.  Barriers: full[s] / empty[s] per stage of the operand
// ring, slot_full[b] (MMA commit) / slot_empty[b] (four warps) per TMEM slot.
// All waits are bounded (mbar_wait).
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
  const int* offsets;      // [E + 1] first row (GROUPED) or k (DW) of each expert, multiples of 128
  const int* tile_expert;  // GROUPED: expert of each 128-row tile
  int E, M, N, nb, kb;     // nb, kb: 128-blocks of N and of the summed dimension
  int mode;
  int mt, nt;              // tiles of M (not GROUPED: from offsets) and N
  DevStatus st;
};

constexpr int kFp8Bk = 128;                // summed elements (bytes) per stage
constexpr int kFp8Box = 128 * kFp8Bk;      // one operand box: 128 rows x 128 bytes
constexpr int kFp8Slots = 4;               // 128-column TMEM slots
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

// Wait for the TMEM loads, tied to the registers of one of them, so that no use
// of these can be moved in front of the wait.
__device__ __forceinline__ void tc_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :
               : "memory");
}

template <int HALVES>
struct Fp8Shape {
  static constexpr int kStage = kFp8Box * (1 + HALVES);
  static constexpr int kEpi = 4 * HALVES;                    // epilogue warps
  static constexpr int kStoreWarp = HALVES == 1 ? 8192 : 4096;  // staging bytes per epilogue warp (64-column boxes)
  static constexpr int kScaleWarp = 2 * 128 * 4;             // BROWS: two blocks' column scales per warp
  static constexpr int kSide = kEpi * (kStoreWarp + kScaleWarp) + 1024;
  static constexpr int kStages = (227 * 1024 - 1024 - kSide) / kStage;
  static constexpr int kStoreOffset = kStages * kStage;
  static constexpr int kScaleOffset = kStoreOffset + kEpi * kStoreWarp;
  static constexpr int kBarOffset = kScaleOffset + kEpi * kScaleWarp;
  static constexpr int kSmem = kBarOffset + 1024 + 1024;     // + alignment of the base
  static constexpr int kThreads = 32 * (2 + kEpi);
  static_assert(kStages >= 4 && kSmem <= 227 * 1024, "operand ring");
};

struct Fp8Tile {
  int e, m0, n0, k0, nkb;
};
// Tile `id` of the launch: M tiles in groups of kFp8Group, inside a group M
// fastest, so that the tiles in flight share both operands in L2.
__device__ __forceinline__ Fp8Tile fp8_tile(const Fp8Params& p, int id, int mt, int bn) {
  Fp8Tile t;
  int plane = 0;
  if (p.mode == FP8_DW) {
    plane = id / (mt * p.nt);
    id -= plane * (mt * p.nt);
  }
  const int per = kFp8Group * p.nt;
  const int g = id / per;
  const int rows = min(kFp8Group, mt - g * kFp8Group);
  const int in = id - g * per;
  const int n = in / rows;
  const int m = g * kFp8Group + in - n * rows;
  t.m0 = m * 128;
  t.n0 = n * bn;
  t.k0 = 0;
  t.nkb = p.kb;
  t.e = 0;
  if (p.mode == FP8_GROUPED) t.e = __ldg(p.tile_expert + m);
  if (p.mode == FP8_DW) {
    t.e = plane;
    if (p.offsets) {
      t.k0 = __ldg(p.offsets + plane);
      t.nkb = (__ldg(p.offsets + plane + 1) - t.k0) / kFp8Bk;
    }
  }
  return t;
}

template <int HALVES, bool BROWS>
__global__ void __launch_bounds__(Fp8Shape<HALVES>::kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8Params p) {
  using SH = Fp8Shape<HALVES>;
  constexpr int S = SH::kStages;
  constexpr int kBn = 128 * HALVES;
  constexpr uint32_t kIdesc = idesc_f8(128, 128);
  constexpr int kTmemCols = 512;

  extern __shared__ uint8_t smem_raw[];
  if (dynamic_smem_bytes() < (uint32_t)SH::kSmem) {
    if (threadIdx.x == 0) raise_status(p.st, ST_DEVICE_CHECK, 0x380);
    return;
  }
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SH::kBarOffset);
  uint64_t* full = bars;
  uint64_t* empty = bars + 8;
  uint64_t* slot_full = bars + 16;
  uint64_t* slot_empty = bars + 20;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 24);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 25);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kFp8Slots; ++b) {
      mbar_init(&slot_full[b], 1);
      mbar_init(&slot_empty[b], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
    tma_prefetch_desc(&p.tmC);
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

  const int mt = p.mode == FP8_GROUPED ? __ldg(p.offsets + p.E) / 128 : p.mt;
  const int tiles = mt * p.nt * (p.mode == FP8_DW ? p.E : 1);

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x) {
        const Fp8Tile t = fp8_tile(p, id, mt, kBn);
        const int eb = p.mode == FP8_GROUPED ? t.e : 0;
        for (int kb = 0; kb < t.nkb; ++kb, ++it) {
          const int s = it % S;
          if (!mbar_wait(smem_u32(&empty[s]), ((it / S) & 1) ^ 1, abort_flag, p.st, 0x381)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&full[s]), dst = base + s * SH::kStage;
          const int k = t.k0 + kb * kFp8Bk;
          mbar_arrive_expect_tx(bar, SH::kStage);
          tma_load_3d(dst, &p.tmA, bar, k, t.m0, 0);
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(dst + (1 + h) * kFp8Box, &p.tmB, bar, k, t.n0 + 128 * h, eb);
        }
      }
    }
  } else if (warp == 1) {
    int it = 0;
    bool ok = true;
    for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x) {
      const Fp8Tile t = fp8_tile(p, id, mt, kBn);
      for (int kb = 0; kb < t.nkb && ok; ++kb, ++it) {
        const int s = it % S;
        if (!mbar_wait(smem_u32(&full[s]), (it / S) & 1, abort_flag, p.st, 0x382)) {
          ok = false;
          break;
        }
        const uint32_t a_s = base + s * SH::kStage;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          const int i = it * HALVES + h;
          const int b = i % kFp8Slots;
          if (!mbar_wait(smem_u32(&slot_empty[b]), ((i / kFp8Slots) & 1) ^ 1, abort_flag, p.st, 0x383)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t b_s = a_s + (1 + h) * kFp8Box;
#pragma unroll
            for (int kk = 0; kk < kFp8Bk / 32; ++kk)
              tc_mma_f8(tmem + b * 128, smem_desc_sw128(a_s + kk * 32, 16, 1024),
                        smem_desc_sw128(b_s + kk * 32, 16, 1024), kIdesc, kk > 0 ? 1u : 0u);
            tc_commit(smem_u32(&slot_full[b]));
            if (h == HALVES - 1) tc_commit(smem_u32(&empty[s]));
          }
          __syncwarp();
        }
      }
    }
  } else {
    const int ew = warp - 2;
    const int h = ew >> 2;    // column half
    const int q = warp & 3;   // TMEM lane quarter: rows 32 q ..
    const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t stg = base + SH::kStoreOffset + ew * SH::kStoreWarp;
    float* cs = reinterpret_cast<float*>(smem + SH::kScaleOffset + ew * SH::kScaleWarp);
    int it = 0;
    bool ok = true;
    for (int id = blockIdx.x; id < tiles && ok; id += gridDim.x) {
      const Fp8Tile t = fp8_tile(p, id, mt, kBn);
      const int m = t.m0 + q * 32 + lane;
      const int nh = t.n0 + 128 * h;  // first column of this half
      const int kb0 = t.k0 / kFp8Bk;
      const float* sa_p = p.sA + (int64_t)kb0 * p.ldsA + min(m, p.M - 1);
      const float* sb_p = BROWS ? p.sB + (int64_t)kb0 * p.ldsB
                                : p.sB + ((int64_t)(p.mode == FP8_GROUPED ? t.e : 0) * p.nb + min(nh / 128, p.nb - 1)) * p.kb;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      float sa = 0.f, sb = 0.f;
      float col[4];
      auto load_scales = [&](int kb) {
        sa = __ldg(sa_p + (int64_t)kb * p.ldsA);
        if constexpr (BROWS) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int n = nh + lane + 32 * j;
            col[j] = n < p.N ? __ldg(sb_p + (int64_t)kb * p.ldsB + n) : 0.f;
          }
        } else {
          sb = __ldg(sb_p + kb);
        }
      };
      if (t.nkb > 0) load_scales(0);
      for (int kb = 0; kb < t.nkb; ++kb, ++it) {
        const int i = it * HALVES + h;
        const int b = i % kFp8Slots;
        const float s = BROWS ? sa : sa * sb;
        float* cb = cs + (kb & 1) * 128;
        if constexpr (BROWS) {
#pragma unroll
          for (int j = 0; j < 4; ++j) cb[lane + 32 * j] = col[j];
          __syncwarp();
        }
        if (kb + 1 < t.nkb) load_scales(kb + 1);
        if (!mbar_wait(smem_u32(&slot_full[b]), (i / kFp8Slots) & 1, abort_flag, p.st, 0x384)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[2][32];
        tmem_ld32(tq + b * 128, v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tc_wait_ld32(v[c & 1]);
          if (c < 3) {
            tmem_ld32(tq + b * 128 + (c + 1) * 32, v[(c + 1) & 1]);
          } else {  // the slot has been read: the next block's MMAs may have it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&slot_empty[b]));
          }
          if constexpr (BROWS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 w = reinterpret_cast<const float4*>(cb)[c * 8 + j];
              const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int u = 0; u < 4; ++u)
                acc[c * 32 + 4 * j + u] =
                    fmaf(__uint_as_float(v[c & 1][4 * j + u]), s * ws[u], acc[c * 32 + 4 * j + u]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[c * 32 + j] = fmaf(__uint_as_float(v[c & 1][j]), s, acc[c * 32 + j]);
          }
        }
      }
      if (!ok) break;
      // C: 32 rows x 64 columns at a time through shared memory
      const int row0 = t.m0 + q * 32;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int n = nh + 64 * x;
        if (n < p.N && n + 64 > p.N && p.N % 8 != 0) {
          // a tensor store is clipped to whole 16-byte chunks: the box with a
          // ragged last chunk goes element by element
          const int r = row0 + lane;
          if (r < p.M) {
            __nv_bfloat16* c = p.C + (p.mode == FP8_DW ? (int64_t)t.e * p.M : 0) * p.ldc + (int64_t)r * p.ldc + n;
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (n + j < p.N) c[j] = __float2bfloat16_rn(acc[x * 64 + j]);
          }
          continue;
        }
        const uint32_t buf = stg + (x * 4096) % SH::kStoreWarp;
        if (SH::kStoreWarp == 4096 || x == 0) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float* a = acc + x * 64 + j * 8;
          st_shared_v4(buf + fp8_sw128(lane, j), make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                            pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7])));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < p.M && n < p.N) {
          tma_store_3d(&p.tmC, buf, n, row0, p.mode == FP8_DW ? t.e : 0);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace moe
