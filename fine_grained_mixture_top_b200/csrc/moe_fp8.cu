// E4M3 quantization with one fp32 scale per block of 128 values: rows (1 x 128
// blocks, gathered by a routing or behind the SwiGLU product if asked),
// columns (128 x 1 blocks, written transposed) and 128 x 128 blocks of expert
// weights (as they are, or transposed).
//
// For a block's largest magnitude m (at least 2^-110, so that neither scale
// nor factor leaves the normal range): scale = m / 448, code = e4m3(x * (448 / m)),
// both divisions in fp32, one per block.  448 is E4M3's largest value, so no
// code saturates.  Every kernel reads its input once and writes a byte per
// value: bound by those bytes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "fp8_gemm.cuh"
#include "moe.h"
#include "moe_internal.h"
#include "rows.cuh"

namespace moe {
namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr int kBlk = 128;  // values per scale
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 7.7037197775489434e-34f;  // 2^-110

// Four values to four E4M3 codes (rounded to nearest even, saturating), the first
// in the lowest byte.
__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// x *= f, two values per instruction
__device__ __forceinline__ void mul8(float (&x)[8], float f) {
  uint64_t ff;
  asm("mov.b64 %0, {%1, %1};" : "=l"(ff) : "f"(f));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x[2 * i]), "f"(x[2 * i + 1]));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(ff));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x[2 * i]), "=f"(x[2 * i + 1]) : "l"(v));
  }
}

// Eight values of a row as they are stored, from element e0 on (a multiple of
// 8), zeros outside [0, width).  FAST: the row's 16-byte pieces are aligned and
// width is a multiple of 8.  Otherwise pieces whose windows stay inside the row
// come from two windows each, and those at its ends element by element.
template <typename T>
struct Raw8 {
  Piece<T> p[8 / kVec<T>];
  __device__ __forceinline__ float operator[](int i) const { return to_float(p[i / kVec<T>].x[i % kVec<T>]); }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8 / kVec<T>; ++i) *reinterpret_cast<uint4*>(&p[i]) = make_uint4(0u, 0u, 0u, 0u);
  }
};
template <typename T, bool FAST>
__device__ __forceinline__ Raw8<T> load8(const T* row, int e0, int width) {
  constexpr int V = kVec<T>;
  Raw8<T> r;
  if (FAST ? e0 < width : (e0 >= V - 1 && e0 + 8 + V - 1 <= width)) {
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) r.p[i] = load_piece<T, FAST>(row + e0 + i * V);
    return r;
  }
  r.clear();
  if constexpr (!FAST) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e0 + i < width) r.p[i / V].x[i % V] = row[e0 + i];
  }
  return r;
}
// Largest magnitude among them (a NaN does not count); 16-bit types two at a time.
__device__ __forceinline__ float amax8(const Raw8<float>& r) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(r[i]));
  return m;
}
__device__ __forceinline__ float amax8(const Raw8<__nv_bfloat16>& r) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r.p[0]);
  const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float amax8(const Raw8<__half>& r) {
  const __half2* h = reinterpret_cast<const __half2*>(&r.p[0]);
  const __half2 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
  return fmaxf(__low2float(m), __high2float(m));
}
template <typename T>
bool fast_rows(const void* in, int64_t ld, int64_t width) {
  return aligned16(in) && ld * (int64_t)sizeof(T) % 16 == 0 && width % 8 == 0;
}

// n / d for n < 2^31 by a product: mul = ceil(2^(31 + s) / d), 2^(s - 1) < d <= 2^s.
struct FastDiv {
  uint32_t mul, shift, d;
  explicit FastDiv(uint32_t d_ = 1) : mul(0), shift(0), d(d_) {
    if (d < 2) return;
    uint32_t s = 1;
    while ((1u << s) < d) ++s;
    mul = (uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d);
    shift = s - 1;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return d < 2 ? n : __umulhi(n, mul) >> shift; }
};

struct QuantArgs {
  int64_t rows, ld_in, ld_codes, ld_scales;
  int cols, kblocks;           // blocks of a row (rows kernel)
  FastDiv by_kblocks;
  const int* row_src;          // nullable: the input row of each row; outside [0, in_rows): zeros
  int64_t in_rows;
  const int* rows_used;        // nullable: rows from here on are left as they are
  uint8_t* codes;
  float* scales;
  int64_t plane_in, plane_codes, plane_scales;  // expert weights: elements per expert
};

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + __expf(-g)) * u; }

// eight codes from column e0 on, clipped to `cols`
__device__ __forceinline__ void store_codes(uint8_t* out, const float (&x)[8], int e0, int cols) {
  const uint2 q = make_uint2(cvt4(x[0], x[1], x[2], x[3]), cvt4(x[4], x[5], x[6], x[7]));
  if (e0 + 8 <= cols) {
    *reinterpret_cast<uint2*>(out) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e0 + j < cols) out[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
  }
}

// Sixteen values from element e0 on (a multiple of 16).  LOAD: 0 any alignment, 1
// as load8's FAST, 2 the row's 32-byte pieces are aligned and width is a multiple
// of 16.
template <typename T, int LOAD>
__device__ __forceinline__ void load16_values(Raw8<T> (&x)[2], const T* row, int e0, int width) {
  if constexpr (LOAD == 2) {
    if (e0 >= width) {
      x[0].clear();
      x[1].clear();
      return;
    }
    constexpr int N = 8 / kVec<T>;  // 16-byte pieces per Raw8
    uint4 u[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) load32(row + e0 + i * 2 * kVec<T>, u[2 * i], u[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) *reinterpret_cast<uint4*>(&x[i / N].p[i % N]) = u[i];
  } else {
    x[0] = load8<T, LOAD == 1>(row, e0, width);
    x[1] = load8<T, LOAD == 1>(row, e0 + 8, width);
  }
}

// Rows: a block of 128 values per 4 lanes, 32 per lane in two runs of 16, 64
// apart, so that 4 lanes read 128 bytes of a 16-bit type and write 64 at a time.
// At memory's rate the kernel has some 16 instructions and 1/12 of a shared
// L1 wavefront per value.  With 8 values per lane and scalar maxima it was bound
// by issue (182 us), with 32 in runs of 8 by L1 wavefronts (120 us); it now takes
// 96 us (16384 tokens of 2048 bf16 values gathered 8 times), and 59 us for 65536
// rows of 2048 as they lie (6.9 TB/s of reads and writes).
template <typename T, int LOAD, bool SWIGLU>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(const QuantArgs a, const T* __restrict__ in) {
  pdl_wait();
  const int l = threadIdx.x & 3;
  const uint32_t unit = blockIdx.x * 64u + (threadIdx.x >> 2);
  const uint32_t row = a.by_kblocks.div(unit);
  const int kb = (int)(unit - row * (uint32_t)a.kblocks);
  const int64_t used = a.rows_used ? min((int64_t)__ldg(a.rows_used), a.rows) : a.rows;
  const bool live = row < used;
  int64_t from = live ? (a.row_src ? (int64_t)__ldg(a.row_src + row) : (int64_t)row) : -1;
  if (a.row_src && from >= a.in_rows) from = -1;
  const int e0 = kb * kBlk + 16 * l;
  const int width = from < 0 ? 0 : a.cols;  // nothing to load: zeros
  const T* src = in + (from < 0 ? 0 : from) * a.ld_in;
  Raw8<T> x[2][2];
  float v[SWIGLU ? 4 : 1][8];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) load16_values<T, LOAD>(x[i], src, e0 + 64 * i, width);
  if constexpr (SWIGLU) {  // the up projection lies behind the gate's `cols` columns
    Raw8<T> up[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) load16_values<T, LOAD>(up[i], src + a.cols, e0 + 64 * i, width);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = silu_mul(x[i >> 1][i & 1][j], up[i >> 1][i & 1][j]);
        m = fmaxf(m, fabsf(v[i][j]));
      }
  } else {
    m = fmaxf(fmaxf(amax8(x[0][0]), amax8(x[0][1])), fmaxf(amax8(x[1][0]), amax8(x[1][1])));
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, kAmaxFloor);
  if (!live) return;
  const float f = kE4m3Max / m;
  uint8_t* out = a.codes + (int64_t)row * a.ld_codes + e0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float w[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 8; ++j) w[h][j] = SWIGLU ? v[SWIGLU ? 2 * i + h : 0][j] : x[i][h][j];
    mul8(w[0], f);
    mul8(w[1], f);
    if (e0 + 64 * i + 16 <= a.cols) {
      *reinterpret_cast<uint4*>(out + 64 * i) =
          make_uint4(cvt4(w[0][0], w[0][1], w[0][2], w[0][3]), cvt4(w[0][4], w[0][5], w[0][6], w[0][7]),
                     cvt4(w[1][0], w[1][1], w[1][2], w[1][3]), cvt4(w[1][4], w[1][5], w[1][6], w[1][7]));
    } else {
      store_codes(out + 64 * i, w[0], e0 + 64 * i, a.cols);
      store_codes(out + 64 * i + 8, w[1], e0 + 64 * i + 8, a.cols);
    }
  }
  if (l == 0) a.scales[(int64_t)kb * a.ld_scales + row] = m / kE4m3Max;
}

// Tiles of 128 rows x 128 columns, one per thread block, held in registers as they
// are stored (which leaves room for more thread blocks than fp32 would): a
// thread has 8 columns of 8 rows (two groups of 4 consecutive ones), so that it
// packs 4 codes of a column into a word for the transposed store.
//   COLS   one scale per column of the tile, codes transposed [cols, rows]
//   !COLS  one scale per tile; TRANS: codes transposed
//   GATHER the tile's rows are in[row_src[r]]
// Thread blocks per SM that the registers are cut for (a tile is loads, a
// barrier, stores, so that several have to overlap), as measured: 16-bit columns
// 4 (32768 x 2048: 51 us, at 2 69), blocks 5 or, unaligned, 6 (32 x 1001 x 1003:
// 32 us, at 4 36); fp32 3.
template <typename T, bool FAST, bool COLS>
constexpr int kTileBlocks = sizeof(T) == 4 ? 3 : COLS ? 4 : FAST ? 5 : 6;
template <typename T, bool FAST, bool COLS, bool TRANS, bool GATHER>
__global__ void __launch_bounds__(256, kTileBlocks<T, FAST, COLS>) fp8_quant_tile_kernel(const QuantArgs a,
                                                                                           const T* __restrict__ in0) {
  pdl_wait();
  __shared__ uint32_t words[TRANS ? kBlk * 33 : 1];  // [column][4-row group], one word of padding
  __shared__ float part[8][COLS ? kBlk : 1];
  __shared__ float factor[COLS ? kBlk : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = (int64_t)blockIdx.y * kBlk;
  const int c0 = (int)blockIdx.x * kBlk;
  const int64_t rows = a.rows_used ? min((int64_t)__ldg(a.rows_used), a.rows) : a.rows;
  if (r0 >= rows) return;
  const T* in = in0 + (int64_t)blockIdx.z * a.plane_in;
  uint8_t* codes = a.codes + (int64_t)blockIdx.z * a.plane_codes;
  float* scales = a.scales + (int64_t)blockIdx.z * a.plane_scales;
  const int col = 8 * (lane & 15);
  const int group = 2 * warp + (lane >> 4);  // rows 4 group .. + 3, and 64 more
  Raw8<T> x[8];
  int from[8];  // row of the tile (GATHER: of `in`), -1: zeros
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * group + (i & 3) + 64 * (i >> 2);
    from[i] = r0 + r < rows ? r : -1;
    if (GATHER && from[i] >= 0) from[i] = __ldg(a.row_src + r0 + r);
  }
  const T* first = GATHER ? in : in + r0 * a.ld_in;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (from[i] >= 0 && (!GATHER || from[i] < a.in_rows))
      x[i] = load8<T, FAST>(first + from[i] * a.ld_in, c0 + col, a.cols);
    else
      x[i].clear();
  }
  float f[8];
  if constexpr (COLS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float m = kAmaxFloor;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i][j]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      if (lane < 16) part[warp][col + j] = m;
    }
    __syncthreads();
    if (threadIdx.x < kBlk) {
      float m = part[0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < 8; ++w) m = fmaxf(m, part[w][threadIdx.x]);
      factor[threadIdx.x] = kE4m3Max / m;
      if (c0 + (int)threadIdx.x < a.cols) scales[(int64_t)blockIdx.y * a.ld_scales + c0 + threadIdx.x] = m / kE4m3Max;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = factor[col + j];
  } else {
    float m = kAmaxFloor;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(x[i]));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    if (lane == 0) part[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, part[w][0]);
    const float g = kE4m3Max / m;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = g;
    if (threadIdx.x == 0)
      scales[TRANS ? (int64_t)blockIdx.x * a.ld_scales + blockIdx.y : (int64_t)blockIdx.y * a.ld_scales + blockIdx.x] =
          m / kE4m3Max;
  }
  if constexpr (TRANS) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        words[(col + j) * 33 + group + 16 * h] = cvt4(x[4 * h][j] * f[j], x[4 * h + 1][j] * f[j],
                                                      x[4 * h + 2][j] * f[j], x[4 * h + 3][j] * f[j]);
    __syncthreads();
    const int64_t r = r0 + 4 * lane;
    for (int c = warp; c < kBlk && c0 + c < a.cols; c += 8) {
      const uint32_t w = words[c * 33 + lane];
      uint8_t* out = codes + (int64_t)(c0 + c) * a.ld_codes + r;
      if (r + 4 <= rows) {
        *reinterpret_cast<uint32_t*>(out) = w;
      } else {
        for (int b = 0; b < 4 && r + b < rows; ++b) out[b] = (uint8_t)(w >> (8 * b));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + 4 * group + (i & 3) + 64 * (i >> 2);
      if (r >= rows) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = x[i][j] * f[j];
      store_codes(codes + r * a.ld_codes + c0 + col, v, c0 + col, a.cols);
    }
  }
}

template <typename T>
cudaError_t launch_rows(const QuantArgs& a, const void* in, bool swiglu, cudaStream_t s) {
  const unsigned grid = (unsigned)cdiv(a.rows * a.kblocks, 64);
  const T* x = static_cast<const T*>(in);
  const bool fast = fast_rows<T>(in, a.ld_in, a.cols);
  const bool wide = fast && reinterpret_cast<uintptr_t>(in) % 32 == 0 && a.ld_in * (int64_t)sizeof(T) % 32 == 0 &&
                    a.cols % 16 == 0;
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(256), 0, s, a, x); };
  if (swiglu)
    return wide ? go(fp8_quant_rows_kernel<T, 2, true>)
                : fast ? go(fp8_quant_rows_kernel<T, 1, true>) : go(fp8_quant_rows_kernel<T, 0, true>);
  return wide ? go(fp8_quant_rows_kernel<T, 2, false>)
              : fast ? go(fp8_quant_rows_kernel<T, 1, false>) : go(fp8_quant_rows_kernel<T, 0, false>);
}

template <typename T, bool COLS, bool TRANS>
cudaError_t launch_tiles(const QuantArgs& a, int E, const void* in, cudaStream_t s) {
  const dim3 grid((unsigned)cdiv(a.cols, kBlk), (unsigned)cdiv(a.rows, kBlk), (unsigned)E);
  const T* x = static_cast<const T*>(in);
  const bool fast = fast_rows<T>(in, a.ld_in, a.cols) && a.plane_in * (int64_t)sizeof(T) % 16 == 0;
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, s, a, x); };
  if constexpr (COLS) {
    if (a.row_src)
      return fast ? go(fp8_quant_tile_kernel<T, true, COLS, TRANS, true>)
                  : go(fp8_quant_tile_kernel<T, false, COLS, TRANS, true>);
  }
  return fast ? go(fp8_quant_tile_kernel<T, true, COLS, TRANS, false>)
              : go(fp8_quant_tile_kernel<T, false, COLS, TRANS, false>);
}

// Copies of rows quantized once: codes[r] = from.codes[row_src[r]] and the same of
// the scales, zeros (and the scale of zeros) where there is no such row.  A block
// has blockDim.y kGatherRows rows, kGatherRows of them in flight per thread, in
// 16-byte pieces of blockDim.x columns; blocks of the first column part take
// their rows' scales.  (One row per thread and blocks for the scales: the
// gather of 16384 tokens of 2048 values to 131072 rows took 137 us in all where
// this takes 85, and quantizing every copied row 96.)
constexpr int kGatherRows = 8;
__global__ void __launch_bounds__(256) fp8_gather_kernel(const QuantArgs a, const uint8_t* __restrict__ codes,
                                                         int64_t ld, const float* __restrict__ scales,
                                                         int64_t ld_scales) {
  pdl_wait();
  const int64_t used = a.rows_used ? min((int64_t)__ldg(a.rows_used), a.rows) : a.rows;
  const int per = blockDim.y * kGatherRows;
  const int64_t r0 = (int64_t)blockIdx.x * per;
  if (r0 >= used) return;
  const int e0 = 16 * (int)(blockIdx.y * blockDim.x + threadIdx.x);
  if (e0 < a.cols) {
    int from[kGatherRows];
    uint4 v[kGatherRows];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      const int64_t r = r0 + i * blockDim.y + threadIdx.y;
      from[i] = r < used ? __ldg(a.row_src + r) : -1;
    }
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if ((uint32_t)from[i] < (uint32_t)a.in_rows) v[i] = load16(codes + from[i] * ld + e0);
    }
    const int64_t step = (int64_t)blockDim.y * a.ld_codes;
    uint8_t* out = a.codes + (r0 + threadIdx.y) * a.ld_codes + e0;
    const int live = (int)min((int64_t)kGatherRows, (used - r0 - threadIdx.y + blockDim.y - 1) / blockDim.y);
    if (e0 + 16 <= a.cols) {
#pragma unroll
      for (int i = 0; i < kGatherRows; ++i)
        if (i < live) *reinterpret_cast<uint4*>(out + i * step) = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < kGatherRows; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (i < live && e0 + j < a.cols) out[i * step + j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
      }
    }
  }
  if (blockIdx.y == 0) {  // a warp per block of columns, its lanes along the rows
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, warps = (blockDim.x * blockDim.y) >> 5;
    for (int i = tid & 31; i < per && r0 + i < used; i += 32) {
      const int from = __ldg(a.row_src + r0 + i);
      const bool real = from >= 0 && from < a.in_rows;
      for (int kb = tid >> 5; kb < a.kblocks; kb += warps)
        a.scales[(int64_t)kb * a.ld_scales + r0 + i] =
            real ? __ldg(scales + (int64_t)kb * ld_scales + from) : kAmaxFloor / kE4m3Max;
    }
  }
}
cudaError_t launch_gather(const QuantArgs& a, const QuantArgs& once, cudaStream_t s) {
  const int64_t pieces = cdiv(a.cols, 16), parts = cdiv(pieces, 256);
  const unsigned x = (unsigned)(cdiv(cdiv(pieces, parts), 32) * 32), y = 256 / x;
  return launch_pdl(fp8_gather_kernel, dim3((unsigned)cdiv(a.rows, y * kGatherRows), (unsigned)cdiv(pieces, x)),
                    dim3(x, y), 0, s, a, (const uint8_t*)once.codes, once.ld_codes, (const float*)once.scales,
                    once.ld_scales);
}

int64_t elem_size(moe_dtype t) { return t == MOE_F32 ? 4 : (t == MOE_BF16 || t == MOE_F16) ? 2 : 0; }
// in may be null where a gather has no input rows: then every row is zeros.
moe_status check_quant(moe_dtype type, const void* in, int64_t ld_in, int64_t width, const void* codes,
                       int64_t ld_codes, int64_t code_cols, const float* scales, bool no_input = false) {
  const int64_t es = elem_size(type);
  if (es == 0) return MOE_ERR_INVALID_ARG;
  if ((!in && !no_input) || !codes || !scales || reinterpret_cast<uintptr_t>(in) % (uintptr_t)es || !aligned16(codes) ||
      (reinterpret_cast<uintptr_t>(scales) & 3u))
    return MOE_ERR_INVALID_ARG;
  if (ld_in < width || ld_codes < code_cols || ld_codes % 16 != 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

#define MOE_TRY_CUDA(...)                                                              \
  do {                                                                                 \
    const cudaError_t moe_e_ = (__VA_ARGS__);                                          \
    if (moe_e_ != cudaSuccess) return api_cuda_failed(moe_e_, "moe_fp8.cu", __LINE__); \
  } while (0)
#define MOE_BY_TYPE(type, CALL)                                   \
  switch (type) {                                                 \
    case MOE_BF16: { using T = __nv_bfloat16; MOE_TRY_CUDA(CALL); break; } \
    case MOE_F16: { using T = __half; MOE_TRY_CUDA(CALL); break; }         \
    default: { using T = float; MOE_TRY_CUDA(CALL); }                      \
  }

extern "C" {

moe_status moe_fp8_quantize_rows(moe_dtype type, const void* in, int64_t ld_in, int64_t in_rows, int64_t rows,
                                 int32_t cols, const int32_t* row_src, const int32_t* rows_used, int32_t swiglu,
                                 void* codes, int64_t ld_codes, float* scales, int64_t ld_scales, void* ws,
                                 size_t ws_bytes, void* stream) {
  ApiRange api_range("moe_fp8_quantize_rows");
  if (rows < 0 || in_rows < 0 || cols < 1 || swiglu < 0 || swiglu > 1) return MOE_ERR_INVALID_ARG;
  const int kb = (int)cdiv(cols, kBlk);
  constexpr int64_t kMostBlocks = (int64_t(1) << 31) - 64;
  if (cols > (1 << 20) || rows >= kMostBlocks || rows * kb >= kMostBlocks) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const moe_status st = check_quant(type, in, ld_in, (int64_t)cols * (1 + swiglu), codes, ld_codes, cols, scales,
                                    row_src && in_rows == 0);
  if (st != MOE_OK) return st;
  if (ld_scales < rows) return MOE_ERR_INVALID_ARG;
  QuantArgs a = {};
  a.rows = rows;
  a.ld_in = ld_in;
  a.ld_codes = ld_codes;
  a.ld_scales = ld_scales;
  a.cols = cols;
  a.kblocks = kb;
  a.by_kblocks = FastDiv((uint32_t)kb);
  a.row_src = row_src;
  a.in_rows = in_rows;
  a.rows_used = rows_used;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t need = moe_fp8_gather_ws(in_rows, cols);
  if (row_src && in_rows > 0 && rows >= in_rows && ws && ws_bytes >= need) {
    if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
    // each input row once into ws, then copies of its codes and scales
    QuantArgs once = a;
    once.rows = in_rows;
    once.row_src = nullptr;
    once.rows_used = nullptr;
    once.ld_codes = cdiv(cols, 16) * 16;
    once.codes = static_cast<uint8_t*>(ws);
    once.ld_scales = in_rows;
    once.scales = reinterpret_cast<float*>(once.codes + in_rows * once.ld_codes);
    {
      ProfScope ps(s, "fp8_quantize_rows");
      MOE_BY_TYPE(type, (launch_rows<T>(once, in, swiglu != 0, s)));
    }
    ProfScope ps(s, "fp8_gather_codes");
    MOE_TRY_CUDA(launch_gather(a, once, s));
    return MOE_OK;
  }
  ProfScope ps(s, "fp8_quantize_rows");
  MOE_BY_TYPE(type, (launch_rows<T>(a, in, swiglu != 0, s)));
  return MOE_OK;
}

size_t moe_fp8_gather_ws(int64_t in_rows, int32_t cols) {
  if (in_rows < 0 || cols < 1) return 0;
  return (size_t)in_rows * ((size_t)cdiv(cols, 16) * 16 + (size_t)cdiv(cols, kBlk) * sizeof(float));
}

moe_status moe_fp8_quantize_cols(moe_dtype type, const void* in, int64_t ld_in, int64_t in_rows, int64_t rows,
                                 int32_t cols, const int32_t* row_src, const int32_t* rows_used, void* codes,
                                 int64_t ld_codes, float* scales, int64_t ld_scales, void* stream) {
  ApiRange api_range("moe_fp8_quantize_cols");
  if (rows < 0 || in_rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (cols > (1 << 20) || cdiv(rows, kBlk) > 65535) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const moe_status st = check_quant(type, in, ld_in, cols, codes, ld_codes, rows, scales, row_src && in_rows == 0);
  if (st != MOE_OK) return st;
  if (ld_scales < cols) return MOE_ERR_INVALID_ARG;
  QuantArgs a = {};
  a.rows = rows;
  a.ld_in = ld_in;
  a.ld_codes = ld_codes;
  a.ld_scales = ld_scales;
  a.cols = cols;
  a.row_src = row_src;
  a.in_rows = in_rows;
  a.rows_used = rows_used;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope ps(s, "fp8_quantize_cols");
  MOE_BY_TYPE(type, (launch_tiles<T, true, true>(a, 1, in, s)));
  return MOE_OK;
}

moe_status moe_fp8_quantize_blocks(moe_dtype type, const void* in, int32_t E, int32_t K, int32_t N, int32_t transpose,
                                   void* codes, int64_t ld_codes, float* scales, void* stream) {
  ApiRange api_range("moe_fp8_quantize_blocks");
  if (E < 0 || K < 1 || N < 1 || transpose < 0 || transpose > 1) return MOE_ERR_INVALID_ARG;
  if (E > 65535 || K > 65535 * kBlk || N > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (E == 0) return MOE_OK;
  const moe_status st = check_quant(type, in, N, N, codes, ld_codes, transpose ? K : N, scales);
  if (st != MOE_OK) return st;
  QuantArgs a = {};
  a.rows = K;
  a.ld_in = N;
  a.ld_codes = ld_codes;
  a.ld_scales = transpose ? cdiv(K, kBlk) : cdiv(N, kBlk);
  a.cols = N;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.plane_in = (int64_t)K * N;
  a.plane_codes = (int64_t)(transpose ? N : K) * ld_codes;
  a.plane_scales = cdiv(K, kBlk) * cdiv(N, kBlk);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope ps(s, "fp8_quantize_blocks");
  if (transpose) {
    MOE_BY_TYPE(type, (launch_tiles<T, false, true>(a, E, in, s)));
  } else {
    MOE_BY_TYPE(type, (launch_tiles<T, false, false>(a, E, in, s)));
  }
  return MOE_OK;
}

// ----------------------------------------------------------------- products
// Launch with a cluster of `split` CTAs and programmatic stream serialization.
static cudaError_t launch_small(const Fp8Params& p, int grid, int smem, cudaStream_t s) {
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(fp8_gemm_small_kernel), 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(Fp8SmallShape::kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = MOE_PDL;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = p.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, fp8_gemm_small_kernel, p);
}

static moe_status fp8_product(int mode, int64_t M, int64_t N, int64_t K, int32_t planes, const moe_routing* rt,
                              const void* A, int64_t lda, const float* sA, int64_t ldsA, const void* B, int64_t ldb,
                              const float* sB, int64_t ldsB, void* C, int64_t ldc, cudaStream_t s) {
  ApiDevice dev;
  if (!api_device(&dev)) return MOE_ERR_CUDA;
  Fp8Params p;
  memset(&p, 0, sizeof(p));
  const bool dw = mode == FP8_DW;
  p.sA = sA;
  p.sB = sB;
  p.ldsA = ldsA;
  p.ldsB = ldsB;
  p.ldc = ldc;
  p.C = static_cast<__nv_bfloat16*>(C);
  p.offsets = rt ? rt->offsets : nullptr;
  p.E = planes;
  p.M = (int)M;
  p.N = (int)N;
  p.nb = (int)cdiv(N, 128);
  p.kb = (int)cdiv(K, 128);
  p.mode = mode;
  p.st = DevStatus{dev.status, dev.spin_limit};
  const uint64_t bplanes = mode == FP8_GROUPED ? planes : 1, cplanes = dw ? planes : 1;
  const uint64_t bplane = (uint64_t)N * ldb;
  // With at most one tile per SM of 128 columns and up to 128 rows: those, with the
  // operands exchanged, of which the machine holds twice as many and which may share
  // their sums (microseconds, pair tiles / exchanged: 16 x 4096 x 7168 28 / 13;
  // 16 x 16384 x 7168, 128 tiles, 31 / 27; 1024 x 2048 x 7168, 128 tiles, 37 / 32;
  // 1001 x 1528 x 2000, 96 tiles, 12.7 / 11.3).  With more, pairs: 1280 x 2048 x 1024,
  // 160 tiles, 8.9 / 11.7; 2048 x 2048 x 2048, 256 tiles, 13 / 19.  Grouped products
  // always take pairs: even with a few rows per expert they read the weights faster
  // (64 tokens x 8 of 128 experts, 1536 x 2048: 118 / 133).
  const int64_t tok_boxes = std::min<int64_t>(4, cdiv(M, 32));
  const bool few = mode == FP8_DENSE && cdiv(M, 32 * tok_boxes) * cdiv(N, 128) <= dev.sms;
  if (few) {
    p.tok_boxes = (int)tok_boxes;
    if (!api_tensor_map(&p.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, B, bplanes, N, K, ldb, bplane, 128, 128) ||
        !api_tensor_map(&p.tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, A, 1, M, K, lda, (uint64_t)M * lda, 32 * p.tok_boxes, 128))
      return MOE_ERR_INVALID_ARG;
    p.mt = (int)cdiv(M, 32 * p.tok_boxes);
    p.nt = p.nb;
    const int tiles = p.mt * p.nt;
    p.split = 1;
    while (p.split < 8 && 2 * tiles * p.split <= dev.sms && p.kb >= 4 * p.split) p.split *= 2;
    ProfScope ps(s, "fp8_gemm");
    MOE_TRY_CUDA(launch_small(p, tiles * p.split, Fp8SmallShape::smem(p.tok_boxes), s));
    return MOE_OK;
  }
  if (!api_tensor_map(&p.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, A, 1, M, K, lda, (uint64_t)M * lda, 128, 128) ||
      !api_tensor_map(&p.tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, B, bplanes, N, K, ldb, bplane, 128, 128) ||
      !api_tensor_map(&p.tmC, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, C, cplanes, M, N, 2 * ldc, (uint64_t)M * 2 * ldc, 32, 64))
    return MOE_ERR_INVALID_ARG;
  p.mt = (int)cdiv(M, 256);
  p.nt = (int)cdiv(N, 256);
  // GROUPED: an expert's odd last tile is a pair tile too
  const int64_t tiles = ((int64_t)p.mt + (mode == FP8_GROUPED ? planes : 0)) * p.nt * cplanes;
  if (tiles >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  using SH = Fp8PairShape;
  const void* fn = dw ? reinterpret_cast<const void*>(fp8_gemm_pair_kernel<true>)
                      : reinterpret_cast<const void*>(fp8_gemm_pair_kernel<false>);
  MOE_TRY_CUDA(set_max_dynamic_smem(fn, SH::kSmem));
  const int most = std::max(1, std::min(dev.sms / 2, resident_pairs(fn, SH::kThreads, SH::kSmem)));
  const int pairs = (int)std::min<int64_t>(tiles, most);
  ProfScope ps(s, dw ? "fp8_gemm_dw" : "fp8_gemm");
  MOE_TRY_CUDA(dw ? launch_pdl(fp8_gemm_pair_kernel<true>, dim3(2 * pairs), dim3(SH::kThreads), SH::kSmem, s, p)
                  : launch_pdl(fp8_gemm_pair_kernel<false>, dim3(2 * pairs), dim3(SH::kThreads), SH::kSmem, s, p));
  return MOE_OK;
}

static moe_status check_product(int64_t M, int64_t N, int64_t K, int32_t E, const moe_routing* rt, const void* A,
                                int64_t lda, const float* sA, const void* B, int64_t ldb, const float* sB,
                                const void* C, int64_t ldc) {
  if (rt && (!rt->offsets || !aligned16(rt->offsets))) return MOE_ERR_INVALID_ARG;
  if (M >= (int64_t(1) << 31) - 256 || N >= (int64_t(1) << 31) - 256 || K >= (int64_t(1) << 31) - 256 || E > 1024 ||
      (!rt && E != 1))
    return MOE_ERR_UNSUPPORTED;
  if (!A || !B || !C || !sA || !sB || !aligned16(A) || !aligned16(B) || !aligned16(C)) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(sA) & 3u) || (reinterpret_cast<uintptr_t>(sB) & 3u)) return MOE_ERR_INVALID_ARG;
  if (lda < K || ldb < K || ldc < N || lda % 16 || ldb % 16 || ldc % 8) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status moe_fp8_gemm(int64_t M, int64_t N, int64_t K, int32_t E, const moe_routing* rt, const void* A, int64_t lda,
                        const float* sA, int64_t ldsA, const void* B, int64_t ldb, const float* sB, void* C,
                        int64_t ldc, void* stream) {
  ApiRange api_range("moe_fp8_gemm");
  if (M < 0 || N < 1 || K < 1 || E < 1) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  const moe_status st = check_product(M, N, K, E, rt, A, lda, sA, B, ldb, sB, C, ldc);
  if (st != MOE_OK) return st;
  if (ldsA < M || (rt && M % 128 != 0)) return MOE_ERR_INVALID_ARG;
  return fp8_product(rt ? FP8_GROUPED : FP8_DENSE, M, N, K, E, rt, A, lda, sA, ldsA, B, ldb, sB, 0, C, ldc,
                     static_cast<cudaStream_t>(stream));
}

moe_status moe_fp8_gemm_dw(int64_t M, int64_t N, int64_t K, int32_t E, const moe_routing* rt, const void* A,
                           int64_t lda, const float* sA, int64_t ldsA, const void* B, int64_t ldb, const float* sB,
                           int64_t ldsB, void* C, int64_t ldc, void* stream) {
  ApiRange api_range("moe_fp8_gemm_dw");
  if (M < 1 || N < 1 || K < 0 || E < 1) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) {  // no tokens: no operands, a gradient of zeros
    if (!C || !aligned16(C) || ldc < N || ldc % 8) return MOE_ERR_INVALID_ARG;
    if (M >= (int64_t(1) << 31) - 256 || N >= (int64_t(1) << 31) - 256 || E > 1024 || (!rt && E != 1))
      return MOE_ERR_UNSUPPORTED;  // as with tokens
    MOE_TRY_CUDA(cudaMemset2DAsync(C, (size_t)ldc * 2, 0, (size_t)N * 2, (size_t)(E * M), s));
    return MOE_OK;
  }
  const moe_status st = check_product(M, N, K, E, rt, A, lda, sA, B, ldb, sB, C, ldc);
  if (st != MOE_OK) return st;
  if (ldsA < M || ldsB < N || (rt && K % 128 != 0)) return MOE_ERR_INVALID_ARG;
  return fp8_product(FP8_DW, M, N, K, E, rt, A, lda, sA, ldsA, B, ldb, sB, ldsB, C, ldc, s);
}

}  // extern "C"
