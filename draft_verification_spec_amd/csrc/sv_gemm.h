// sv_gemm.h -- the tiled matrix product behind the vocabulary-head operators,
// for gfx950 (MI355X): C[m][n] = sum_k X[m][k] Y[n][k], both operands with k
// contiguous ("rows against rows"), in bf16, fp32 or int8.
//
// One core for the three types: a step takes 128 bytes of k (64 bf16, 32 fp32,
// 128 int8) of every row of both tiles, and a matrix instruction takes from
// each lane 16 bytes of one row: lane l holds row l & 15 and 16-byte piece
// l >> 4 of a 64-byte half step.  Which k those bytes are does not matter as
// long as both operands agree, so the three types differ in one instruction
// (four for fp32, whose instruction takes one element a lane) and nowhere else.
//
// Tiles go from memory to LDS by direct 16-byte loads (no registers between),
// the next step's while this step is computed, two buffers, one barrier a
// step.  A direct load writes 64 consecutive pieces, so a row's eight pieces
// are permuted on the memory side: piece p of row r lies at place p ^ (r & 7),
// and the 16 rows that a fragment load touches fall on different banks.
// The columns' fragment is the instruction's first operand: a lane then holds
// four consecutive n of one m, which row-major stores want.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_head.h"

namespace sv_gemm {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int STEP = 128;                // bytes of k a step

template <int DT> struct Mma;
template <> struct Mma<SV_BF16> {
  static constexpr int E = 2;
  typedef f32x4 Acc;
  static __device__ __forceinline__ void mul(Acc &c, u32x4 a, u32x4 b) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <> struct Mma<SV_F32> {
  static constexpr int E = 4;
  typedef f32x4 Acc;
  static __device__ __forceinline__ void mul(Acc &c, u32x4 a, u32x4 b) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
  }
};
template <> struct Mma<SV_I8> {
  static constexpr int E = 1;
  typedef i32x4 Acc;
  static __device__ __forceinline__ void mul(Acc &c, u32x4 a, u32x4 b) {
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};

// A workgroup's tile: WM x WN waves, each of FM x FN fragments of 16 x 16.
template <int FM_, int FN_, int WM_, int WN_> struct Tile {
  static constexpr int FM = FM_, FN = FN_, WM = WM_, WN = WN_;
  static constexpr int NW = WM * WN, TPB = 64 * NW;
  static constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  static constexpr int BUF = (BM + BN) * STEP;           // bytes of one LDS buffer
  static constexpr int LDS = 2 * BUF;
};

// One tile's rows of an operand: the first row, the distance of rows in bytes,
// the rows that exist (>= 1; rows past them repeat the last one, their products
// are not used) and the bytes of a row that exist.
struct Rows {
  const char *base;
  int64_t ld;
  int rows;
  int64_t bytes;
};

// The products of one tile over steps [0, nk) from byte k0 of the rows.
template <int DT, class T>
__device__ __forceinline__ void product(typename Mma<DT>::Acc (&acc)[T::FM][T::FN], char *lds, const Rows &X,
                                        const Rows &Y, int k0, int nk) {
#ifdef __HIP_DEVICE_COMPILE__            // (the host pass knows no gfx950 builtins)
  constexpr int NX = T::BM / 8 / T::NW, NY = T::BN / 8 / T::NW;
  static_assert(NX >= 1 && NY >= 1 && T::BM % (8 * T::NW) == 0 && T::BN % (8 * T::NW) == 0, "tile of whole loads");
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wid / T::WN, wn = wid % T::WN;
  // no load leaves the rows that exist: the resource ends with the last one
  const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
      (void *)X.base, 0, (int)((int64_t)(X.rows - 1) * X.ld + X.bytes), 0x00020000);
  const __amdgpu_buffer_rsrc_t yr = __builtin_amdgcn_make_buffer_rsrc(
      (void *)Y.base, 0, (int)((int64_t)(Y.rows - 1) * Y.ld + Y.bytes), 0x00020000);
  int xo[NX], yo[NY];
  const int sub = lane >> 3, piece = ((lane & 7) ^ sub) * 16;
#pragma unroll
  for (int j = 0; j < NX; ++j) {
    const int r = (wid + j * T::NW) * 8 + sub;
    xo[j] = (r < X.rows ? r : X.rows - 1) * (int)X.ld + piece;
  }
#pragma unroll
  for (int j = 0; j < NY; ++j) {
    const int r = (wid + j * T::NW) * 8 + sub;
    yo[j] = (r < Y.rows ? r : Y.rows - 1) * (int)Y.ld + piece;
  }
  auto issue = [&](char *buf, int ko) {
#pragma unroll
    for (int j = 0; j < NX; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xr, (__attribute__((address_space(3))) void *)(buf + (wid + j * T::NW) * 1024), 16, xo[j], ko, 0, 0);
#pragma unroll
    for (int j = 0; j < NY; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          yr, (__attribute__((address_space(3))) void *)(buf + T::BM * STEP + (wid + j * T::NW) * 1024), 16, yo[j], ko,
          0, 0);
  };
  const int xf = wm * T::FM * 16 * STEP, yf = T::BM * STEP + wn * T::FN * 16 * STEP;
  int at[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) at[h] = (lane & 15) * STEP + (((h * 4 + (lane >> 4)) ^ (lane & 7)) << 4);

  if (nk > 0) issue(lds, k0);
  for (int s = 0; s < nk; ++s) {
    // this step's tiles have landed for every wave, and every wave is done with
    // the buffer that the next step's loads write
    __builtin_amdgcn_s_waitcnt(0x0f70);                  // vmcnt(0)
    __syncthreads();
    if (s + 1 < nk) issue(lds + ((s + 1) & 1) * T::BUF, k0 + (s + 1) * STEP);
    const char *b = lds + (s & 1) * T::BUF;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 x[T::FM], y[T::FN];
#pragma unroll
      for (int f = 0; f < T::FM; ++f) x[f] = *(const u32x4 *)(b + xf + at[h] + f * 16 * STEP);
#pragma unroll
      for (int f = 0; f < T::FN; ++f) y[f] = *(const u32x4 *)(b + yf + at[h] + f * 16 * STEP);
#pragma unroll
      for (int f = 0; f < T::FM; ++f)
#pragma unroll
        for (int g = 0; g < T::FN; ++g) Mma<DT>::mul(acc[f][g], y[g], x[f]);
    }
  }
#endif
}

template <int DT, class T>
__device__ __forceinline__ void clear(typename Mma<DT>::Acc (&acc)[T::FM][T::FN]) {
#pragma unroll
  for (int f = 0; f < T::FM; ++f)
#pragma unroll
    for (int g = 0; g < T::FN; ++g) acc[f][g] = 0;
}

// Workgroup b of `total` to its place in the order of tiles: the GPU deals
// workgroups to its 8 XCDs in turn, and each XCD takes one run of that order,
// so that neighbours share its L2.
__device__ __forceinline__ int run_of_xcd(int b, int total) {
  const int xcd = b & 7, q = total >> 3, r = total & 7;
  return xcd * q + (xcd < r ? xcd : r) + (b >> 3);
}

// Place in the order to (row tile, column tile): bands of `band` row tiles, in
// each band column by column, so that an XCD's workgroups form a block of tiles.
__device__ __forceinline__ void tile_at(int id, int mt, int nt, int band, int &im, int &in) {
  const int per = band * nt, g = id / per, in_band = id - g * per;
  const int h = mt - g * band < band ? mt - g * band : band;
  in = in_band / h;
  im = g * band + (in_band - in * h);
}

}  // namespace sv_gemm
