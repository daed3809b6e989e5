// sv_act8.h -- hidden rows to 8-bit codes and back, shared by sv_act8_pack,
// sv_act8_unpack and the token side of sv_head_logits.  gfx950 (MI355X).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_device.h"
#include "sv_head.h"
#include "sv_head_host.h"

namespace sv_act8 {

using sv_dev::u32x4;

// 16 bytes of a row, wherever it begins (the GPU takes 16-byte accesses at any address)
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <int DT> struct In;
template <> struct In<SV_BF16> {
  static constexpr int E = 2;
  static __device__ __forceinline__ float one(const char *p) {
    return __uint_as_float((uint32_t)*(const uint16_t *)p << 16);
  }
  static __device__ __forceinline__ float of(u32x4 v, int i) {
    const uint32_t w = v[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <> struct In<SV_F32> {
  static constexpr int E = 4;
  static __device__ __forceinline__ float one(const char *p) { return *(const float *)p; }
  static __device__ __forceinline__ float of(u32x4 v, int i) { return __uint_as_float(v[i]); }
};

// The code of x under scale s > 0: x / s rounded to even as if it were exact.
// The fp32 quotient may round across a border k + 1/2; the remainder
// x - (k +- 1/2) s is exact in sign as one fused step, and puts the code back.  Its last
// place is half of the scale's: below 2^-125 that is no fp32 number (a remainder of
// 2^-150 would round to a tie), so small rows are taken 2^64 larger, which is exact.
__device__ __forceinline__ int code_of(float x, float s) {
  if (s < 0x1p-100f) {
    x *= 0x1p64f;
    s *= 0x1p64f;
  }
  float r = __builtin_rintf(x / s);
  if (fmaf(-(r + 0.5f), s, x) > 0.f) r += 1.f;
  else if (fmaf(-(r - 0.5f), s, x) < 0.f) r -= 1.f;
  else if (((int)r & 1) && (fmaf(-(r + 0.5f), s, x) == 0.f)) r += 1.f;
  else if (((int)r & 1) && (fmaf(-(r - 0.5f), s, x) == 0.f)) r -= 1.f;
  return (int)fminf(fmaxf(r, -127.f), 127.f);
}

// Four codes of a row in one word: x / s as a product with 1 / s that is rounded to a
// whole number by adding 3 * 2^22, whose low byte is the code.  It may be off by one
// next to a border: the remainder x - r s is exact in fp32 (a multiple of half the
// scale's last place, and no larger than the scale), and where it reaches half the
// scale the code moves on, at half to the even one; FIX does that, and without it
// `edge` tells whether it is needed.  (A division per element kept the row pass at
// 2.5 TB/s, bound by its arithmetic; now 5.1.)
template <bool FIX>
__device__ __forceinline__ uint32_t four_codes(const float (&x)[4], float s, float inv, float half, bool &edge) {
  constexpr float MAGIC = 12582912.f;
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = fmaf(x[i], inv, MAGIC), e = fmaf(-(y - MAGIC), s, x[i]);
    q[i] = __float_as_uint(y);
    if constexpr (FIX) q[i] += (e > half || (e == half && (q[i] & 1))) - (e < -half || (e == -half && (q[i] & 1)));
    else edge |= fabsf(e) >= half;
  }
  const uint32_t lo = __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400), hi = __builtin_amdgcn_perm(q[3], q[2], 0x0c0c0400);
  return lo | hi << 16;
}

// The scale of a row from the largest magnitude's bits (a NaN's or an
// infinity's are at or above those of infinity).
__device__ __forceinline__ float scale_of(uint32_t top) {
  return top >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float(top) / 127.f;
}

struct Pack {
  const char *x;
  int64_t x_ld;                          // bytes
  int8_t *codes;
  int64_t c_ld;                          // bytes
  float *scale;
  int32_t H, Hp;                         // columns; columns written (zeros past H)
  int32_t vec;                           // 16-byte aligned x rows, codes rows aligned for their stores
};

// The largest magnitude (its bit pattern, as an integer maximum, keeps NaN and
// infinity above every number), then the codes.  HBM bound.  A wave takes a row, or
// the four of a workgroup do where there are too few rows to fill the chip with (32
// rows of 4096: 8.4 to 4 us); they hold it in registers, REGS 16-byte vectors a lane,
// so it is read once.  Rows too long for that, or codes that four-byte stores do not
// fit, take a workgroup and a second read from the caches.
template <int DT, int REGS, int WAVES> __global__ __launch_bounds__(256) void pack_rows_kernel(Pack P, int N) {
  constexpr int E = In<DT>::E, W = 16 / E, L = 64 * WAVES;
  static_assert(WAVES == 1 || WAVES == 4, "a wave or a workgroup per row");
  const int lane = threadIdx.x % L;
  const int64_t n = WAVES == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (n >= N) return;
  const char *x = P.x + n * P.x_ld;
  int8_t *c = P.codes + n * P.c_ld;
  const int nv = P.H / W;                // whole vectors; up to W - 1 elements behind them, a lane each
  u32x4 v[REGS];
#pragma unroll
  for (int r = 0; r < REGS; ++r) {
    v[r] = 0;
    if (r * L + lane < nv) v[r] = __builtin_nontemporal_load((const u32x4_any *)x + r * L + lane);
  }
  const int k = nv * W + lane;
  const float rest = k < P.H ? In<DT>::one(x + (int64_t)k * E) : 0.f;
  uint32_t top = __float_as_uint(rest) & 0x7fffffffu;
#pragma unroll
  for (int r = 0; r < REGS; ++r)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t u = __float_as_uint(In<DT>::of(v[r], i)) & 0x7fffffffu;
      top = u > top ? u : top;
    }
  top = (uint32_t)sv_dev::wave_max_i((int)top);
  if constexpr (WAVES == 4) {
    __shared__ uint32_t tops[4];
    if ((lane & 63) == 0) tops[lane >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) top = tops[w] > top ? tops[w] : top;
  }
  const float s = scale_of(top);
  if (lane == 0) P.scale[n] = s;
  const bool none = !(s > 0.f);          // a row of zeros, of magnitudes whose scale rounds to 0, or NaN
  if (!(s > 1e-30f)) {                   // or one whose 1 / s or s / 2 is no ordinary number
    for (int i = lane; i < P.Hp; i += L)
      c[i] = i < P.H && !none ? (int8_t)code_of(In<DT>::one(x + (int64_t)i * E), s) : (int8_t)0;
    return;
  }
  const float inv = 1.f / s, half = 0.5f * s;
#pragma unroll
  for (int r = 0; r < REGS; ++r) {
    const int q = r * L + lane;
    if (q >= nv) continue;
    uint32_t o[W / 4];
    bool edge = false;
#pragma unroll
    for (int w = 0; w < W / 4; ++w) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = In<DT>::of(v[r], 4 * w + i);
      o[w] = four_codes<false>(f, s, inv, half, edge);
    }
    if (edge) {
#pragma unroll
      for (int w = 0; w < W / 4; ++w) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = In<DT>::of(v[r], 4 * w + i);
        o[w] = four_codes<true>(f, s, inv, half, edge);
      }
    }
    if constexpr (W == 8) *(uint64_t *)(c + (int64_t)q * 8) = ((uint64_t)o[1] << 32) | o[0];
    else *(uint32_t *)(c + (int64_t)q * 4) = o[0];
  }
  for (int i = k; i < P.Hp; i += L) c[i] = i < P.H ? (int8_t)code_of(rest, s) : (int8_t)0;
}

template <int DT> __global__ __launch_bounds__(256) void pack_kernel(Pack P) {
  constexpr int E = In<DT>::E, W = 16 / E;
  __shared__ uint32_t top_of[4];
  const int tid = threadIdx.x;
  const int64_t n = blockIdx.x;
  const char *x = P.x + n * P.x_ld;
  int8_t *c = P.codes + n * P.c_ld;
  const int nv = P.vec ? P.H / W : 0;
  uint32_t top = 0;
  for (int q = tid; q < nv; q += 256) {
    const u32x4 v = *(const u32x4 *)(x + (int64_t)q * 16);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t u = __float_as_uint(In<DT>::of(v, i)) & 0x7fffffffu;
      top = u > top ? u : top;
    }
  }
  for (int i = nv * W + tid; i < P.H; i += 256) {
    const uint32_t u = __float_as_uint(In<DT>::one(x + (int64_t)i * E)) & 0x7fffffffu;
    top = u > top ? u : top;
  }
  top = (uint32_t)sv_dev::wave_max_i((int)top);
  if ((tid & 63) == 0) top_of[tid >> 6] = top;
  __syncthreads();
  top = top_of[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) top = top_of[w] > top ? top_of[w] : top;
  const float s = scale_of(top);
  const bool none = !(s > 0.f);          // a row of zeros, of magnitudes whose scale rounds to 0, or NaN
  if (tid == 0) P.scale[n] = s;
  for (int q = tid; q < nv; q += 256) {
    const u32x4 v = *(const u32x4 *)(x + (int64_t)q * 16);
    uint32_t o[W / 4];
#pragma unroll
    for (int w = 0; w < W / 4; ++w) {
      o[w] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!none) o[w] |= (uint32_t)(code_of(In<DT>::of(v, 4 * w + i), s) & 0xff) << (8 * i);
    }
    if constexpr (W == 8) *(uint64_t *)(c + (int64_t)q * 8) = ((uint64_t)o[1] << 32) | o[0];
    else *(uint32_t *)(c + (int64_t)q * 4) = o[0];
  }
  for (int i = nv * W + tid; i < P.Hp; i += 256)
    c[i] = (i < P.H && !none) ? (int8_t)code_of(In<DT>::one(x + (int64_t)i * E), s) : (int8_t)0;
}

template <int DT> void pack_as(int N, Pack P, hipStream_t st) {
  constexpr int E = In<DT>::E, W = 16 / E;
  const bool codes = ((uintptr_t)P.codes & (W - 1)) == 0 && (P.c_ld & (W - 1)) == 0;
  P.vec = codes && ((uintptr_t)P.x & 15) == 0 && (P.x_ld & 15) == 0 ? 1 : 0;
  const dim3 rows((unsigned)((N + 3) / 4)), each((unsigned)N), block(256);
  constexpr int MID = DT == SV_BF16 ? 8 : 16;   // (eight registers of fp32 compile to many more)
  if (codes && N <= 2048 && P.H > 4 * W * 16 && P.H <= 4 * W * 256)
    hipLaunchKernelGGL((pack_rows_kernel<DT, 4, 4>), each, block, 0, st, P, N);
  else if (codes && P.H <= 4 * W * 64) hipLaunchKernelGGL((pack_rows_kernel<DT, 4, 1>), rows, block, 0, st, P, N);
  else if (codes && P.H <= MID * W * 64) hipLaunchKernelGGL((pack_rows_kernel<DT, MID, 1>), rows, block, 0, st, P, N);
  else if (codes && P.H <= 16 * W * 64) hipLaunchKernelGGL((pack_rows_kernel<DT, 16, 1>), rows, block, 0, st, P, N);
  else hipLaunchKernelGGL((pack_kernel<DT>), each, block, 0, st, P);
}

inline void pack(int dtype, int N, Pack P, hipStream_t st) {
  for (int64_t left = N; left > 0; left -= sv_head_host::MAX_ROWS) {
    const int n = (int)(left < sv_head_host::MAX_ROWS ? left : sv_head_host::MAX_ROWS);
    if (dtype == SV_BF16) pack_as<SV_BF16>(n, P, st);
    else pack_as<SV_F32>(n, P, st);
    P.x += n * P.x_ld;
    P.codes += n * P.c_ld;
    P.scale += n;
  }
}

}  // namespace sv_act8
