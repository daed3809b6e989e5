// sv_mx4.hip -- microscaled 4-bit rows (sv_mx4_pack, sv_mx4_unpack) and the vocabulary head
// held in them (sv_head_logits4), for gfx950 (MI355X).
//
// The matrix instruction takes 32 codes of a row from a lane, which is one block: lane l
// holds row l & 15 and block l >> 4 of 128 elements of k, its scale beside it, and scales the
// block's sum of products itself.  Products of two codes are exact; sums are fp32.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <atomic>

#include "sv_device.h"
#include "sv_gemm.h"
#include "sv_mx4.h"
#include "sv_mx4_host.h"

namespace {

using namespace sv_gemm;
using sv_mx4_host::cdiv;
using sv_mx4_host::tiled_scale;

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ rows to codes
constexpr int64_t FEW = 8 * sv_mx4_host::CUS * 1024;     // items (lanes' shares) that take a thread each

// Eight elements of a row: a lane's share.  Four lanes hold a block.
template <int DT> __device__ __forceinline__ void load8(const char *row, int64_t k, int64_t H, float (&v)[8]) {
  if (k + 8 <= H) {
    if constexpr (DT == SV_BF16) {
      const u32x4 u = __builtin_nontemporal_load((const u32x4_any *)(row + k * 2));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    } else {
      const u32x4 a = __builtin_nontemporal_load((const u32x4_any *)(row + k * 4));
      const u32x4 b = __builtin_nontemporal_load((const u32x4_any *)(row + k * 4) + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.f;
      if (k + i < H) {
        if constexpr (DT == SV_BF16) v[i] = __uint_as_float((uint32_t)((const uint16_t *)row)[k + i] << 16);
        else v[i] = ((const float *)row)[k + i];
      }
    }
  }
}

// 2^(e - 127) of a scale byte below 255
__device__ __forceinline__ float power_of(uint32_t e) { return __uint_as_float(e ? e << 23 : 1u << 22); }

// The codes of a lane's eight elements (the first in the low bits) and its block's scale.
// The block's largest magnitude comes from its four lanes, which all take part.
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], uint32_t &e) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = sv_dev::fmax_nan(m, fabsf(v[i]));
  uint32_t top = __float_as_uint(m);
  m = sv_dev::fmax_nan(m, __uint_as_float(sv_dev::dpp<0xb1, 0xf, 0xf>(top, top)));
  top = __float_as_uint(m);
  m = sv_dev::fmax_nan(m, __uint_as_float(sv_dev::dpp<0x4e, 0xf, 0xf>(top, top)));
  top = __float_as_uint(m) & 0x7fffffffu;
  uint32_t c = 0;
#ifdef __HIP_DEVICE_COMPILE__
  if (top >= 0x7f800000u) {
    e = 255;
  } else {
    const uint32_t b = top >> 23;
    e = b > 2 ? b - 2 : 0;
    const float s = power_of(e);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  }
#endif
  return c;
}

// `n` bytes (below 4) of a word
__device__ __forceinline__ void store_bytes(uint8_t *p, uint32_t c, int n) {
  for (int i = 0; i < n; ++i) p[i] = (uint8_t)(c >> (8 * i));
}

// Where codes and scales go: rows as the caller lays them, the hidden rows' image of the
// streaming product, or their rows and scales of the tiled one.
enum Form { ROWS_OUT, HELD, TILED };
struct Out {
  uint8_t *codes, *scale;
  int64_t c_ld, s_ld;                    // ROWS_OUT, TILED: bytes between code rows; ROWS_OUT: scale rows
  int64_t N, H;                          // HELD: rows; ROWS_OUT: columns
  int64_t groups;                        // TILED: 16-block groups of scales in a row
};

// HELD: piece (block, row) of 16 bytes; the scales of blocks 4 j + q, j = 4 i .. 4 i + 3, in a
// word at (i, q, row).
__device__ __forceinline__ int64_t held_piece(int64_t block, int64_t row, int64_t N) { return block * N + row; }
__device__ __forceinline__ int64_t held_scale(int64_t block, int64_t row, int64_t N) {
  return ((block / 16 * 4 + block % 4) * N + row) * 4 + block / 4 % 4;
}

template <int FORM>
__device__ __forceinline__ void put(const Out &o, int64_t row, int64_t g, uint32_t c, uint32_t e) {
  if constexpr (FORM == ROWS_OUT) {
    const int64_t at = 4 * g, end = (o.H + 1) / 2;
    uint8_t *p = o.codes + row * o.c_ld + at;
    if (at + 4 <= end) *(u32_any *)p = c;
    else if (at < end) store_bytes(p, c, (int)(end - at));
    if (g % 4 == 0) o.scale[row * o.s_ld + g / 4] = (uint8_t)e;
  } else if constexpr (FORM == HELD) {
    *(uint32_t *)(o.codes + held_piece(g / 4, row, o.N) * 16 + g % 4 * 4) = c;
    if (g % 4 == 0) o.scale[held_scale(g / 4, row, o.N)] = (uint8_t)e;
  } else {
    const int64_t b = g / 4;
    *(uint32_t *)(o.codes + row * o.c_ld + 4 * g) = c;
    if (g % 4 == 0) o.scale[tiled_scale(row, b / 16, b % 4 * 16 + row % 16, o.groups) * 4 + b / 4 % 4] = (uint8_t)e;
  }
}

struct Rows {
  const char *x;                         // elements, or SV_MX4: codes
  int64_t x_ld;                          // bytes
  const uint8_t *scale;                  // SV_MX4
  int64_t s_ld;
  int64_t H;
  int64_t items;                         // rows x lanes of a row
  int32_t lanes;                         // of a row: 4 for each block written
};

// A lane's eight elements as codes, formed or copied (what lies behind column H is 0).
template <int SRC> __device__ __forceinline__ uint32_t take(const Rows &R, int64_t row, int64_t g, uint32_t &e) {
  if constexpr (SRC == SV_MX4) {
    const int64_t k = 8 * g;
    uint32_t c = 0;
    e = 0;
    if (k < R.H) {
      const uint8_t *p = (const uint8_t *)R.x + row * R.x_ld + 4 * g;
      if (k + 8 <= R.H) {
        c = *(const u32_any *)p;
      } else {
        const int n = (int)(R.H - k);
        for (int i = 0; 2 * i < n; ++i) c |= (uint32_t)p[i] << (8 * i);
        c &= (1u << (4 * n)) - 1;
      }
      e = R.scale[row * R.s_ld + g / 4];
    }
    return c;
  } else {
    float v[8];
    load8<SRC>(R.x + row * R.x_ld, 8 * g, R.H, v);
    return codes_of(v, e);
  }
}

// Lanes over all rows' items, PER a thread.  HBM bound: 151936 rows of 4096 bf16 265 us (1.58 GB),
// one a thread 310; 4999 of 1111 fp32 8.1 us with one, 9.4 with four.
template <int SRC, int FORM, int PER> __global__ __launch_bounds__(256) void rows_kernel(Rows R, Out O) {
  const int64_t first = (int64_t)blockIdx.x * (256 * PER);
  const int64_t row0 = first / R.lanes;
  const int rest = (int)(first - row0 * R.lanes);
#pragma unroll
  for (int s = 0; s < PER; ++s) {
    const int64_t i = first + s * 256 + threadIdx.x;
    if (i >= R.items) return;            // (whole blocks: items are)
    const int at = rest + s * 256 + (int)threadIdx.x, r = at / R.lanes;
    uint32_t e;
    const uint32_t c = take<SRC>(R, row0 + r, at - r * R.lanes, e);
    put<FORM>(O, row0 + r, at - r * R.lanes, c, e);
  }
}

template <int FORM> void launch_rows(int src, Rows R, Out O, int64_t rows, hipStream_t st) {
  R.items = rows * R.lanes;
  const bool few = R.items < FEW;
  const dim3 grid((unsigned)cdiv(R.items, few ? 256 : 1024)), block(256);
  auto go = [&](auto S) {
    constexpr int SRC = decltype(S)::value;
    if (few) hipLaunchKernelGGL((rows_kernel<SRC, FORM, 1>), grid, block, 0, st, R, O);
    else hipLaunchKernelGGL((rows_kernel<SRC, FORM, 4>), grid, block, 0, st, R, O);
  };
  if (src == SV_BF16) go(std::integral_constant<int, SV_BF16>());
  else if (src == SV_F32) go(std::integral_constant<int, SV_F32>());
  else if constexpr (FORM != ROWS_OUT) go(std::integral_constant<int, SV_MX4>());
}

// ------------------------------------------------------------------ codes to rows
// HBM bound as well: 151936 rows of 4096 into bf16 300 us (1.58 GB).
template <int DT, int PER> __global__ __launch_bounds__(256) void unpack_kernel(Rows R, char *y) {
  const int64_t first = (int64_t)blockIdx.x * (256 * PER);
  const int64_t row0 = first / R.lanes;
  const int rest = (int)(first - row0 * R.lanes);
  constexpr int E = DT == SV_BF16 ? 2 : 4;
#pragma unroll
  for (int s = 0; s < PER; ++s) {
    const int64_t i = first + s * 256 + threadIdx.x;
    if (i >= R.items) return;
    const int at = rest + s * 256 + (int)threadIdx.x, r = at / R.lanes;
    const int64_t row = row0 + r, g = at - r * R.lanes, k = 8 * g;
    uint32_t e;
    const uint32_t c = take<SV_MX4>(R, row, g, e);
    const float p = power_of(e);
    float v[8] = {};
#ifdef __HIP_DEVICE_COMPILE__
#define TWO(n)                                                        \
  {                                                                   \
    const f32x2 t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, p, n); \
    v[2 * n] = t[0];                                                  \
    v[2 * n + 1] = t[1];                                              \
  }
    TWO(0) TWO(1) TWO(2) TWO(3)
#undef TWO
#endif
    if (e == 255)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __builtin_nanf("");
    char *o = y + (row * R.H + k) * E;
    if (k + 8 <= R.H) {
      if constexpr (DT == SV_BF16) {
        __builtin_nontemporal_store(u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])},
                                    (u32x4_any *)o);
      } else {
        __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4_any *)o);
        __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, (f32x4_any *)o + 1);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + j < R.H) {
          if constexpr (DT == SV_BF16) ((__bf16 *)o)[j] = (__bf16)v[j];
          else ((float *)o)[j] = v[j];
        }
    }
  }
}

// ----------------------------------------------------------------------- products
struct LogitsP {
  Rows x;                                // fused: the hidden rows themselves
  const uint8_t *xc, *xs;                // staged codes and scales
  int64_t x_ld;                          // tiles: bytes between code rows
  const uint8_t *w, *ws;                 // weight codes and scales
  int64_t w_ld, s_ld;                    // bytes
  int64_t w_bytes;                       // tiles: what exists of a code row
  char *out;
  int64_t out_ld;                        // elements
  int32_t N, V, H;
  int32_t nks;                           // held: 128-element steps
  int32_t groups;                        // held: 16-row groups of the vocabulary; tiles: 16-block groups of k
  int32_t mt, nt, band;
};

#ifdef __HIP_DEVICE_COMPILE__
__device__ __forceinline__ i32x8 eight(u32x4 v) { return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0}; }
// c += (w's codes times x's), w's scale in byte WB of sw, x's in byte XB of sx
template <int WB, int XB> __device__ __forceinline__ void mul(f32x4 &c, u32x4 w, uint32_t sw, u32x4 x, uint32_t sx) {
  c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(eight(w), eight(x), c, 4, 4, WB, (int)sw, XB, (int)sx);
}
#endif

template <int OT> __device__ __forceinline__ void store4(char *out, int64_t at, int left, f32x4 v) {
  if constexpr (OT == SV_BF16) {
    if (left >= 4) {
      *(u32x2_any *)(out + at * 2) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) ((__bf16 *)out)[at + i] = (__bf16)v[i];
    }
  } else {
    if (left >= 4) {
      *(f32x4_any *)(out + at * 4) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) ((float *)out)[at + i] = v[i];
    }
  }
}

// Eight steps of k (1024 elements) of 16 vocabulary rows: a lane's codes, and its row's
// scales, of which byte l >> 4 of word i is the lane's at step i.
struct Chunk {
  u32x4 w[8];
  uint32_t s[8];
};

// Few rows: each workgroup holds all of their codes in LDS, and each of its waves streams
// 16 vocabulary rows at a time from memory to registers, a chunk ahead, with no barrier;
// rows lie at any address and distance.  Bound by reading the head: 32 rows of 4096 x 151936
// 70 us (330 MB, 4.9 TB/s with the logits), 64 79.  Loads past the cache (nontemporal) fetch
// each line's halves apart: 76 us for the 32 rows.  Beyond 64 rows the registers (140 and more)
// leave a CU one workgroup, though LDS may hold two.
template <int FM, int SRC, int OT, int WAVES> __global__ __launch_bounds__(64 * WAVES, FM > 4 ? 2 : 4) void held_kernel(LogitsP P) {
  extern __shared__ __align__(16) uint8_t held[];
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4;
  const int nc = (P.nks + 7) / 8, nb = (P.H + 31) / 32, bytes = (P.H + 1) / 2;
  const int64_t N = P.N;
  uint8_t *const scales = held + N * P.nks * 64;
  const int wave = __builtin_amdgcn_readfirstlane((int)blockIdx.x * WAVES + (tid >> 6)), waves = (int)gridDim.x * WAVES;

  auto load = [&](Chunk &t, int g, int c) {
    const int64_t r = (int64_t)g * 16 + i, row = r < P.V ? r : P.V - 1;
    const uint8_t *w = P.w + row * P.w_ld, *s = P.ws + row * P.s_ld + c * 32;
    const int at = c * 512 + q * 16;
    if ((c + 1) * 512 <= bytes) {
#pragma unroll
      for (int k = 0; k < 8; ++k) t.w[k] = *(const u32x4_any *)(w + at + k * 64);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        t.w[k] = 0;
        if (at + k * 64 + 16 <= bytes) t.w[k] = *(const u32x4_any *)(w + at + k * 64);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int a = at + k * 64;
        if (a < bytes && a + 16 > bytes) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (a + j < bytes) t.w[k][j / 4] |= (uint32_t)w[a + j] << (j % 4 * 8);
        }
      }
    }
    if ((c + 1) * 32 <= nb) {
      const u32x4 a = *(const u32x4_any *)s, b = *((const u32x4_any *)s + 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        t.s[k] = a[k];
        t.s[4 + k] = b[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) t.s[k] = c * 32 + k * 4 + q < nb ? (uint32_t)s[k * 4 + q] << (8 * q) : 0u;
    }
  };

  // chunks of a group begin at different places, so that rows a power of two apart do not
  // meet in one memory channel
  Chunk a, b;
  int g = wave, c = g < P.groups ? g % nc : 0, done = 0;
  if (g < P.groups) load(a, g, c);
  // the hidden rows
  if constexpr (SRC == SV_MX4) {
    const int n = (int)(N * P.nks * 4), m = (int)(N * ((P.nks + 3) / 4));
    // (eight loads under way together: 128 rows of 2048 x 151936 54 to 50 us)
    for (int j = tid; j < n; j += 8 * 64 * WAVES) {
      u32x4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i * 64 * WAVES < n) v[i] = ((const u32x4 *)P.xc)[j + i * 64 * WAVES];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i * 64 * WAVES < n) ((u32x4 *)held)[j + i * 64 * WAVES] = v[i];
    }
    for (int j = tid; j < m; j += 64 * WAVES) ((u32x4 *)scales)[j] = ((const u32x4 *)P.xs)[j];
  } else {
    const Out o = {held, scales, 0, 0, N, 0, 0};
    const int lanes = P.nks * 16;
    for (int j = tid; j < N * lanes; j += 64 * WAVES) {
      const int row = j / lanes;
      uint32_t e;
      const uint32_t v = take<SRC>(P.x, row, j - row * lanes, e);
      put<HELD>(o, row, j - row * lanes, v, e);
    }
  }
  __syncthreads();
  int64_t m[FM];
#pragma unroll
  for (int f = 0; f < FM; ++f) m[f] = f * 16 + i < N ? f * 16 + i : N - 1;
  f32x4 acc[FM];
#pragma unroll
  for (int f = 0; f < FM; ++f) acc[f] = 0;
  auto work = [&](const Chunk &t) {
#ifdef __HIP_DEVICE_COMPILE__
    const int have = P.nks - c * 8;
    auto four = [&](int h) {             // steps 4 h .. 4 h + 3 of the chunk
      uint32_t sx[FM];
#pragma unroll
      for (int f = 0; f < FM; ++f) sx[f] = ((const uint32_t *)scales)[((c * 2 + h) * 4 + q) * N + m[f]];
      auto one = [&](auto K) {
        constexpr int k = decltype(K)::value;
        if (4 * h + k < have) {
#pragma unroll
          for (int f = 0; f < FM; ++f) {
            const u32x4 x = ((const u32x4 *)held)[((c * 8 + 4 * h + k) * 4 + q) * N + m[f]];
            mul<0, k>(acc[f], h ? t.w[4 + k] : t.w[k], (h ? t.s[4 + k] : t.s[k]) >> (8 * q), x, sx[f]);
          }
        }
      };
      one(std::integral_constant<int, 0>());
      one(std::integral_constant<int, 1>());
      one(std::integral_constant<int, 2>());
      one(std::integral_constant<int, 3>());
    };
    if (have > 0) four(0);
    if (have > 4) four(1);
#endif
  };
  auto step = [&](Chunk &now, Chunk &next) {
    int g2 = g, c2 = c + 1 == nc ? 0 : c + 1;
    const bool last = done + 1 == nc;
    if (last) {
      g2 = g + waves;
      c2 = g2 % nc;
    }
    if (g2 < P.groups) load(next, g2, c2);
    work(now);
    ++done;
    if (last) {
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        if (f * 16 + i < N) {
          const int v = g * 16 + q * 4;
          store4<OT>(P.out, (int64_t)(f * 16 + i) * P.out_ld + v, P.V - v, acc[f]);
        }
        acc[f] = 0;
      }
      done = 0;
    }
    g = g2;
    c = c2;
  };
  while (g < P.groups) {
    step(a, b);
    if (g >= P.groups) break;
    step(b, a);
  }
}

// The weight's scales as the lanes of the tiled product take them (tiled_scale).  A thread takes
// 16 scales of four rows 16 apart: it turns four words of four blocks into four of every
// fourth, and stores those of the four rows together (151936 rows of 128: a row a thread 13 us,
// this 11).  0 past the rows' end (codes of the hidden rows are 0 there; what lies in
// memory might stand for NaN).
__global__ __launch_bounds__(256) void scales_kernel(const uint8_t *s, int64_t ld, int64_t V, int nb, int groups,
                                                     int64_t items, u32x4 *o) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= items) return;
  const int64_t rest = i / groups, row = rest / 16 * 64 + rest % 16;   // neighbours: groups of a row
  const int group = (int)(i - rest * groups), b = group * 16;
  u32x4 w[4];                            // w[q][f]: blocks 4 k + q of row 16 f
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    u32x4 v = 0;
    if (row + 16 * f < V) {
      const uint8_t *p = s + (row + 16 * f) * ld + b;
      if (b + 16 <= nb) {
        v = *(const u32x4_any *)p;
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (b + k < nb) v[k / 4] |= (uint32_t)p[k] << (k % 4 * 8);
      }
    }
    const uint32_t lo = __builtin_amdgcn_perm(v[1], v[0], 0x05010400), hi = __builtin_amdgcn_perm(v[3], v[2], 0x05010400);
    const uint32_t lo2 = __builtin_amdgcn_perm(v[1], v[0], 0x07030602), hi2 = __builtin_amdgcn_perm(v[3], v[2], 0x07030602);
    w[0][f] = __builtin_amdgcn_perm(hi, lo, 0x05040100);
    w[1][f] = __builtin_amdgcn_perm(hi, lo, 0x07060302);
    w[2][f] = __builtin_amdgcn_perm(hi2, lo2, 0x05040100);
    w[3][f] = __builtin_amdgcn_perm(hi2, lo2, 0x07060302);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) o[tiled_scale(row, group, 16 * q + row % 16, groups) / 4] = w[q];
}

#ifdef __HIP_DEVICE_COMPILE__
// Four products of one hidden fragment, scales in byte K of their words.  The compiler gives
// the builtin's result registers of its own, and with all of them taken moves sums about
// (five moves to two products; 1024 rows of 4096 x 151936 457 us), so the sums are tied
// here.  s_nop: what the compiler may write to a source right before.
#define SV_MUL4(SEL)                                                                                 \
  asm volatile("s_nop 1\n\t"                                                                         \
               "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %4, %8, %0, %9, %13 " SEL " cbsz:4 blgp:4\n\t"  \
               "v_mfma_scale_f32_16x16x128_f8f6f4 %1, %5, %8, %1, %10, %13 " SEL " cbsz:4 blgp:4\n\t" \
               "v_mfma_scale_f32_16x16x128_f8f6f4 %2, %6, %8, %2, %11, %13 " SEL " cbsz:4 blgp:4\n\t" \
               "v_mfma_scale_f32_16x16x128_f8f6f4 %3, %7, %8, %3, %12, %13 " SEL " cbsz:4 blgp:4"      \
               : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3])                                      \
               : "v"(y[0]), "v"(y[1]), "v"(y[2]), "v"(y[3]), "v"(x), "v"(sy[0]), "v"(sy[1]), "v"(sy[2]), "v"(sy[3]), "v"(sx))
template <int K> __device__ __forceinline__ void mul4(f32x4 *c, const u32x4 *y, u32x4 sy, u32x4 x, uint32_t sx) {
  if constexpr (K == 0) SV_MUL4("op_sel:[0,0,0] op_sel_hi:[0,0,0]");
  else if constexpr (K == 1) SV_MUL4("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
  else if constexpr (K == 2) SV_MUL4("op_sel:[0,0,0] op_sel_hi:[1,1,0]");
  else SV_MUL4("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
}
#undef SV_MUL4
#endif

// Many rows: tiles of both operands through LDS, two buffers each, laid as in sv_gemm.h; a
// pair of steps at a time, whose four scales of a row are a word.  A wave holds one set of
// fragments of the hidden rows and two of the weight's: a hidden fragment of the next half
// step is read into the registers of this one's as soon as its products are issued.  The one
// barrier of a step stands in its middle: by then every wave has read all of the step's
// buffers, which later loads may overwrite, and the next step's tiles have landed.
//
// A workgroup takes one tile after another, and its loads run on into the next: a tile's
// results leave while the next one's first steps come in (1024 rows of 512 x 65536 54 to 45
// us, of 4096 x 151936 398 to 379).  Rows a power of two apart lie on few memory channels at
// any one step, so neighbouring tiles of the vocabulary begin at different pairs.
//
// 1024 rows of 4096 x 151936 take 363 to 382 us (on several GPUs), 3.4 PFLOP/s; without the loads 290 (230 of them the
// matrix instructions, 23 cycles each, 60 the results' ways out).  A third buffer of the
// weight, eight waves of half the size, stores of 128 bytes a row and workgroups begun at
// times of their own each changed it by 1% or less; tiles of 128 x 128 take a quarter longer.
// With bf16 results the large tiles' wave is 7 registers beyond its 512: they are spilled and read
// again outside the loop over k, where results leave.
template <class T, int OT> __global__ __launch_bounds__(T::TPB) void tile_kernel(LogitsP P) {
  __shared__ __align__(16) char lds[2 * (T::XBUF + T::YBUF)];
#ifdef __HIP_DEVICE_COMPILE__
  typedef Side<SV_I8, T::BM, T::FM, T::NW, ROWS> SX;
  typedef Side<SV_I8, T::BN, T::FN, T::NW, ROWS> SY;
  static_assert(T::FM % 4 == 0 && T::FN % 4 == 0 && T::FN <= T::FM, "products in fours, weight reads beside hidden ones");
  constexpr int LD = SX::NL + SY::NL, PER = (LD + T::FM - 1) / T::FM;   // loads of a step, beside a fragment's products
  constexpr int STORES = T::FM * T::FN / (OT == SV_BF16 ? 2 : 1);       // of a wave's whole tile
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wid / T::WN, wn = wid % T::WN, gx = wm * T::FM, gy = wn * T::FN;
  const int total = P.mt * P.nt, pairs = P.groups, nk = 2 * pairs;
  SX sx;
  SY sy;
  const u32x4 *xs, *ws;
  int m0, n0, from;
  // the loads' tile
  auto start = [&](int id) {
    int im, in;
    tile_at(run_of_xcd(id, total), P.mt, P.nt, P.band, im, in);
    m0 = im * T::BM;
    n0 = in * T::BN;
    from = in % pairs;
    const Part X = {(const char *)P.xc + (int64_t)m0 * P.x_ld, P.x_ld, P.N - m0 < T::BM ? P.N - m0 : T::BM, (int64_t)pairs * 256};
    const Part Y = {(const char *)P.w + (int64_t)n0 * P.w_ld, P.w_ld, P.V - n0 < T::BN ? P.V - n0 : T::BN, P.w_bytes};
    sx.start(X, 0, nk, 2 * from);
    sy.start(Y, 0, nk, 2 * from);
    xs = (const u32x4 *)P.xs + (int64_t)(m0 / 64 + gx / 4) * pairs * 64 + lane;
    ws = (const u32x4 *)P.ws + (int64_t)(n0 / 64 + gy / 4) * pairs * 64 + lane;
  };
  u32x4 x[T::FM], y0[T::FN], y1[T::FN];
  u32x4 sa[T::FM / 4], sb[T::FN / 4], sa2[T::FM / 4], sb2[T::FN / 4];   // a word a fragment
  f32x4 acc[T::FM][T::FN];
  clear<SV_BF16, T>(acc);
  // this wave's first fragments in a buffer at half step 0 and 1
  const int o0 = (lane & 15) * STEP + (((lane >> 4) ^ (lane & 7)) << 4), o1 = o0 ^ 64;
  char *const x0b = lds, *const x1b = lds + T::XBUF, *const y0b = lds + 2 * T::XBUF, *const y1b = y0b + T::YBUF;
  const int fx = gx * 16 * STEP, fy = gy * 16 * STEP;
  // This wave's LDS reads are done and its loads have landed, and so are all others'.  The
  // results of the tile before, which it may have stored since, need not have.
  bool stored = false;
  auto landed = [&]() {
    asm volatile("" ::: "memory");
    constexpr int S = STORES < 63 ? STORES : 63;
    if (stored) __builtin_amdgcn_s_waitcnt(0x0070 | (S & 15) | (S >> 4) << 14);
    else wait_loads<0, 1>(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // Products of half step K of a pair; beside them the reads of the next half's fragments from
  // xb and yb, a later step's loads into xl and yl, and a pair's scales.
  auto half = [&](auto K, u32x4 (&y)[T::FN], u32x4 (&yn)[T::FN], const char *xb, const char *yb, auto loads, char *xl,
                  char *yl, auto scales) {
#pragma unroll
    for (int f = 0; f < T::FM; ++f) {
#pragma unroll
      for (int g = 0; g < T::FN; g += 4) mul4<decltype(K)::value>(&acc[f][g], &y[g], sb[g / 4], x[f], sa[f / 4][f % 4]);
      x[f] = *(const u32x4 *)(xb + f * 16 * STEP);
      if (f < T::FN) yn[f] = *(const u32x4 *)(yb + f * 16 * STEP);
      if constexpr (decltype(loads)::value) {
#pragma unroll
        for (int j = f * PER; j < (f + 1) * PER && j < LD; ++j) {
          if (j < SX::NL) sx.issue_one(xl, j);
          else sy.issue_one(yl, j - SX::NL);
        }
      }
      if constexpr (decltype(scales)::value) {
        if (f < T::FM / 4) sa2[f] = xs[(f * pairs + from) * 64];
        if (f < T::FN / 4) sb2[f] = ws[(f * pairs + from) * 64];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (decltype(loads)::value) {
      sx.next(nk);
      sy.next(nk);
    }
  };
  typedef std::true_type Yes;
  typedef std::false_type No;
  int id = blockIdx.x;
  start(id);
#pragma unroll
  for (int f = 0; f < T::FM / 4; ++f) sa[f] = xs[(f * pairs + from) * 64];
#pragma unroll
  for (int f = 0; f < T::FN / 4; ++f) sb[f] = ws[(f * pairs + from) * 64];
  sx.issue(x0b, true, nk);
  sy.issue(y0b, true, nk);
  sx.issue(x1b, true, nk);
  sy.issue(y1b, true, nk);
  landed();
#pragma unroll
  for (int f = 0; f < T::FM; ++f) x[f] = *(const u32x4 *)(x0b + fx + o0 + f * 16 * STEP);
#pragma unroll
  for (int f = 0; f < T::FN; ++f) y0[f] = *(const u32x4 *)(y0b + fy + o0 + f * 16 * STEP);
  const Beside beside;
  for (;;) {
    const int m1 = m0, n1 = n0;          // this tile, when the loads are at the next
    for (int p = 0; p < pairs; ++p) {
      const bool last = p + 1 == pairs;
      from = from + 1 == pairs ? 0 : from + 1;
      if (last) {
        id += gridDim.x;
        if (id < total) {
          start(id);
        } else {                         // loads read nothing, and what is read of LDS is not used
          sx.stop();
          sy.stop();
        }
      }
      half(std::integral_constant<int, 0>(), y0, y1, x0b + fx + o1, y0b + fy + o1, No(), nullptr, nullptr, No());
      landed();
      stored = false;
      half(std::integral_constant<int, 1>(), y1, y0, x1b + fx + o0, y1b + fy + o0, Yes(), x0b, y0b, Yes());
      half(std::integral_constant<int, 2>(), y0, y1, x1b + fx + o1, y1b + fy + o1, No(), nullptr, nullptr, No());
      landed();
      half(std::integral_constant<int, 3>(), y1, y0, x0b + fx + o0, y0b + fy + o0, Yes(), x1b, y1b, No());
      // The last products' results, before an instruction of the compiler's own touches them: 20
      // wait states, more than any matrix instruction asks for, most of them the last product's
      // own time.  What reads a sum from here on reads what the statements behind the wait give,
      // and these keep their order to it.  Both stand in every turn: behind the loop, or in its
      // last turn alone, the sums have two homes and are moved from one to the other before the
      // wait (150 rows of 4096 x 8000 20.6 to 20.0 us, 1024 of 151936 the same).
      asm volatile("s_nop 15\n\ts_nop 3" ::: "memory");
#pragma unroll
      for (int f = 0; f < T::FM; ++f)
#pragma unroll
        for (int g = 0; g < T::FN; g += 4)
          asm volatile("" : "+a"(acc[f][g]), "+a"(acc[f][g + 1]), "+a"(acc[f][g + 2]), "+a"(acc[f][g + 3]));
#pragma unroll
      for (int f = 0; f < T::FM / 4; ++f) sa[f] = sa2[f];
#pragma unroll
      for (int f = 0; f < T::FN / 4; ++f) sb[f] = sb2[f];
    }
    stored = m1 + T::BM <= P.N && n1 + T::BN <= P.V;
#pragma unroll
    for (int f = 0; f < T::FM; ++f) {
      const int m = m1 + (gx + f) * 16 + (lane & 15);
      if (stored || m < P.N) {
        const int64_t row = (int64_t)m * P.out_ld;
#pragma unroll
        for (int g = 0; g < T::FN; g += OT == SV_BF16 ? 2 : 1) {
          const int n = n1 + (gy + g) * 16;
          if constexpr (OT == SV_BF16) {
            float u[4], v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              u[i] = acc[f][g][i];
              v[i] = acc[f][g + 1][i];
            }
            const u32x4 r = Beside::eight(u, v);
            if (stored) *(u32x4_any *)(P.out + (row + n + beside.at) * 2) = r;
            else store8(P.out, row, n + beside.at, P.V, r);
          } else {
            const int c = n + (lane >> 4) * 4;
            store4<SV_F32>(P.out, row + c, stored ? 4 : P.V - c, acc[f][g]);
          }
        }
      }
    }
    if (id >= total) break;
    clear<SV_BF16, T>(acc);
  }
  __builtin_amdgcn_s_waitcnt(0x0070);    // no load is left that writes to LDS
#endif
}

template <int FM, int SRC, int OT, int WAVES> void launch_held(const LogitsP &P, int64_t lds, hipStream_t st) {
  const int64_t by = cdiv(P.groups, WAVES), most = sv_mx4_host::CUS * (2 * lds <= sv_mx4_host::LDS_ROWS ? 2 : 1);
  // (more than 64 KB of LDS has to be asked for, once on each device)
  static std::atomic<uint64_t> asked{0};
  int dev = 0;
  if (lds > (64 << 10) && hipGetDevice(&dev) == hipSuccess && !(asked.load() >> (dev & 63) & 1)) {
    (void)hipFuncSetAttribute((const void *)held_kernel<FM, SRC, OT, WAVES>, hipFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sv_mx4_host::LDS_ROWS);
    asked.fetch_or((uint64_t)1 << (dev & 63));
  }
  hipLaunchKernelGGL((held_kernel<FM, SRC, OT, WAVES>), dim3((unsigned)(by < most ? by : most)), dim3(64 * WAVES),
                     (unsigned)lds, st, P);
}
template <int FM, int SRC, int WAVES = 8> void launch_held(const LogitsP &P, int ot, int64_t lds, hipStream_t st) {
  if (ot == SV_BF16) launch_held<FM, SRC, SV_BF16, WAVES>(P, lds, st);
  else launch_held<FM, SRC, SV_F32, WAVES>(P, lds, st);
}

template <class T> void launch_tiles(LogitsP P, int ot, hipStream_t st) {
  P.mt = (int)cdiv(P.N, T::BM);
  P.nt = (int)cdiv(P.V, T::BN);
  P.band = 8;
  const int64_t tiles = (int64_t)P.mt * P.nt, most = sv_mx4_host::CUS * (T::BM == 256 ? 1 : 2);   // as LDS holds
  const dim3 grid((unsigned)(tiles < most ? tiles : most)), block(T::TPB);
  if (ot == SV_BF16) hipLaunchKernelGGL((tile_kernel<T, SV_BF16>), grid, block, 0, st, P);
  else hipLaunchKernelGGL((tile_kernel<T, SV_F32>), grid, block, 0, st, P);
}

}  // namespace

extern "C" int sv_mx4_pack(int32_t N, int32_t H, int32_t dtype, const void *x, int64_t x_stride, uint8_t *codes,
                           int64_t codes_stride, uint8_t *scale, int64_t scale_stride, void *stream) {
  using namespace sv_mx4_host;
  const int rc = check_rows(N, H, dtype, x, x_stride, codes, codes_stride, scale, scale_stride);
  if (rc != SV_OK || N == 0) return rc;
  Rows R = {(const char *)x, (x_stride ? x_stride : H) * esize(dtype), nullptr, 0, H, 0, (int32_t)(4 * blocks(H))};
  Out O = {codes, scale, codes_stride ? codes_stride : code_bytes(H), scale_stride ? scale_stride : blocks(H), N, H, 0};
  const int64_t most = sv_head_host::max_groups(256) * 1024 / R.lanes;   // rows of a launch
  for (int64_t n = 0; n < N; n += most) {
    const int64_t rows = N - n < most ? N - n : most;
    launch_rows<ROWS_OUT>(dtype, R, O, rows, (hipStream_t)stream);
    R.x += rows * R.x_ld;
    O.codes += rows * O.c_ld;
    O.scale += rows * O.s_ld;
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

extern "C" int sv_mx4_unpack(int32_t N, int32_t H, const uint8_t *codes, int64_t codes_stride, const uint8_t *scale,
                             int64_t scale_stride, int32_t y_dtype, void *y, void *stream) {
  using namespace sv_mx4_host;
  const int rc = check_rows(N, H, y_dtype, y, 0, codes, codes_stride, scale, scale_stride);
  if (rc != SV_OK || N == 0) return rc;
  Rows R = {(const char *)codes, codes_stride ? codes_stride : code_bytes(H), scale,
            scale_stride ? scale_stride : blocks(H), H, 0, (int32_t)(4 * blocks(H))};
  char *o = (char *)y;
  const int64_t most = sv_head_host::max_groups(256) * 1024 / R.lanes;
  for (int64_t n = 0; n < N; n += most) {
    const int64_t rows = N - n < most ? N - n : most;
    R.items = rows * R.lanes;
    const bool few = R.items < FEW;
    const dim3 grid((unsigned)cdiv(R.items, few ? 256 : 1024)), block(256);
    const hipStream_t st = (hipStream_t)stream;
    if (y_dtype == SV_BF16) {
      if (few) hipLaunchKernelGGL((unpack_kernel<SV_BF16, 1>), grid, block, 0, st, R, o);
      else hipLaunchKernelGGL((unpack_kernel<SV_BF16, 4>), grid, block, 0, st, R, o);
    } else {
      if (few) hipLaunchKernelGGL((unpack_kernel<SV_F32, 1>), grid, block, 0, st, R, o);
      else hipLaunchKernelGGL((unpack_kernel<SV_F32, 4>), grid, block, 0, st, R, o);
    }
    R.x += rows * R.x_ld;
    R.scale += rows * R.s_ld;
    o += rows * H * esize(y_dtype);
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

extern "C" size_t sv_head_logits4_workspace_bytes(const sv_logits4_shape_t *s) {
  if (!s || !sv_mx4_host::shape_ok(s)) return 0;
  return sv_mx4_host::plan_for(s).total;
}

extern "C" int sv_head_logits4(const sv_logits4_shape_t *shape, const void *hidden, const uint8_t *hidden_scale,
                               const uint8_t *weight_codes, const uint8_t *weight_scale, void *logits, void *workspace,
                               size_t workspace_bytes, void *stream) {
  using namespace sv_mx4_host;
  bool nothing;
  const int rc = check_logits(shape, hidden, hidden_scale, weight_codes, weight_scale, logits, workspace,
                              workspace_bytes, &nothing);
  if (rc != SV_OK || nothing) return rc;
  const sv_logits4_shape_t s = *shape;
  const hipStream_t st = (hipStream_t)stream;
  const Plan L = plan_for(&s);
  uint8_t *ws = (uint8_t *)workspace;
  const bool given = s.hidden_dtype == SV_MX4;
  LogitsP P = {};
  P.x = Rows{(const char *)hidden, given ? (s.hidden_stride ? s.hidden_stride : code_bytes(s.H))
                                         : (s.hidden_stride ? s.hidden_stride : s.H) * esize(s.hidden_dtype),
             hidden_scale, s.hidden_scale_stride ? s.hidden_scale_stride : blocks(s.H), s.H, 0, 0};
  P.xc = ws + L.codes;
  P.xs = ws + L.scales;
  P.w_ld = s.weight_stride ? s.weight_stride : code_bytes(s.H);
  P.s_ld = s.weight_scale_stride ? s.weight_scale_stride : blocks(s.H);
  P.out_ld = s.out_stride ? s.out_stride : s.V;
  P.N = s.N;
  P.H = s.H;
  if (L.held) {
    P.w = weight_codes;
    P.ws = weight_scale;
    P.out = (char *)logits;
    P.V = s.V;
    P.nks = (int32_t)L.nks;
    P.groups = (int32_t)cdiv(s.V, 16);
    if (!L.fused) {
      Rows R = P.x;
      R.lanes = (int32_t)(L.nks * 16);
      launch_rows<HELD>(s.hidden_dtype, R, Out{ws + L.codes, ws + L.scales, 0, 0, s.N, 0, 0}, s.N, st);
    }
    const int64_t lds = held_bytes(s.N, s.H);
    if (L.fused) {                       // (16 rows at most)
      if (s.hidden_dtype == SV_BF16) launch_held<1, SV_BF16>(P, s.out_dtype, lds, st);
      else launch_held<1, SV_F32>(P, s.out_dtype, lds, st);
    } else {
      switch (L.frags) {
        case 1: launch_held<1, SV_MX4>(P, s.out_dtype, lds, st); break;
        case 2: launch_held<2, SV_MX4>(P, s.out_dtype, lds, st); break;
        case 3: launch_held<3, SV_MX4>(P, s.out_dtype, lds, st); break;
        case 4: launch_held<4, SV_MX4>(P, s.out_dtype, lds, st); break;
        case 5: launch_held<5, SV_MX4>(P, s.out_dtype, lds, st); break;
        case 6: launch_held<6, SV_MX4>(P, s.out_dtype, lds, st); break;
        default: launch_held<8, SV_MX4>(P, s.out_dtype, lds, st);
      }
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
  }
  {
    Rows R = P.x;
    R.lanes = (int32_t)(L.Kp / 4);
    Out O = {ws + L.codes, ws + L.scales, L.x_ld, 0, s.N, 0, L.groups};
    for (int64_t n = 0; n < s.N; n += L.rows) {
      const int64_t rows = s.N - n < L.rows ? s.N - n : L.rows;
      launch_rows<TILED>(s.hidden_dtype, R, O, rows, st);
      R.x += rows * R.x_ld;
      if (given) R.scale += rows * R.s_ld;
      O.codes += rows * O.c_ld;
      O.scale += rows * L.groups * 16;
    }
  }
  P.x_ld = L.x_ld;
  P.groups = (int32_t)L.groups;
  const bool direct = codes_direct(P.w_ld, (uintptr_t)weight_codes);
  const int64_t w_ld = P.w_ld, s_ld = P.s_ld, step = direct ? L.scaled : L.piece;
  const int oe = esize(s.out_dtype);
  for (int64_t v0 = 0; v0 < s.V; v0 += step) {
    P.V = (int32_t)(s.V - v0 < step ? s.V - v0 : step);
    if (direct) {
      P.w = weight_codes + v0 * w_ld;
      // a load's range is checked by whole dwords: the last one of a row counts if any of its
      // bytes does (aligned, so it lies in that byte's memory)
      P.w_bytes = up(code_bytes(s.H), 4);
    } else {
      copy_rows(weight_codes + v0 * w_ld, w_ld, code_bytes(s.H), (char *)ws + L.weight, L.x_ld, L.Kp, P.V, st);
      P.w = ws + L.weight;
      P.w_ld = L.x_ld;
      P.w_bytes = L.Kp;
    }
    const int64_t items = up(P.V, 256) / 4 * L.groups;
    hipLaunchKernelGGL(scales_kernel, dim3((unsigned)cdiv(items, 256)), dim3(256), 0, st, weight_scale + v0 * s_ld, s_ld,
                       (int64_t)P.V, (int)blocks(s.H), (int)L.groups, items, (u32x4 *)(ws + L.wscale));
    P.ws = ws + L.wscale;
    P.out = (char *)logits + v0 * oe;
    if (L.large) launch_tiles<Tile<8, 8, 2, 2, 2, 2>>(P, s.out_dtype, st);
    else launch_tiles<Tile<4, 4, 2, 2, 2, 2>>(P, s.out_dtype, st);
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
