// sv_gemm.h -- the tiled matrix product behind the vocabulary-head operators,
// for gfx950 (MI355X): C[m][n] = sum_k X(m, k) Y(n, k) in bf16, fp32 or int8.
// Each operand lies with k along its rows ("rows": X[m][k]), with k down its columns
// ("columns": X[k][m]), or in 16-byte blocks of k of one m ("blocks": X[k / 8][m][8]
// in bf16, X[k / 4][m][4] in fp32), so the gradients' products read the weight as it
// lies and nothing is transposed in memory.
//
// One core for the three types: a step takes 128 bytes of k (64 bf16, 32 fp32,
// 128 int8) of both tiles, and a matrix instruction takes from each lane 16
// bytes of k of one m or n: lane l holds index l & 15 and 16-byte piece l >> 4 of
// a 64-byte half step.  Which k those bytes are does not matter as long as both
// operands agree, so the types differ in one instruction (four for fp32, whose
// instruction takes one element a lane) and in how columns are read.
//
// Tiles go from memory to LDS by direct 16-byte loads (no registers between).  A wave
// holds two sets of fragments: while the matrix instructions work on one half step,
// the next half step's fragments are read.  The one barrier of a step stands in its
// middle: by then every wave has read all of the step's buffers, which later loads may
// overwrite, and the next step's tiles have landed.  Loads land in order, so how long
// they may take is the smaller number of an operand's buffers, less one, in steps: the
// large tiles have room for two and three (the columns' operand comes from farther),
// and three of both pay for a few tokens against 8-bit weights, which only read (one
// token of 4096 x 151936 120 to 111 us; four no more).
//
// A direct load writes 64 consecutive 16-byte pieces, so pieces are permuted on
// the memory side to keep LDS reads off each other's banks.  Rows: piece p of row
// r lies at place p ^ (r & 7), and the 8 rows read together hit 8 places.
// Columns: a lane reads, for each of its k, the neighbouring columns that its F
// fragments hold (fragment f's index i is column i F + f), and bf16 pairs of k are
// put together by byte permutes; the parts of k read together are turned against
// each other.  Blocks: a piece is a lane's, as with rows.  (The LDS read that
// transposes by itself does not serve: the compiler lets it wait for every load into
// LDS, those for later steps among them; dW ran at 1.0 PFLOP/s with it, measured at
// 2048 x 4096 x 65536.)
// The columns' fragment is the instruction's first operand: a lane then holds
// four n of one m; index_of tells which.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sv_head.h"
#include "sv_head_host.h"

namespace sv_gemm {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// at any address (the GPU takes such accesses; on elements' addresses they are as fast)
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef f32x4 f32x4_any __attribute__((aligned(1)));

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

// A workgroup's tile: WM x WN waves, each of FM x FN fragments of 16 x 16; XB and YB
// buffers of the operands (2 and 3, or as many of both).
template <int FM_, int FN_, int WM_, int WN_, int XB_ = 2, int YB_ = 3> struct Tile {
  static constexpr int FM = FM_, FN = FN_, WM = WM_, WN = WN_, XB = XB_, YB = YB_;
  static_assert(XB == YB || (XB == 2 && YB == 3), "buffers");
  static constexpr int NW = WM * WN, TPB = 64 * NW;
  static constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  static constexpr int XBUF = BM * STEP, YBUF = BN * STEP;   // bytes of one LDS buffer
  static constexpr int LDS = XB * XBUF + YB * YBUF;
};

// One tile's part of an operand.
//   rows:    base at the tile's first row; `count` rows exist (>= 1; rows past them
//            repeat the last one, their products are not used)
//   columns: base at the tile's first column of k = 0; `count` k exist, at least
//            one in each step taken (later ones repeat the last: the other operand
//            holds zeros there)
// ld: bytes between rows (of m or of k); bytes: what exists of a row from base.
struct Part {
  const char *base;
  int64_t ld;
  int64_t count;
  int64_t bytes;
};

// How an operand lies in memory.  For blocks a row is one of blocks: ld and bytes are
// its, count counts blocks of k.
enum Lie { ROWS, COLS, BLOCKS };

#ifdef __HIP_DEVICE_COMPILE__            // (the host pass knows no gfx950 builtins)
// Loads and reads of one operand's tile: R indices (m or n), F fragments a wave.
template <int DT, int R, int F, int NW, Lie LIE> struct Side {
  static constexpr bool COL = LIE != ROWS;               // k down the memory's rows
  static constexpr int E = LIE == BLOCKS ? 16 : Mma<DT>::E, KR = STEP / E;   // bytes of an entry, entries of k a step
  static constexpr int NL = R / 8 / NW;                  // 16-byte loads a thread and step
  static_assert(NL >= 1 && NL < 16 && R % (8 * NW) == 0, "tile of whole loads");
  static constexpr int PR = COL ? R * E / 16 : 8;        // pieces of an LDS row
  // columns: k of a lane's 16 bytes, bytes that 16 lanes read of one k, and how
  // many such parts are read together
  static constexpr int KL = 16 / E, SPAN = 16 * F * E, PARTS = SPAN >= 256 ? 1 : 256 / SPAN;
  static_assert(LIE != COLS || (E > 1 && (F == 2 || F == 4 || F == 8)), "whole reads of columns");
  typedef __attribute__((address_space(3))) void lds_void;

  __amdgpu_buffer_rsrc_t rsrc;
  const char *base;
  int64_t ld, left, bytes;
  int off[NL];                                           // a load's byte offset from its step
  int wid;

  // the byte in its row that LDS piece q of k r holds
  static __device__ __forceinline__ int piece(int q, int r) { return q * 16 ^ (r / KL & (PARTS - 1)) * SPAN; }
  // steps from s0 whose k all exist
  __device__ __forceinline__ int whole(int nk) const {
    if constexpr (COL) return left / KR < nk ? (int)(left / KR) : nk;
    else return nk;
  }

  int pos, end;                                          // rows: the next step's byte, and the line's end

  // from step s0 on; rows: `from` steps later, in a circle of nk
  __device__ __forceinline__ void start(const Part &p, int s0, int nk, int from) {
    pos = (s0 + from) * STEP;
    end = (s0 + nk) * STEP;
    wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    ld = p.ld;
    bytes = p.bytes;
    if constexpr (COL) {
      base = p.base + (int64_t)s0 * KR * ld;
      left = p.count - (int64_t)s0 * KR;
    } else {
      base = p.base;
      left = p.count;
      // no load leaves the rows that exist: the resource ends with the last one
      rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)((left - 1) * ld + bytes), 0x00020000);
    }
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      const int c = (wid + j * NW) * 64 + (threadIdx.x & 63), r = c / PR, q = c % PR;
      if constexpr (COL) off[j] = r * (int)ld + piece(q, r);
      else off[j] = (int)((r < left ? r : left - 1) * ld) + (q ^ (r & 7)) * 16;
    }
  }
  // the next step's loads; all: every k of it exists
  __device__ __forceinline__ void issue(char *buf, bool all, int nk) {
    if constexpr (COL) {
      const int have = all || left >= KR ? KR : (int)left;
      rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)((have - 1) * ld + bytes), 0x00020000);
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        int o = off[j];
        if (!all) {
          int c = (wid + j * NW) * 64 + (threadIdx.x & 63);
          asm volatile("" : "+v"(c));    // (formed again in the few steps that need it, not held)
          const int r = c / PR;
          if (r >= have) o -= (r - (have - 1)) * (int)ld;
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(buf + (wid + j * NW) * 1024), 16, o, 0, 0, 0);
      }
      base += KR * ld;
      left -= KR;
    } else {
#pragma unroll
      for (int j = 0; j < NL; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(buf + (wid + j * NW) * 1024), 16, off[j], pos, 0, 0);
      pos = pos + STEP == end ? end - nk * STEP : pos + STEP;
    }
  }
  // rows: the next step's load j alone, and the step after it
  __device__ __forceinline__ void issue_one(char *buf, int j) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(buf + (wid + j * NW) * 1024), 16, off[j], pos, 0, 0);
  }
  __device__ __forceinline__ void next(int nk) { pos = pos + STEP == end ? end - nk * STEP : pos + STEP; }
  // rows: from here on loads read nothing and put zeros
  __device__ __forceinline__ void stop() { rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, 0, 0x00020000); }
  static constexpr int READS = LIE == COLS ? KL : F;
  // what the wave's fragments g0 .. g0 + F - 1 (of 16 indices) of half step h hold,
  // for columns in the order of k
  static __device__ __forceinline__ void read(u32x4 (&v)[F], const char *buf, int g0, int h) {
    const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
    if constexpr (!COL) {
      const char *at = buf + g0 * 16 * STEP + i * STEP + (((h * 4 + q) ^ (lane & 7)) << 4);
#pragma unroll
      for (int f = 0; f < F; ++f) v[f] = *(const u32x4 *)(at + f * 16 * STEP);
    } else if constexpr (LIE == BLOCKS) {
      const char *at = buf + (h * 4 + q) * (R * 16) + (g0 * 16 + i) * 16;
#pragma unroll
      for (int f = 0; f < F; ++f) v[f] = *(const u32x4 *)(at + f * 256);
    } else {
      constexpr int B = F * E;                           // bytes a lane reads of one k
      const char *at = buf + (h * 4 + q) * KL * (R * E) + ((g0 * 16 * E + i * B) ^ (q & (PARTS - 1)) * SPAN);
#pragma unroll
      for (int e = 0; e < KL; ++e) {
        const char *p = at + e * (R * E);
        if constexpr (B == 16) {
          v[e] = *(const u32x4 *)p;
        } else if constexpr (B == 8) {
          const u32x2 w = *(const u32x2 *)p;
          v[e / 2][e % 2 * 2] = w[0];
          v[e / 2][e % 2 * 2 + 1] = w[1];
        } else {
          v[e / 4][e % 4] = *(const uint32_t *)p;
        }
      }
    }
  }
  // fragments from what was read
  static __device__ __forceinline__ void finish(u32x4 (&v)[F]) {
    if constexpr (LIE == COLS) {
      constexpr int WORDS = F * E / 4;                   // words read of one k
      u32x4 o[F];
#pragma unroll
      for (int w = 0; w < WORDS; ++w)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          if constexpr (DT == SV_BF16) {
            const uint32_t a = v[(2 * d * WORDS + w) >> 2][(2 * d * WORDS + w) & 3];
            const uint32_t b = v[((2 * d + 1) * WORDS + w) >> 2][((2 * d + 1) * WORDS + w) & 3];
            o[2 * w][d] = __builtin_amdgcn_perm(b, a, 0x05040100);
            o[2 * w + 1][d] = __builtin_amdgcn_perm(b, a, 0x07060302);
          } else {
            o[w][d] = v[(d * WORDS + w) >> 2][(d * WORDS + w) & 3];
          }
        }
#pragma unroll
      for (int f = 0; f < F; ++f) v[f] = o[f];
    }
  }
};
#endif

#ifdef __HIP_DEVICE_COMPILE__
// The order of a half step's instructions: MM matrix instructions with LD loads,
// then RD LDS reads, spread evenly between them.
template <int MM, int RD, int LD> __device__ __forceinline__ void mix() {
  constexpr int N = RD + LD, K = MM / N > 0 ? MM / N : 1;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, K, 0);
    if (i < LD) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  if constexpr (MM > N * K) __builtin_amdgcn_sched_group_barrier(0x008, MM - N * K, 0);
}
#endif

#ifdef __HIP_DEVICE_COMPILE__
// This wave's LDS reads are done, and its loads but for the last g groups of NL
// (g at most G).
template <int G, int NL> __device__ __forceinline__ void wait_loads(int g) {
  if constexpr (G == 0) {
    __builtin_amdgcn_s_waitcnt(0x0070);                  // vmcnt(0) lgkmcnt(0)
  } else {
    static_assert(G * NL < 64, "the counter's range");
    if (g >= G) __builtin_amdgcn_s_waitcnt(0x0070 | ((G * NL) & 15) | ((G * NL) >> 4) << 14);
    else wait_loads<G - 1, NL>(g);
  }
}
#endif

// The products of one tile over steps [s0, s0 + nk); from: the step of them to begin
// with, where both operands are rows.  Rows a power of two apart lie on few memory
// channels at any one step, so where reading the columns' operand is the bound, tiles
// begin at different steps (int8 rows of 4096 bytes: 4.3 to 5.2 TB/s; where the matrix
// units are the bound it changes nothing).
template <int DT, class T, Lie XC = ROWS, Lie YC = ROWS>
__device__ __forceinline__ void product(typename Mma<DT>::Acc (&acc)[T::FM][T::FN], char *lds, const Part &X,
                                        const Part &Y, int s0, int nk, int from = 0) {
#ifdef __HIP_DEVICE_COMPILE__
  typedef Side<DT, T::BM, T::FM, T::NW, XC> SX;
  typedef Side<DT, T::BN, T::FN, T::NW, YC> SY;
  if (nk <= 0) return;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int gx = wid / T::WN * T::FM, gy = wid % T::WN * T::FN;
  SX sx;
  SY sy;
  sx.start(X, s0, nk, from);
  sy.start(Y, s0, nk, from);
  constexpr bool EVEN = T::XB == T::YB;                  // as many buffers of both
  constexpr int B = T::YB;
  char *const yl = lds + T::XB * T::XBUF;
  u32x4 x0[T::FM], y0[T::FN], x1[T::FM], y1[T::FN];
  auto read = [&](u32x4 (&x)[T::FM], u32x4 (&y)[T::FN], int s, int b, int h) {
    SX::read(x, lds + (EVEN ? b : s & 1) * T::XBUF, gx, h);
    SY::read(y, yl + b * T::YBUF, gy, h);
  };
  // One barrier: this wave's LDS reads are done and its loads have landed, but for g
  // groups of later steps: even buffers, of both operands' loads of a step; else of the
  // columns' loads of the step after next.  Written out, because a fence would wait for
  // those too; the empty asm keeps the compiler's accesses on their side.
  constexpr int NL = EVEN ? SX::NL + SY::NL : SY::NL;
  auto landed = [&](auto most, int g) {
    asm volatile("" ::: "memory");
    wait_loads<decltype(most)::value, NL>(g);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  typedef std::integral_constant<int, EVEN ? B - 2 : 1> Later;
  typedef typename Mma<DT>::Acc Acc;
  auto mul = [&](Acc (&c)[T::FM][T::FN], u32x4 (&x)[T::FM], u32x4 (&y)[T::FN]) {
    SX::finish(x);
    SY::finish(y);
#pragma unroll
    for (int f = 0; f < T::FM; ++f)
#pragma unroll
      for (int g = 0; g < T::FN; ++g) Mma<DT>::mul(c[f][g], y[g], x[f]);
  };
  const int wx = sx.whole(nk), wy = sy.whole(nk), full = wx < wy ? wx : wy;
  if constexpr (EVEN) {
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (j < nk) {
        sx.issue(lds + j * T::XBUF, false, nk);
        sy.issue(yl + j * T::YBUF, false, nk);
      }
    landed(std::integral_constant<int, B - 1>(), nk - 1);
  } else {
    sx.issue(lds, false, nk);
    sy.issue(yl, false, nk);
    if (nk > 1) sy.issue(yl + T::YBUF, false, nk);
    landed(Later(), nk - 1);
    if (nk > 1) sx.issue(lds + T::XBUF, false, nk);
    if (nk > 2) sy.issue(yl + 2 * T::YBUF, false, nk);
  }
  read(x0, y0, 0, 0, 0);
  int b = 0;                                             // this step's buffer
  // One step.  Loads and LDS reads are spread between the matrix instructions: a
  // wave issues in order, and eight waves that all ask for their fragments first
  // keep the matrix units waiting for the LDS.
  constexpr int MM = T::FM * T::FN * (DT == SV_F32 ? 4 : 1);
  constexpr int RD = SX::READS + SY::READS, LD = SX::NL + SY::NL;
  auto step = [&](int s, Acc (&c)[T::FM][T::FN], auto whole) {
    constexpr bool W = decltype(whole)::value;           // B more whole steps follow
    read(x1, y1, s, b, 1);
    mul(c, x0, y0);
    mix<MM, RD, 0>();
    landed(Later(), W ? B : nk - 2 - s);
    if (W || s + T::XB < nk) sx.issue(lds + (EVEN ? b : s & 1) * T::XBUF, W, nk);
    if (W || s + B < nk) sy.issue(yl + b * T::YBUF, W, nk);
    b = b == B - 1 ? 0 : b + 1;
    if (W || s + 1 < nk) read(x0, y0, s + 1, b, 0);
    mul(c, x1, y1);
    if constexpr (W) mix<MM, RD, LD>();
  };
  auto sum = [&](int s, auto whole) {
    if constexpr (DT == SV_F32) {
      // fp32 sums are kept in two levels, 32 terms and then the steps: the error of
      // a long sum grows with the number of steps, not of terms
      Acc part[T::FM][T::FN];
#pragma unroll
      for (int f = 0; f < T::FM; ++f)
#pragma unroll
        for (int g = 0; g < T::FN; ++g) part[f][g] = 0;
      step(s, part, whole);
#pragma unroll
      for (int f = 0; f < T::FM; ++f)
#pragma unroll
        for (int g = 0; g < T::FN; ++g) acc[f][g] += part[f][g];
    } else {
      step(s, acc, whole);
    }
  };
  int s = 0;
  for (; s + B < full; ++s) sum(s, std::true_type());
  for (; s < nk; ++s) sum(s, std::false_type());
#endif
}

// The index in its tile of index i (0 .. 15) of fragment f of wave w.
template <int F, Lie LIE> __device__ __forceinline__ int index_of(int w, int f, int i) {
  return LIE == COLS ? (w * 16 + i) * F + f : (w * F + f) * 16 + i;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16;
}

// columns n .. n + 7 of a row of N bf16, wherever they begin
__device__ __forceinline__ void store8(char *p, int64_t row, int n, int N, u32x4 v) {
  if (n + 8 <= N) {
    *(u32x4_any *)(p + (row + n) * 2) = v;
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (n + r < N) ((uint16_t *)p)[row + n + r] = (uint16_t)(v[r / 2] >> (r % 2 * 16));
  }
}

// bf16 results of two neighbouring fragments, four columns a lane of each, as eight
// neighbouring columns a lane: the lanes 16 apart that hold a row swap halves, so that
// a row's store is 64 bytes together instead of 32 (8-bit logits of 1024 rows of 4096 x
// 128256 557 to 457 us, dW of 4096 rows 3050 to 2935).  at: the first of a lane's
// columns, from the first fragment's first.
struct Beside {
  int at;
  __device__ __forceinline__ Beside() {
    const int q = (threadIdx.x & 63) >> 4;
    at = (q & 1) * 16 + (q >> 1) * 8;
  }
  static __device__ __forceinline__ u32x4 eight(const float (&g)[4], const float (&h)[4]) {
#ifdef __HIP_DEVICE_COMPILE__
    const auto a = __builtin_amdgcn_permlane16_swap(pack2(g[0], g[1]), pack2(h[0], h[1]), false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(pack2(g[2], g[3]), pack2(h[2], h[3]), false, false);
    return u32x4{a[0], b[0], a[1], b[1]};
#else
    return u32x4{};
#endif
  }
};

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

// Rows of `bytes` bytes that the products cannot read where they lie, at any
// alignment, into rows of whole steps with zeros behind them: 16 bytes a lane, as
// many lanes a row (1 << lg) as share it out evenly (53559 rows of 144 bytes 16 to
// 9 us, 50000 of 2000 bytes 70 to 38 us, against a workgroup a row and an element a lane).
static __global__ __launch_bounds__(256) void copy_rows_kernel(const char *src, int64_t ld, int64_t bytes, char *dst,
                                                               int64_t d_ld, int chunks, int rows, int lg) {
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg;
  if (row >= rows) return;
  const char *s = src + row * ld;
  char *d = dst + row * d_ld;
  for (int c = threadIdx.x & ((1 << lg) - 1); c < chunks; c += 1 << lg) {
    const int64_t at = (int64_t)c * 16;
    u32x4 v = 0;
    if (at + 16 <= bytes) {
      v = *(const u32x4_any *)(s + at);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (at + i < bytes) v[i / 4] |= (uint32_t)(uint8_t)s[at + i] << (i % 4 * 8);
    }
    *(u32x4 *)(d + at) = v;
  }
}

static inline void copy_rows(const void *src, int64_t ld, int64_t bytes, char *dst, int64_t d_ld, int64_t d_bytes,
                             int64_t rows, hipStream_t st) {
  const int chunks = (int)(d_bytes / 16);
  int lg = 3;                                            // (whole steps: 8 chunks or more)
  while (lg < 6 && (1 << lg) < chunks) ++lg;
  for (int64_t r = 0; r < rows; r += sv_head_host::MAX_ROWS) {
    const int64_t n = rows - r < sv_head_host::MAX_ROWS ? rows - r : sv_head_host::MAX_ROWS;
    hipLaunchKernelGGL(copy_rows_kernel, dim3((unsigned)((n + (256 >> lg) - 1) / (256 >> lg))), dim3(256), 0, st,
                       (const char *)src + r * ld, ld, bytes, dst + r * d_ld, d_ld, chunks, (int)n, lg);
  }
}

}  // namespace sv_gemm
