// sv_logits8.hip -- 8-bit hidden rows (sv_act8_pack, sv_act8_unpack) and the
// vocabulary head in 8-bit integers (sv_head_logits), for gfx950 (MI355X).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "sv_act8.h"
#include "sv_device.h"
#include "sv_gemm.h"
#include "sv_head.h"
#include "sv_head_host.h"

namespace {

using namespace sv_gemm;
using sv_head_host::cdiv;

// codes * scale, in fp32, rounded once to the output's type: a wave takes a row,
// each lane the codes of a 16-byte store at a time, at any alignment.  HBM bound: 32768
// rows of 4096 into bf16 70 us (403 MB), of 4097 86, one code at a time 187.
template <int DT> __global__ __launch_bounds__(256) void unpack_kernel(const int8_t *codes, int64_t c_ld,
                                                                       const float *scale, char *y, int H, int N) {
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (n >= N) return;
  const int8_t *c = codes + n * c_ld;
  const float s = scale[n];
  constexpr int W = DT == SV_F32 ? 4 : 8;                // codes of a 16-byte store
  typedef uint32_t u32_any __attribute__((aligned(1)));
  u32x4_any *o = (u32x4_any *)(y + n * H * (16 / W));
  for (int q = lane; q < H / W; q += 64) {
    uint32_t w[2];
    if constexpr (W == 8) {
      const u32x2 u = __builtin_nontemporal_load((const u32x2_any *)c + q);
      w[0] = u[0];
      w[1] = u[1];
    } else {
      w[0] = __builtin_nontemporal_load((const u32_any *)c + q);
    }
    float v[W];
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] = (float)(int8_t)(w[k >> 2] >> (8 * (k & 3))) * s;
    u32x4 u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (W == 4) u[k] = __float_as_uint(v[k]);
      else
        u[k] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * k]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * k + 1]) << 16;
    }
    __builtin_nontemporal_store(u, o + q);
  }
  for (int k = H / W * W + lane; k < H; k += 64) {
    const float v = (float)c[k] * s;
    if constexpr (DT == SV_F32) ((float *)y)[n * H + k] = v;
    else ((__bf16 *)y)[n * H + k] = (__bf16)v;
  }
}

struct LogitsP {
  const char *x;                         // token codes, rows of whole steps
  int64_t x_ld;
  const float *sx;
  const char *w;                         // weight codes
  int64_t w_ld, w_bytes;
  const float *sw;
  char *out;
  int64_t out_ld;                        // elements
  int N, V, mt, nt, nk, band;
};

// One tile of logits.  The int32 sums are exact; three fp32 roundings follow, of the sum
// (beyond 2^24), of the two scales' product and of the product of both, and the output's.  1024 rows of 4096 x
// 128256 456 us, 2.36 POP/s (matrix instructions); 32 rows of 4096 x 151936 114 us, 5.5
// TB/s, and one of 1024 x 32000 6.4 us, 5.1 TB/s (reading the head).
template <class T, int OT> __global__ __launch_bounds__(T::TPB) void logits_kernel(LogitsP P) {
  __shared__ __align__(16) char lds[T::LDS];
  int im, in;
  tile_at(run_of_xcd(blockIdx.x, P.mt * P.nt), P.mt, P.nt, P.band, im, in);
  const int m0 = im * T::BM, n0 = in * T::BN;
  i32x4 acc[T::FM][T::FN];
  clear<SV_I8, T>(acc);
  const Part X = {P.x + (int64_t)m0 * P.x_ld, P.x_ld, P.N - m0 < T::BM ? P.N - m0 : T::BM, (int64_t)P.nk * STEP};
  const Part Y = {P.w + (int64_t)n0 * P.w_ld, P.w_ld, P.V - n0 < T::BN ? P.V - n0 : T::BN, P.w_bytes};
  product<SV_I8, T>(acc, lds, X, Y, 0, P.nk, T::BM < 256 ? in % P.nk : 0);
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, wm = wid / T::WN, wn = wid % T::WN;
  const Beside beside;
  float sw[T::FN][4];
#pragma unroll
  for (int g = 0; g < T::FN; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + (wn * T::FN + g) * 16 + (lane >> 4) * 4 + i;
      sw[g][i] = n < P.V ? P.sw[n] : 0.f;
    }
#pragma unroll
  for (int f = 0; f < T::FM; ++f) {
    const int m = m0 + (wm * T::FM + f) * 16 + (lane & 15);
    if (m >= P.N) continue;
    const float sx = P.sx[m];
    const int64_t row = (int64_t)m * P.out_ld;
    float v[T::FN][4];
#pragma unroll
    for (int g = 0; g < T::FN; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[g][i] = (float)acc[f][g][i] * (sx * sw[g][i]);
#pragma unroll
    for (int g = 0; g < T::FN; g += OT == SV_BF16 ? 2 : 1) {
      const int n = n0 + (wn * T::FN + g) * 16;
      if constexpr (OT == SV_BF16) {
        store8(P.out, row, n + beside.at, P.V, Beside::eight(v[g], v[g + 1]));
      } else {
        const int c = n + (lane >> 4) * 4;
        if (c + 4 <= P.V) {
          *(f32x4_any *)(P.out + (row + c) * 4) = f32x4{v[g][0], v[g][1], v[g][2], v[g][3]};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < P.V) ((float *)P.out)[row + c + i] = v[g][i];
        }
      }
    }
  }
}

template <class T> void launch_logits(LogitsP P, int ot, hipStream_t st) {
  P.mt = (int)cdiv(P.N, T::BM);
  P.nt = (int)cdiv(P.V, T::BN);
  P.band = 8;
  const dim3 grid((unsigned)((int64_t)P.mt * P.nt)), block(T::TPB);
  if (ot == SV_BF16) hipLaunchKernelGGL((logits_kernel<T, SV_BF16>), grid, block, 0, st, P);
  else hipLaunchKernelGGL((logits_kernel<T, SV_F32>), grid, block, 0, st, P);
}

}  // namespace

extern "C" int sv_act8_pack(int32_t N, int32_t H, int32_t dtype, const void *x, int64_t x_stride, int8_t *codes,
                            int64_t codes_stride, float *scale, void *stream) {
  const int rc = sv_head_host::check_act8(N, H, dtype, x, x_stride, codes, codes_stride, scale);
  if (rc != SV_OK || N == 0) return rc;
  sv_act8::Pack P = {(const char *)x, (x_stride ? x_stride : H) * (int64_t)sv_head_host::esize(dtype), codes,
                     codes_stride ? codes_stride : H, scale, H, H, 0};
  sv_act8::pack(dtype, N, P, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

extern "C" int sv_act8_unpack(int32_t N, int32_t H, const int8_t *codes, int64_t codes_stride, const float *scale,
                              int32_t y_dtype, void *y, void *stream) {
  const int rc = sv_head_host::check_act8(N, H, y_dtype, y, 0, codes, codes_stride, scale);
  if (rc != SV_OK || N == 0) return rc;
  const int64_t ld = codes_stride ? codes_stride : H;
  char *o = (char *)y;
  for (int64_t left = N; left > 0; left -= sv_head_host::MAX_ROWS) {
    const int n = (int)(left < sv_head_host::MAX_ROWS ? left : sv_head_host::MAX_ROWS);
    const dim3 grid((unsigned)cdiv(n, 4)), block(256);
    if (y_dtype == SV_BF16)
      hipLaunchKernelGGL((unpack_kernel<SV_BF16>), grid, block, 0, (hipStream_t)stream, codes, ld, scale, o, H, n);
    else
      hipLaunchKernelGGL((unpack_kernel<SV_F32>), grid, block, 0, (hipStream_t)stream, codes, ld, scale, o, H, n);
    codes += n * ld;
    scale += n;
    o += (int64_t)n * H * sv_head_host::esize(y_dtype);
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

extern "C" size_t sv_head_logits_workspace_bytes(const sv_logits_shape_t *s) {
  if (!s || !sv_head_host::logits_shape_ok(s)) return 0;
  return sv_head_host::logits_layout(s).total;
}

extern "C" int sv_head_logits(const sv_logits_shape_t *shape, const void *hidden, const float *hidden_scale,
                              const int8_t *weight_codes, const float *weight_scale, void *logits, void *workspace,
                              size_t workspace_bytes, void *stream) {
  bool nothing;
  const int rc = sv_head_host::check_logits(shape, hidden, hidden_scale, weight_codes, weight_scale, logits, workspace,
                                            workspace_bytes, &nothing);
  if (rc != SV_OK || nothing) return rc;
  const sv_logits_shape_t s = *shape;
  const hipStream_t st = (hipStream_t)stream;
  const sv_head_host::LogitsLayout L = sv_head_host::logits_layout(&s);
  char *ws = (char *)workspace;
  int8_t *codes = (int8_t *)(ws + L.codes);
  const int64_t hs = s.hidden_stride ? s.hidden_stride : s.H, wst = s.weight_stride ? s.weight_stride : s.H;
  const int64_t os = s.out_stride ? s.out_stride : s.V;
  const int oe = sv_head_host::esize(s.out_dtype);
  LogitsP P = {};
  P.x = (const char *)codes;
  P.x_ld = L.Kp;
  P.sx = (float *)(ws + L.scale);
  if (s.hidden_dtype == SV_I8) {
    copy_rows(hidden, hs, s.H, ws + L.codes, L.Kp, L.Kp, s.N, st);
    P.sx = hidden_scale;
  } else {
    sv_act8::Pack Q = {(const char *)hidden, hs * sv_head_host::esize(s.hidden_dtype), codes, L.Kp,
                       (float *)(ws + L.scale), s.H, (int32_t)L.Kp, 0};
    sv_act8::pack(s.hidden_dtype, s.N, Q, st);
  }
  P.N = s.N;
  P.nk = (int)(L.Kp / STEP);
  P.out_ld = os;
  const bool direct = sv_head_host::logits_direct(wst, (uintptr_t)weight_codes);
  const int64_t step = direct ? s.V : L.piece;
  for (int64_t v0 = 0; v0 < s.V; v0 += step) {
    P.V = (int)(s.V - v0 < step ? s.V - v0 : step);
    if (direct) {
      P.w = (const char *)weight_codes;
      P.w_ld = wst;
      // a load's range is checked by whole dwords: the last one of a row counts if
      // any of its bytes does (aligned, so it lies in that byte's memory); the token
      // codes are 0 past H, so what else it holds adds nothing
      P.w_bytes = sv_head_host::up(s.H, 4);
    } else {
      copy_rows(weight_codes + v0 * wst, wst, s.H, ws + L.weight, L.Kp, L.Kp, P.V, st);
      P.w = ws + L.weight;
      P.w_ld = P.w_bytes = L.Kp;
    }
    P.sw = weight_scale + v0;
    P.out = (char *)logits + v0 * oe;
    // up to 32 rows 32 x 128: the rest of a taller tile would be multiplied in vain (24 rows
    // of 4096 x 151936 147 to 119 us; 33 to 64 rows in two of them 142 to 152 against 130)
    if (sv_head_host::large_tiles(s.N, s.V)) launch_logits<Tile<8, 4, 2, 4>>(P, s.out_dtype, st);
    else if (s.N > 32) launch_logits<Tile<4, 4, 2, 2>>(P, s.out_dtype, st);
    else launch_logits<Tile<2, 2, 1, 4, 3, 3>>(P, s.out_dtype, st);
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
