// sv_head.hip -- cross entropy and top-32 distillation from hidden rows under a
// vocabulary head, with the gradients of rows and head, for gfx950 (MI355X).
//
// With z = (1/T) x W^T, lse = ln sum exp z and u the row's weight,
//   loss = sum u (lse - z_t)              (or sum u KL over the stored 32)
//   dz = u (exp(z - lse) - pt),  dx = (1/T) dz W,  dW = (1/T) dz^T x.
// The logits are never stored.  Forward: one product whose tiles keep only each
// row's maximum and sum of exps; a small gather forms the z of the targets.
// Backward: a piece of the vocabulary at a time, the product again, its tiles
// turned into dz in the operands' type, then two products with dz.  A piece is
// complete for dW and adds to dx in fp32.  That is four products for the three
// that stored logits would need, and memory for a piece in place of N x V.
//
// Rows are put in an order first: those with a gradient, then those with a loss
// only, then those left out (ignored or with bad inputs); each product covers
// its front part and stops there, so padding and prompt positions cost nothing.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "sv_device.h"
#include "sv_gemm.h"
#include "sv_head.h"
#include "sv_head_host.h"
#include "sv_kd.h"

namespace {

using namespace sv_gemm;
using sv_dev::NEG_INF;
using sv_dev::wave_max_f;
using sv_dev::wave_or;
using sv_dev::wave_sum_d;
using sv_dev::wave_sum_f;
using sv_head_host::cdiv;
using sv_head_host::Plan;
using sv_head_host::TOP;

constexpr float LOG2E = 1.44269504f;
constexpr double LN2 = 0.6931471805599453;
// A logit from its exponent z * LOG2E.  LOG2E is low by 1.3e-8 of itself; ln 2 in place of
// this would leave that in lse alone (a sure row of z = 1000: nll -1.3e-5).
constexpr double PER_LOG2E = 1.0 / (double)LOG2E;

template <int DT> __device__ __forceinline__ float load_real(const char *p, int64_t i) {
  if constexpr (DT == SV_BF16) return __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16);
  else if constexpr (DT == SV_F32) return ((const float *)p)[i];
  else return (float)((const int8_t *)p)[i];
}
template <int DT> __device__ __forceinline__ void store_real(char *p, int64_t i, float v) {
  if constexpr (DT == SV_BF16) ((__bf16 *)p)[i] = (__bf16)v;
  else ((float *)p)[i] = v;
}
// four consecutive elements, wherever they begin (40 rows of 1001 x 50000 in fp32: dW
// 132 to 83 us against a store an element)
template <int DT> __device__ __forceinline__ void store4(char *p, int64_t i, const float (&v)[4]) {
  if constexpr (DT == SV_BF16) *(u32x2_any *)(p + i * 2) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
  else *(f32x4_any *)(p + i * 4) = f32x4{v[0], v[1], v[2], v[3]};
}

// A lane's results of a row where the columns' operand lies k down its columns: F
// fragments hold 4 F neighbouring columns from n (index_of), v[g][i] column n + i F + g.
template <int DT, int F>
__device__ __forceinline__ void store_columns(char *p, int64_t row, int n, int N, const f32x4 (&v)[F]) {
#pragma unroll
  for (int q = 0; q < F; ++q) {
    float d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = v[(4 * q + i) % F][(4 * q + i) / F];
    const int c = n + 4 * q;
    if (c + 4 <= N) store4<DT>(p, row + c, d);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < N) store_real<DT>(p, row + c + i, d[i]);
  }
}

// Up to PAIR rows in bf16 take half a step of dW's sum and half a tile of dx's, whose
// times are the head's and dW's bytes anyway: the other halves hold what dz's rounding to
// bf16 leaves, in rows PAIR further on.  Few rows' gradients hang on few entries of dz,
// whose roundings do not average: 24 rows of 1024 x 20000, distillation, an error of 0.0023
// to 0.0026 of the norm with one term, 0.0017 with two, which is the results' own
// rounding; 3 us of 66, and 24 rows of 4096 x 151936 no more at all.
//
// At more rows the caller may ask for the second term (SV_GRAD_TWO_TERMS), for a second
// product of each gradient: its rows lie behind all rows of the first term for dx,
// which takes them in a product of their own, and behind those with a gradient, in whole
// steps, for dW, whose sum runs over both and whose rows of x are there twice.
constexpr int PAIR = 32;
__device__ __forceinline__ float rest_of(float d) { return d - (float)(__bf16)d; }

// What the kernels share: the call's arrays and the workspace.
struct Head {
  int32_t N, H, V, T;                    // T: targets per row
  int32_t grads;
  int32_t ignore;
  float inv_t;
  int64_t Kp, Np;
  int64_t x_ld, dz_ld;                   // bytes between rows of xs, of dz
  int64_t xw_ld, dzw_ld;                 // bytes between rows of blocks
  int32_t keep;                          // the forward product leaves its logits in dz (fp32, one piece)
  int32_t split;                         // dz in two bf16 terms (PAIR)
  int32_t terms;                         // 2: dz in two bf16 terms, in rows of their own
  const char *hidden;
  int64_t h_ld;                          // bytes
  const float *h_scale;
  const char *weight;
  int64_t w_ld;                          // bytes
  // cross entropy
  const int32_t *targets;
  const float *row_weight;
  // distillation
  const float *tval;
  const int32_t *tidx, *row_sample;
  const float *rewards;
  int32_t S, G;
  float w_max;
  // results
  float *rows, *lse, *weight_out, *loss;
  int32_t *status;
  char *gh, *gw;
  // workspace (per place in the order unless said otherwise)
  int32_t *counts;                       // rows with a gradient, rows with a loss
  int32_t *perm;                         // the row at a place
  float *alpha;                          // factor of the product: scale / T
  float *ga;                             // factor of dz: u / T and the normaliser's part beyond fp32
  float *lse2;                           // base-2 normaliser, rounded; the rest of it is in ga
  float *w;                              // per row: u (distillation)
  int32_t *flags;                        // per row: data-error bits (distillation)
  float *zt;                             // [.., T] logits of the targets
  float *pt;                             // [.., T] their probabilities (distillation)
  double *term;                          // loss terms
  float2 *part;                          // [column tiles][N] base-2 maximum and sum of exps
  char *xs;                              // rows with a loss
  char *dz;                              // a piece's dz, rows for dx
  char *dzw;                             // the same, times the rows' scales (8-bit rows), in blocks for dW
  char *xw;                              // rows with a gradient in blocks for dW
  char *wt;                              // a copied piece of the weight
  float *acc;                            // sums of dx, per workgroup and tile
};

// ---------------------------------------------------------------- rows' inputs
// The distillation's weight and data errors of a row: one wave per row (a launch's
// time: 4.5 us at 24 rows, 6.4 at 4096).
__global__ __launch_bounds__(256) void kd_rows_kernel(Head P) {
  const int lane = threadIdx.x & 63;
  const int n = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (n >= P.N) return;
  const int s = P.row_sample[n];
  const bool badw = s < 0 || s >= P.S;
  double w = 0.0;
  if (!badw) {
    const int g0 = s / P.G * P.G;
    double sum = 0.0;
    for (int l = 0; l < P.G; l += 64) sum += wave_sum_d(l + lane < P.G ? (double)P.rewards[g0 + l + lane] : 0.0);
    w = sum > 0.0 ? (double)P.rewards[s] / sum : 0.0;
    w = w > 0.0 ? w : 0.0;               // negative and NaN weights count as 0
    w = w < (double)P.w_max ? w : (double)P.w_max;
  }
  const float v = lane < TOP ? P.tval[(int64_t)n * TOP + lane] : NEG_INF;
  const int x = lane < TOP ? P.tidx[(int64_t)n * TOP + lane] : -1;
  const bool pad = v == NEG_INF || x == -1;
  int F = 0;
  if (!pad && (x < 0 || x >= P.V)) F |= SV_KD_BAD_INDEX;
  if (lane < TOP && !(v == v)) F |= SV_KD_NAN;
  if (lane < TOP && v == __builtin_inff()) F |= SV_KD_POSINF;
  const int mine = pad ? -1 : x, in = (!pad && x >= 0 && x < P.V) ? x : -1;
  bool dup = false;
  for (int e = 0; e < TOP; ++e) dup |= e < lane && in >= 0 && __builtin_amdgcn_readlane(mine, e) == in;
  if (dup) F |= SV_KD_DUP_INDEX;
  F = wave_or(F) | (badw ? SV_KD_BAD_INDEX : 0);
  if (!F && wave_max_f(pad ? NEG_INF : v) == NEG_INF) F = SV_KD_EMPTY;
  if (lane == 0) {
    P.w[n] = (float)w;
    P.flags[n] = F;
    if (P.weight_out) P.weight_out[n] = (float)w;
  }
}

// 0: a gradient, 1: a loss only, 2: left out
template <bool KD> __device__ __forceinline__ int class_of(const Head &P, int n, int &bits) {
  bits = 0;
  if constexpr (KD) {
    bits = P.flags[n];
    return (P.grads && !bits && P.w[n] > 0.f) ? 0 : 1;
  } else {
    const int t = P.targets[n];
    if (t == P.ignore) return 2;
    if (t < 0 || t >= P.V) bits |= SV_HEAD_BAD_TARGET;
    const float w = P.row_weight ? P.row_weight[n] : 1.f;
    if (!(fabsf(w) < __builtin_inff())) bits |= SV_HEAD_BAD_WEIGHT;
    if (bits) return 2;
    return (P.grads && w != 0.f) ? 0 : 1;
  }
}

// The results of a row that is left out.
__device__ __forceinline__ void left_out(const Head &P, int n, int bits) {
  const float r = bits ? __builtin_nanf("") : 0.f;
  P.rows[n] = r;
  if (P.lse) P.lse[n] = r;
  if (P.status) P.status[n] = bits;
}

// The order of rows: by class, by index within a class.  One workgroup; two
// passes over N small entries (12 us at 4096 rows).
template <bool KD> __global__ __launch_bounds__(1024) void order_kernel(Head P) {
  __shared__ int cnt[3][16];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  int c[3] = {0, 0, 0};
  for (int n = tid; n < P.N; n += 1024) {
    int bits;
    const int k = class_of<KD>(P, n, bits);
#pragma unroll
    for (int q = 0; q < 3; ++q) c[q] += k == q;
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const int s = sv_dev::wave_sum_i(c[q]);
    if (lane == 0) cnt[q][wid] = s;
  }
  __syncthreads();
  int base[3] = {0, 0, 0}, tot[3] = {0, 0, 0};
  for (int w = 0; w < 16; ++w)
#pragma unroll
    for (int q = 0; q < 3; ++q) tot[q] += cnt[q][w];
  base[1] = tot[0];
  base[2] = tot[0] + tot[1];
  if (tid == 0) { P.counts[0] = tot[0]; P.counts[1] = tot[0] + tot[1]; }
  for (int n0 = 0; n0 < P.N; n0 += 1024) {
    const int n = n0 + tid;
    int bits = 0;
    const int k = n < P.N ? class_of<KD>(P, n, bits) : 3;
    int at = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const uint64_t b = __ballot(k == q);
      if (k == q) at = __popcll(b & ((1ull << lane) - 1));
      if (lane == 0) cnt[q][wid] = __popcll(b);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      int before = 0, all = 0;
      for (int w = 0; w < 16; ++w) { before += w < wid ? cnt[q][w] : 0; all += cnt[q][w]; }
      if (k == q) P.perm[base[q] + before + at] = n;
      base[q] += all;
    }
    if (k == 2) left_out(P, n, bits);
  }
}

// Rows with a loss, in order, in the operands' type, zeros up to whole steps; for the
// distillation also z of the stored entries (fp32 sums, an entry a wave).  8-bit codes
// are exact in bf16 and fp32; their scale goes into alpha.  FIND: a workgroup per row
// that finds its place itself, for batches of at most FIND_ROWS rows (each looks at
// all of them), which saves the order's launch.  Bound by reading: 4096 rows of 4096 in
// bf16 26 us; with the stored entries' logits 32 rows of the head a row, 4096 of 2048
// 109 us (537 MB, 4.9 TB/s).
constexpr int FIND_ROWS = 1024;

template <int HT, int DT, bool KD, bool FIND>
__global__ __launch_bounds__(KD ? 1024 : 256) void stage_rows_kernel(Head P) {
  constexpr int TPB = KD ? 1024 : 256, NW = TPB / 64;
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  int at = blockIdx.x, n = at;
  if constexpr (FIND) {
    __shared__ int cnt[NW][3];
    int bits, c[3] = {0, 0, 0};          // rows before this one, rows of class 0, of class 1
    const int k = class_of<KD>(P, n, bits);
    for (int i = tid; i < P.N; i += TPB) {
      int other;
      const int q = class_of<KD>(P, i, other);
      c[0] += q < k || (q == k && i < n);
      c[1] += q == 0;
      c[2] += q == 1;
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      c[q] = sv_dev::wave_sum_i(c[q]);
      if (lane == 0) cnt[wid][q] = c[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      c[q] = 0;
      for (int w = 0; w < NW; ++w) c[q] += cnt[w][q];
    }
    at = c[0];
    if (tid == 0) {
      P.perm[at] = n;
      if (n == 0) { P.counts[0] = c[1]; P.counts[1] = c[1] + c[2]; }
      if (k == 2) left_out(P, n, bits);
    }
    if (k == 2) return;
  } else {
    if (at >= P.counts[1]) return;
    n = P.perm[at];
  }
  const char *src = P.hidden + (int64_t)n * P.h_ld;
  char *dst = P.xs + (int64_t)at * P.x_ld;
  for (int k = tid; k < (int)P.Kp; k += TPB) store_real<DT>(dst, k, k < P.H ? load_real<HT>(src, k) : 0.f);
  const float alpha = HT == SV_I8 ? P.h_scale[n] * P.inv_t : P.inv_t;
  if (tid == 0) P.alpha[at] = alpha;
  if constexpr (KD) {
    __syncthreads();                     // the row as stored, for every wave
    constexpr int E = Mma<DT>::E, W = 16 / E;
    const int nv = P.H / W;
    for (int j = wid; j < TOP; j += NW) {
      const int id = P.tidx[(int64_t)n * TOP + j];
      float s = 0.f;
      if (id >= 0 && id < P.V) {
        const char *w = P.weight + (int64_t)id * P.w_ld;
        for (int q = lane; q < nv; q += 64) {
          const u32x4 a = *(const u32x4 *)(dst + (int64_t)q * 16), b = *(const u32x4_any *)(w + (int64_t)q * 16);
#pragma unroll
          for (int e = 0; e < W; ++e) s = fmaf(sv_dev::unpack<DT>(a, e), sv_dev::unpack<DT>(b, e), s);
        }
        for (int k = nv * W + lane; k < P.H; k += 64) s = fmaf(load_real<DT>(dst, k), load_real<DT>(w, k), s);
        s = wave_sum_f(s);
      }
      if (lane == 0) P.zt[(int64_t)at * TOP + j] = s * alpha;
    }
  }
}

// -------------------------------------------------------------------- products
struct Prod {
  const char *x;
  int64_t x_ld;
  const char *y;
  int64_t y_ld;
  int64_t v0;                            // first vocabulary entry
  int32_t M, N;                          // rows and columns of the result
  int32_t mt, nt, band, nk;
  int32_t tile0;                         // column tile of the row statistics at column 0
  int32_t first;
  // dx: chunks of a piece, steps of one; least steps of a workgroup, workgroups, tiles each may touch
  int32_t chunks, full, per0, groups, slots;
};

// The step with which a tile of few rows begins: by its place in the vocabulary, not in
// the piece, so that a logit's sum has one order however the vocabulary is cut, which
// depends on whether there are gradients (pieces are whole tiles).
template <class T> __device__ __forceinline__ int first_step(const Prod &G, int in) {
  return T::BM == 32 ? (int)((G.v0 / T::BN + in) % G.nk) : 0;
}

// Forward tile: each row's maximum m (base 2) and sum of 2^(z log2 e - m) over
// the tile's columns.  A NaN makes both NaN, +inf alone only the sum.  Bound by the
// matrix instructions (a rollout of 4096 rows of 4096 x 151936 in bf16, a quarter of
// them left out: 2.85 ms, 1.34 PFLOP/s; a library's product of 8192^3 reaches 1.43), and
// by reading the head where rows are few (24 rows 280 us, 4.4 TB/s).
template <int DT, class T> __global__ __launch_bounds__(T::TPB) void stats_kernel(Head P, Prod G) {
  __shared__ __align__(16) char lds[T::LDS];
  const int M = P.counts[1], mt = (M + T::BM - 1) / T::BM;
  if ((int)blockIdx.x >= mt * G.nt) return;
  int im, in;                            // (over the rows there are: each XCD gets its share of them)
  tile_at(run_of_xcd(blockIdx.x, mt * G.nt), mt, G.nt, G.band, im, in);
  const int m0 = im * T::BM, n0 = in * T::BN;
  typename Mma<DT>::Acc acc[T::FM][T::FN];
  clear<DT, T>(acc);
  const Part X = {G.x + (int64_t)m0 * G.x_ld, G.x_ld, M - m0 < T::BM ? M - m0 : T::BM, (int64_t)G.nk * STEP};
  const Part Y = {G.y + (int64_t)n0 * G.y_ld, G.y_ld, G.N - n0 < T::BN ? G.N - n0 : T::BN, (int64_t)G.nk * STEP};
  product<DT, T>(acc, lds, X, Y, 0, G.nk, first_step<T>(G, in));
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, wm = wid / T::WN, wn = wid % T::WN;
  __syncthreads();                       // the tiles are done with: their LDS takes the waves' results
  float2 *red = (float2 *)lds;           // [WN][BM]
#pragma unroll
  for (int f = 0; f < T::FM; ++f) {
    const int r = (wm * T::FM + f) * 16 + (lane & 15);
    const float a = m0 + r < M ? P.alpha[m0 + r] : 0.f;
    // cross entropy: the target's own z, where it lies in this tile
    const int64_t t = P.T == 1 && m0 + r < M ? P.targets[P.perm[m0 + r]] - G.v0 : -1;
    float m = NEG_INF;
#pragma unroll
    for (int g = 0; g < T::FN; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + (wn * T::FN + g) * 16 + (lane >> 4) * 4 + i;
        const float z = n < G.N ? acc[f][g][i] * a : NEG_INF;
        acc[f][g][i] = z;
        if (n == t) P.zt[m0 + r] = z;
        m = sv_dev::fmax_nan(m, z);
      }
    m = sv_dev::fmax_nan(m, __shfl_xor(m, 16));
    m = sv_dev::fmax_nan(m, __shfl_xor(m, 32));
    if constexpr (DT == SV_F32) {
      if (P.keep && m0 + r < M)
#pragma unroll
        for (int g = 0; g < T::FN; ++g)
          *(f32x4 *)(P.dz + (m0 + r) * P.dz_ld + (int64_t)(n0 + (wn * T::FN + g) * 16 + (lane >> 4) * 4) * 4) = acc[f][g];
    }
    const float hi = m == NEG_INF ? NEG_INF : m * LOG2E, ref = hi == NEG_INF ? 0.f : hi;
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < T::FN; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) s += __builtin_amdgcn_exp2f(fmaf(acc[f][g][i], LOG2E, -ref));
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lane < 16) red[wn * T::BM + r] = make_float2(hi, s);
  }
  __syncthreads();
  for (int r = threadIdx.x; r < T::BM; r += T::TPB) {
    if (m0 + r >= M) break;
    float2 t = red[r];
    for (int q = 1; q < T::WN; ++q) {
      const float2 o = red[q * T::BM + r];
      const float m = sv_dev::fmax_nan(t.x, o.x), ref = m == NEG_INF ? 0.f : m;
      t.y = t.y * __builtin_amdgcn_exp2f(t.x - ref) + o.y * __builtin_amdgcn_exp2f(o.x - ref);
      t.x = m;
    }
    P.part[(int64_t)(G.tile0 + in) * P.N + m0 + r] = t;
  }
}

// A fragment turned into blocks: a lane starts with four columns n .. n + 3 of its row
// m and ends with rows of one column.  Lanes whose rows differ in one bit swap what
// the other one keeps: rows 2j and 2j + 1, then rows two apart (fp32: 16 bytes now),
// and for bf16 then rows of the other half of eight, between two fragments.  That
// last swap mirrors the eight lanes, so lanes of the upper half keep their columns
// in mirrored order.
__device__ __forceinline__ uint32_t pick(bool b, uint32_t x, uint32_t y) { return b ? x : y; }
template <int CTRL> __device__ __forceinline__ uint32_t swap_lanes(uint32_t v) { return sv_dev::dpp<CTRL, 0xf, 0xf>(0u, v); }
constexpr int LANE_1 = 0xb1, LANE_2 = 0x4e, LANE_7 = 0x141;   // DPP: lane ^ 1, lane ^ 2, lane ^ 7

struct Turn {                            // the lane's bits, and the bits of the column it keeps
  bool b0, b1, b2, k0, k1;
  __device__ __forceinline__ Turn() {
    b0 = threadIdx.x & 1;
    b1 = threadIdx.x & 2;
    b2 = threadIdx.x & 4;
    k0 = b0 != b2;
    k1 = b1 != b2;
  }
  // bf16: rows (m & ~3) .. + 3 of column n + 2 k0 + k1
  __device__ __forceinline__ u32x2 four(uint32_t lo, uint32_t hi) const {
    const uint32_t mine = pick(k0, hi, lo), o = swap_lanes<LANE_1>(pick(k0, lo, hi));
    const uint32_t x = pick(b0, o, mine), y = pick(b0, mine, o);   // of the even row, of the odd one
    const uint32_t p = __builtin_amdgcn_perm(y, x, 0x05040100), q = __builtin_amdgcn_perm(y, x, 0x07060302);
    const uint32_t own = pick(k1, q, p), r = swap_lanes<LANE_2>(pick(k1, p, q));
    return u32x2{pick(b1, r, own), pick(b1, own, r)};
  }
  // bf16: rows (m & ~7) .. + 7 of that column of fragment g, in the upper half of g + 1
  __device__ __forceinline__ u32x4 eight(u32x2 g, u32x2 h) const {
    const uint32_t o0 = pick(b2, h[0], g[0]), o1 = pick(b2, h[1], g[1]);
    const uint32_t r0 = swap_lanes<LANE_7>(pick(b2, g[0], h[0])), r1 = swap_lanes<LANE_7>(pick(b2, g[1], h[1]));
    return u32x4{pick(b2, r0, o0), pick(b2, r1, o1), pick(b2, o0, r0), pick(b2, o1, r1)};
  }
  // fp32: rows (m & ~3) .. + 3 of column n + b0 + 2 b1
  __device__ __forceinline__ u32x4 four(const float (&d)[4]) const {
    uint32_t x[2], y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __float_as_uint(d[2 * i]), b = __float_as_uint(d[2 * i + 1]);
      const uint32_t mine = pick(b0, b, a), o = swap_lanes<LANE_1>(pick(b0, a, b));
      x[i] = pick(b0, o, mine);
      y[i] = pick(b0, mine, o);
    }
    const uint32_t r = swap_lanes<LANE_2>(pick(b1, x[0], x[1])), s = swap_lanes<LANE_2>(pick(b1, y[0], y[1]));
    return u32x4{pick(b1, r, x[0]), pick(b1, s, y[0]), pick(b1, x[1], r), pick(b1, y[1], s)};
  }
};

// Workgroup 0 of these: the loss terms, in order (a fixed run per thread, then the
// waves).  The others put the rows that the sum of dW runs over into blocks, with zeros for
// rows without a term of their own: those with a data error (their values may be NaN)
// and those up to a whole step.
// 256 threads, more leave; red: 4 in LDS.  Where there are gradients they are the last workgroups of
// the first piece's dz, which needs nothing of theirs: no launch of their own (4 to 5
// us of 24 rows' 73).
template <int DT> __device__ __forceinline__ void loss_part(const Head &P, int block, double *red) {
  if (threadIdx.x >= 256) return;
  if (block > 0) {
    constexpr int E = Mma<DT>::E, Q = STEP / E, B = 16 / E;
    const int at = B * (block - 1), M = P.counts[0], whole = (M + Q - 1) / Q * Q;
    if (at >= whole) return;
    bool on[B];
#pragma unroll
    for (int r = 0; r < B; ++r) on[r] = at + r < M && P.ga[at + r] != 0.f;
    const char *x = P.xs + at * P.x_ld;
    u32x4 *o = (u32x4 *)(P.xw + at / B * P.xw_ld);
    for (int k = threadIdx.x; k < (int)P.Kp; k += 256) {
      u32x4 v;
      if constexpr (DT == SV_BF16) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t a = on[2 * r] ? ((const uint16_t *)(x + 2 * r * P.x_ld))[k] : 0u;
          const uint32_t b = on[2 * r + 1] ? ((const uint16_t *)(x + (2 * r + 1) * P.x_ld))[k] : 0u;
          v[r] = a | b << 16;
        }
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = on[r] ? ((const uint32_t *)(x + r * P.x_ld))[k] : 0u;
      }
      o[k] = v;
      if (DT == SV_BF16 && P.terms > 1) ((u32x4 *)(P.xw + (at + whole) / B * P.xw_ld))[k] = v;
    }
    return;
  }
  const int M = P.counts[1], per = (M + 255) / 256;
  double s = 0.0;
  for (int i = threadIdx.x * per; i < M && i < (int)(threadIdx.x + 1) * per; ++i) s += P.term[i];
  s = wave_sum_d(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) P.loss[0] = (float)(((red[0] + red[1]) + red[2]) + red[3]);
}

// Backward tile of a piece: dz = u (2^(z log2 e - lse2)), rounded to the
// operands' type; zeros in the rows up to a whole step and in the columns up to a
// whole tile, so that both gradients can sum whole steps.  The product again: keeping
// the logits would be 2.5 GB at 4096 rows, and their reading and writing as long as a
// third of it.  The rollout of the forward tile: 3.4 ms, with 1.9 GB written for dx, dW.
template <int DT, class T, bool TERMS>
__global__ __launch_bounds__(T::TPB) void dz_kernel(Head P, Prod G) {
  __shared__ __align__(16) char lds[T::LDS];
  constexpr int Q = STEP / Mma<DT>::E;
  constexpr bool SPLIT = DT == SV_BF16 && T::BM == PAIR, TWO = SPLIT || TERMS;
  const int M = P.counts[0], Mp = SPLIT ? (M ? PAIR : 0) : (M + Q - 1) / Q * Q, mt = (Mp + T::BM - 1) / T::BM;
  if ((int)blockIdx.x >= G.mt * G.nt) {
    loss_part<DT>(P, blockIdx.x - G.mt * G.nt, (double *)lds);
    return;
  }
  if ((int)blockIdx.x >= mt * G.nt) return;
  int im, in;
  tile_at(run_of_xcd(blockIdx.x, mt * G.nt), mt, G.nt, G.band, im, in);
  const int m0 = im * T::BM, n0 = in * T::BN;
  typename Mma<DT>::Acc acc[T::FM][T::FN];
  clear<DT, T>(acc);
  if (m0 < M && n0 < G.N) {
    const Part X = {G.x + (int64_t)m0 * G.x_ld, G.x_ld, M - m0 < T::BM ? M - m0 : T::BM, (int64_t)G.nk * STEP};
    const Part Y = {G.y + (int64_t)n0 * G.y_ld, G.y_ld, G.N - n0 < T::BN ? G.N - n0 : T::BN, (int64_t)G.nk * STEP};
    product<DT, T>(acc, lds, X, Y, 0, G.nk, first_step<T>(G, in));
  }
  // rows from a term to the next
  const int64_t next = SPLIT ? PAIR : P.Np, next_w = SPLIT ? PAIR : Mp;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, wm = wid / T::WN, wn = wid % T::WN;
  const Turn turn;
  const Beside beside;
#pragma unroll
  for (int f = 0; f < T::FM; ++f) {
    const int m = m0 + (wm * T::FM + f) * 16 + (lane & 15);
    const bool on = m < M;
    const float a = on ? P.alpha[m] : 0.f, l2 = on ? P.lse2[m] : 0.f, ga = on ? P.ga[m] : 0.f;
    const int row = on ? P.perm[m] : 0;
    const float s = P.h_scale && on && ga != 0.f ? P.h_scale[row] : 1.f;
    // cross entropy: the target and u / T, which its dz has less
    const int64_t t = P.T == 1 && on ? P.targets[row] - G.v0 : -1;
    const float u = P.T == 1 && on ? (P.row_weight ? P.row_weight[row] : 1.f) * P.inv_t : 0.f;
    float d[T::FN][4];
#pragma unroll
    for (int g = 0; g < T::FN; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + (wn * T::FN + g) * 16 + (lane >> 4) * 4 + i;
        const float v = fmaf(__builtin_amdgcn_exp2f(fmaf(acc[f][g][i] * a, LOG2E, -l2)), ga, n == t ? -u : 0.f);
        d[g][i] = n < G.N && ga != 0.f ? v : 0.f;
      }
    const int n = n0 + wn * T::FN * 16 + (lane >> 4) * 4;
    if (P.gh && m < Mp) {
      if constexpr (DT == SV_BF16) {
#pragma unroll
        for (int g = 0; g < T::FN; g += 2)
#pragma unroll
          for (int k = 0; k < (TWO ? 2 : 1); ++k) {
            float r[2][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i / 4][i % 4] = k ? rest_of(d[g + i / 4][i % 4]) : d[g + i / 4][i % 4];
            *(u32x4 *)(P.dz + (m + k * next) * P.dz_ld + (int64_t)(n0 + (wn * T::FN + g) * 16 + beside.at) * 2) =
                Beside::eight(r[0], r[1]);
          }
      } else {
#pragma unroll
        for (int g = 0; g < T::FN; ++g) store4<DT>(P.dz + m * P.dz_ld, n + g * 16, d[g]);
      }
    }
    if (P.gw) {
      char *at = P.dzw + m / (16 / Mma<DT>::E) * P.dzw_ld;
      u32x4 o[T::FN];                    // bf16: every second one, and in the others what is left of it
#pragma unroll
      for (int g = 0; g < T::FN; ++g) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[g][i] *= s;
        if constexpr (DT == SV_F32) o[g] = turn.four(d[g]);
      }
      if constexpr (DT == SV_BF16) {
#pragma unroll
        for (int g = 0; g < T::FN; g += 2)
#pragma unroll
          for (int k = 0; k < (TWO ? 2 : 1); ++k) {
            float r[2][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i / 4][i % 4] = k ? rest_of(d[g + i / 4][i % 4]) : d[g + i / 4][i % 4];
            o[g + k] = turn.eight(turn.four(pack2(r[0][0], r[0][1]), pack2(r[0][2], r[0][3])),
                                  turn.four(pack2(r[1][0], r[1][1]), pack2(r[1][2], r[1][3])));
          }
        at += (n + 2 * turn.k0 + turn.k1 + 16 * turn.b2) * 16;
      } else {
        at += (n + turn.b0 + 2 * turn.b1) * 16;
      }
      if (m < Mp) {
#pragma unroll
        for (int g = 0; g < T::FN; g += DT == SV_BF16 ? 2 : 1) {
          *(u32x4 *)(at + g * 256) = o[g];
          if constexpr (TWO) *(u32x4 *)(at + next_w / 8 * P.dzw_ld + g * 256) = o[g + 1];
        }
      }
    }
  }
}

// The same from logits that the forward product kept: fp32 products are slow enough
// (154 TFLOP/s) that a piece's logits are worth their memory where the piece is all of
// the vocabulary.  A thread takes 4 rows x 4 columns (24 rows x 20000 6.6 us, most of it
// the launch).
__global__ __launch_bounds__(256) void dz_kept_kernel(Head P, Prod G) {
  const int M = P.counts[0], Mp = (M + 31) / 32 * 32;
  if ((int)blockIdx.x >= G.mt) {         // (G.mt: groups of rows)
    __shared__ double red[4];
    if (blockIdx.y == 0) loss_part<SV_F32>(P, blockIdx.x - G.mt, red);
    return;
  }
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4, r0 = blockIdx.x * 4;
  if (r0 >= Mp || c >= G.M) return;      // (G.M: columns in whole tiles)
  f32x4 w[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int m = r0 + r;
    const bool on = m < M;
    const float l2 = on ? P.lse2[m] : 0.f, ga = on ? P.ga[m] : 0.f;
    const int row = on ? P.perm[m] : 0;
    const float s = P.h_scale && on && ga != 0.f ? P.h_scale[row] : 1.f;
    const int64_t t = P.T == 1 && on ? P.targets[row] : -1;
    const float u = P.T == 1 && on ? (P.row_weight ? P.row_weight[row] : 1.f) * P.inv_t : 0.f;
    f32x4 *z = (f32x4 *)(P.dz + m * P.dz_ld + (int64_t)c * 4);
    f32x4 v = 0;
    if (ga != 0.f) v = *z;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float d = fmaf(__builtin_amdgcn_exp2f(fmaf(v[i], LOG2E, -l2)), ga, c + i == t ? -u : 0.f);
      v[i] = c + i < G.N && ga != 0.f ? d : 0.f;
    }
    *z = v;
    w[r] = v * s;
  }
  if (P.gw)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(f32x4 *)(P.dzw + (r0 >> 2) * P.dzw_ld + (int64_t)(c + i) * 16) = f32x4{w[0][i], w[1][i], w[2][i], w[3][i]};
}

// Distillation: dz at the stored entries of a piece, u (q - pt), over what the tiles
// stored there.  bf16: from the entries' own logits, as the tiles' u q was rounded.
// fp32: from the tiles' u q, whose logit is the one in the normaliser: where a few
// entries hold most of q, the roundings of two different sums of it do not cancel
// (24 rows of 512 x 20000 whose first four entries do: 1.7e-6 of dx, so 2.7e-7).
template <int DT> __global__ __launch_bounds__(256) void fix_kernel(Head P, Prod G) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int at = (int)(i / TOP), j = (int)(i - (int64_t)at * TOP);
  if (at >= P.counts[0]) return;
  const float ga = P.ga[at];
  if (ga == 0.f) return;
  const int64_t n = P.perm[at], c = P.tidx[n * TOP + j] - G.v0;
  if (c < 0 || c >= G.N || !(P.tval[n * TOP + j] > NEG_INF)) return;   // another piece, or padding
  constexpr int B = 16 / Mma<DT>::E;
  const float u = P.w[n] * P.pt[i], s = P.h_scale ? P.h_scale[n] : 1.f;
  char *const z = P.dz + at * P.dz_ld, *const zw = P.dzw + at / B * P.dzw_ld;
  if constexpr (DT == SV_F32) {          // (an entry stands once in a row)
    if (P.gh) store_real<DT>(z, c, load_real<DT>(z, c) - u);
    if (P.gw) store_real<DT>(zw, c * B + at % B, fmaf(-u, s, load_real<DT>(zw, c * B + at % B)));
  } else {
    // ga holds the normaliser's part beyond fp32, which is q's alone
    const float d = fmaf(__builtin_amdgcn_exp2f(fmaf(P.zt[i], LOG2E, -P.lse2[at])), ga, -u);
    if (P.gh) store_real<DT>(z, c, d);
    if (P.gw) store_real<DT>(zw, c * B + at % B, d * s);
    if (P.split || P.terms > 1) {
      const int64_t next = P.split ? PAIR : P.Np, next_w = P.split ? PAIR : (P.counts[0] + 63) / 64 * 64;
      if (P.gh) store_real<DT>(z + next * P.dz_ld, c, rest_of(d));
      if (P.gw) store_real<DT>(zw + next_w / B * P.dzw_ld, c * B + at % B, rest_of(d * s));
    }
  }
}

// How a piece's dx is shared out: its steps are cut into a few chunks (as many as
// workgroups share a tile, at most 8: then an XCD's workgroups take all tiles of the
// same entries, and dz and the weight are read into one L2 instead of eight: 1000 rows
// of 2048 x 151936 590 to 516 us, 180 of 4096 475 to 365); the steps of all tiles in a
// chunk in one line, cut into equal runs, one per workgroup, so that the chip is full
// whatever the number of tiles.  A run touches a few tiles and adds its part of each to
// a sum of its own (fp32, kept from piece to piece); a tile's sums are joined at the end.
// The rollout of the forward tile: 3.2 ms, 1.19 PFLOP/s; beside the matrix instructions
// the byte permutes that pair up the head's rows take the vector units' time.
struct Share {
  int nt, full, per, runs;               // column tiles, steps of a tile's chunk, of a run; runs of a chunk
  __device__ __forceinline__ Share(const Prod &G, int M, int bm) {
    nt = G.nt;
    full = G.full;
    runs = G.groups / G.chunks;
    const int64_t total = (int64_t)((M + bm - 1) / bm) * nt * full;
    const int64_t p = (total + runs - 1) / runs;
    per = (int)(p > G.per0 ? p : G.per0);
  }
};

// whether tile T of dx holds dz's two terms
template <int DT, class T> constexpr bool BOTH = DT == SV_BF16 && T::BM == 2 * PAIR;
// a wave's fragment rows of one term (the other's lie in the same wave), and a tile's sums
template <int DT, class T> constexpr int TERM = BOTH<DT, T> ? T::FM / 2 : T::FM;
template <int DT, class T> constexpr int SUM = T::BM * T::BN / (T::FM / TERM<DT, T>);

template <int DT, class T> __global__ __launch_bounds__(T::TPB) void dx_kernel(Head P, Prod G) {
  __shared__ __align__(16) char lds[T::LDS];
  const int M = BOTH<DT, T> ? (P.counts[0] ? 2 * PAIR : 0) : P.counts[0];
  const Share S(G, M, T::BM);
  const int mt = (M + T::BM - 1) / T::BM;
  const int64_t total = (int64_t)mt * S.nt * S.full;
  const int b = run_of_xcd(blockIdx.x, G.groups), c = b / S.runs;
  const int64_t at = (int64_t)(b - c * S.runs) * S.per;
  if (at >= total) return;
  int left = __builtin_amdgcn_readfirstlane((int)(at + S.per < total ? S.per : total - at));
  int t = __builtin_amdgcn_readfirstlane((int)(at / S.full)), from = __builtin_amdgcn_readfirstlane((int)(at % S.full));
  float *out = P.acc + (int64_t)b * G.slots * SUM<DT, T> + threadIdx.x * 4;
  for (; left > 0; ++t, from = 0, out += SUM<DT, T>) {
    int ns = left < S.full - from ? left : S.full - from;
    left -= ns;
    const int s0 = c * S.full + from;
    if (s0 + ns > G.nk) ns = G.nk - s0;  // the last chunk, a shorter last piece
    if (ns <= 0) {
      if (!G.first) continue;
      ns = 0;                            // its sum starts at zero all the same
    }
    int im, in;
    tile_at(t, mt, S.nt, G.band, im, in);
    const int m0 = im * T::BM, n0 = in * T::BN;
    typename Mma<DT>::Acc acc[T::FM][T::FN];
    clear<DT, T>(acc);
    const Part X = {G.x + (int64_t)m0 * G.x_ld, G.x_ld, M - m0 < T::BM ? M - m0 : T::BM, (int64_t)G.nk * STEP};
    const Part Y = {G.y + (int64_t)n0 * Mma<DT>::E, G.y_ld, G.M, (P.Kp - n0) * Mma<DT>::E};
    product<DT, T, ROWS, COLS>(acc, lds, X, Y, s0, ns);
#pragma unroll
    for (int f = 0; f < TERM<DT, T>; ++f)
#pragma unroll
      for (int g = 0; g < T::FN; ++g) {
        f32x4 *o = (f32x4 *)(out + (f * T::FN + g) * (T::TPB * 4));
        f32x4 v = acc[f][g];
        if constexpr (BOTH<DT, T>) v += acc[f + TERM<DT, T>][g];
        if (!G.first) v += *o;
        *o = v;
      }
    __syncthreads();                     // the tile's LDS is free for the next
  }
}

// dx of every row: its tile's sums in a fixed order, rounded once; zeros for rows
// without a gradient.  A workgroup per fragment row of a tile's wave: the tile's sums
// are added in RUNS runs, four loads under way at a time, shared out over WS waves, and
// the first wave joins them.  (Few rows have many sums of a few steps each: 128 at 24
// rows of 512 in fp32, which one run took 21 us for; tiles of 256 rows are about as
// many as workgroups and have few.)
template <class T> constexpr int RUNS = T::BM == 256 ? 1 : 8;
template <class T> using Runs = f32x4[RUNS<T> > 1 ? RUNS<T> - 1 : 1][T::FN][64];
template <int DT, class T, int WS>
__device__ __forceinline__ void dx_rows_part(const Head &P, const Prod &G, int block, Runs<T> &red) {
  const int M = P.counts[0], lane = threadIdx.x & 63, ws = threadIdx.x >> 6;
  constexpr int PER = T::NW * TERM<DT, T>;
  const int tile = block / PER, f = block % PER / T::NW, wid = block % T::NW;
  const int in = tile % G.nt, im = tile / G.nt, m0 = im * T::BM, n0 = in * T::BN;
  const int wm = wid / T::WN, wn = wid % T::WN;
  const int m = m0 + index_of<T::FM, ROWS>(wm, f, lane & 15);
  const Share S(G, M, T::BM);
  const int mt = (M + T::BM - 1) / T::BM, g = im / G.band, h = mt - g * G.band < G.band ? mt - g * G.band : G.band;
  const int64_t t = m0 < M ? (int64_t)g * G.band * G.nt + (int64_t)in * h + (im - g * G.band) : 0;
  const int b0 = (int)(t * S.full / S.per), b1 = (int)(((t + 1) * S.full - 1) / S.per);
  const int n = b1 - b0 + 1, all = m0 < M ? n * G.chunks : 0;   // sums: a chunk's, all
  const int run = (all + RUNS<T> - 1) / RUNS<T>;
  // in a run of dx that begins before the tile, the tile's sum lies behind those of its
  // other tiles; in the others it is the first
  const int k0 = (int)(t - (int64_t)b0 * S.per / S.full);
  const float *s = P.acc + f * T::FN * (T::TPB * 4) + (wid * 64 + lane) * 4;
  f32x4 v[T::FN];
#pragma unroll
  for (int p = RUNS<T> - WS + ws; p >= 0; p -= WS) {
#pragma unroll
    for (int q = 0; q < T::FN; ++q) v[q] = 0;
    const int first = p * run, end = first + run < all ? first + run : all;
    int c = first / n, r = first - c * n;
    for (int b = first; b < end; b += 4) {
      f32x4 o[4][T::FN];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t slot = (int64_t)(c * S.runs + b0 + r) * G.slots + (r == 0 ? k0 : 0);
        if (++r == n) { r = 0; ++c; }
#pragma unroll
        for (int q = 0; q < T::FN; ++q) {
          o[e][q] = 0;
          if (b + e < end) o[e][q] = *(const f32x4 *)(s + slot * SUM<DT, T> + q * (T::TPB * 4));
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int q = 0; q < T::FN; ++q) v[q] += o[e][q];
    }
    if (RUNS<T> > 1 && p > 0) {
#pragma unroll
      for (int q = 0; q < T::FN; ++q) red[p - 1][q][lane] = v[q];
    }
  }
  if constexpr (RUNS<T> > 1) {
    __syncthreads();
    if (ws > 0) return;
    for (int w = 0; w < RUNS<T> - 1; ++w)
#pragma unroll
      for (int q = 0; q < T::FN; ++q) v[q] += red[w][q][lane];
  }
  if (m >= P.N) return;
  if (m >= M || P.ga[m] == 0.f)
#pragma unroll
    for (int q = 0; q < T::FN; ++q) v[q] = 0;
  store_columns<DT, T::FN>(P.gh, (int64_t)P.perm[m] * P.H, n0 + index_of<T::FN, COLS>(wn, 0, (lane >> 4) * 4), P.H, v);
}

template <int DT, class T> __global__ __launch_bounds__(64 * RUNS<T>) void dx_rows_kernel(Head P, Prod G, int block0) {
  __shared__ Runs<T> red;
  dx_rows_part<DT, T, RUNS<T>>(P, G, block0 + blockIdx.x, red);
}

// dW of a piece: complete, in the weight's type.  The rollout of the forward tile: 2.95
// ms, 1.30 PFLOP/s; 750 rows of 2048 x 151936 500 us, of which its 622 MB take 120.
template <int DT, class T> __global__ __launch_bounds__(T::TPB) void dw_kernel(Head P, Prod G) {
  __shared__ __align__(16) char lds[T::LDS];
  int im, in;
  tile_at(run_of_xcd(blockIdx.x, G.mt * G.nt), G.mt, G.nt, G.band, im, in);
  const int m0 = im * T::BM, n0 = in * T::BN;
  typename Mma<DT>::Acc acc[T::FM][T::FN];
  clear<DT, T>(acc);
  constexpr int Q = STEP / Mma<DT>::E;
  const int nk = (P.counts[0] + Q - 1) / Q * P.terms;
  const Part X = {G.x + (int64_t)m0 * 16, G.x_ld, (int64_t)nk * (STEP / 16), G.x_ld - (int64_t)m0 * 16};
  const Part Y = {G.y + (int64_t)n0 * 16, G.y_ld, (int64_t)nk * (STEP / 16), G.y_ld - (int64_t)n0 * 16};
  product<DT, T, BLOCKS, BLOCKS>(acc, lds, X, Y, 0, nk);
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, wm = wid / T::WN, wn = wid % T::WN;
  char *out = P.gw + G.v0 * P.H * Mma<DT>::E;
  const Beside beside;
#pragma unroll
  for (int f = 0; f < T::FM; ++f) {
    const int m = m0 + index_of<T::FM, BLOCKS>(wm, f, lane & 15);
    if (m >= G.M) continue;
    const int64_t row = (int64_t)m * P.H;
    if constexpr (DT == SV_BF16) {
#pragma unroll
      for (int g = 0; g < T::FN; g += 2) {
        const float a[4] = {acc[f][g][0], acc[f][g][1], acc[f][g][2], acc[f][g][3]};
        const float b[4] = {acc[f][g + 1][0], acc[f][g + 1][1], acc[f][g + 1][2], acc[f][g + 1][3]};
        store8(out, row, n0 + index_of<T::FN, BLOCKS>(wn, g, 0) + beside.at, G.N, Beside::eight(a, b));
      }
    } else {
#pragma unroll
      for (int g = 0; g < T::FN; ++g) {
        const int n = n0 + index_of<T::FN, BLOCKS>(wn, g, (lane >> 4) * 4);
        const float v[4] = {acc[f][g][0], acc[f][g][1], acc[f][g][2], acc[f][g][3]};
        if (n + 4 <= G.N) {
          store4<DT>(out, row + n, v);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < G.N) store_real<DT>(out, row + n + i, v[i]);
        }
      }
    }
  }
}

// dW where all rows fit one step (64 in bf16, 32 in fp32): bound by writing it.  A
// wave keeps its 64 entries' dz in registers and runs along the hidden width, 64
// columns at a time; blocks come straight from memory, each lane's 16 bytes being a
// fragment's, so no LDS and no barrier stand between the stores (20000 x 1024 in
// bf16: 18 us through the tiled product).  The first `sums` workgroups join dx's sums
// (X), which saves that launch: 5 us of 24 rows' 75.
template <int DT, class T> __global__ __launch_bounds__(256) void dw_few_kernel(Head P, Prod G, int span, Prod X, int sums) {
  typedef typename Mma<DT>::Acc Acc;
  if ((int)blockIdx.x < sums) {
    __shared__ Runs<T> red;
    dx_rows_part<DT, T, 4>(P, X, blockIdx.x, red);
    return;
  }
  const int block = blockIdx.x - sums, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int nm = (G.M + 255) / 256, m0 = (block % nm) * 256 + (threadIdx.x >> 6) * 64;
  const int c0 = block / nm * span, c1 = c0 + span < G.N ? c0 + span : G.N;
  constexpr int Q = STEP / Mma<DT>::E;
  // 64-byte half steps with rows in them
  const int halves = P.counts[0] > Q / 2 || (P.split && P.counts[0]) ? 2 : P.counts[0] > 0 ? 1 : 0;
  if (m0 >= G.M) return;
  u32x4 x[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      x[h][f] = 0;                       // (dz has whole tiles of 256 entries)
      if (h < halves) x[h][f] = *(const u32x4 *)(G.x + (h * 4 + q) * G.x_ld + (int64_t)(m0 + f * 16 + i) * 16);
    }
  // the column of index j of fragment g: four lanes' 16-byte stores make 64 bytes of a row
  auto column = [](int g, int j) { return DT == SV_F32 ? g * 16 + j : g / 2 * 32 + j / 4 * 8 + g % 2 * 4 + j % 4; };
  char *out = P.gw + G.v0 * P.H * Mma<DT>::E;
  for (int c = c0; c < c1; c += 64) {
    Acc acc[4][4];
    u32x4 y[4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int g = 0; g < 4; ++g) acc[f][g] = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h >= halves) break;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (h && P.split) break;         // both terms meet the same rows
        const int n = c + column(g, i);
        y[g] = *(const u32x4 *)(G.y + (h * 4 + q) * G.y_ld + (int64_t)(n < G.N ? n : G.N - 1) * 16);
      }
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int g = 0; g < 4; ++g) Mma<DT>::mul(acc[f][g], y[g], x[h][f]);
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int m = m0 + f * 16 + i;
      if (m >= G.M) continue;
      const int64_t row = (int64_t)m * P.H;
#pragma unroll
      for (int g = 0; g < 4; g += DT == SV_BF16 ? 2 : 1) {
        const int n = c + column(g, 4 * q);
        if constexpr (DT == SV_BF16) {
          const f32x4 a = acc[f][g], b = acc[f][g + 1];
          const u32x4 v = {pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(b[0], b[1]), pack2(b[2], b[3])};
          store8(out, row, n, G.N, v);
        } else if (n + 4 <= G.N) {
          *(f32x4_any *)(out + (row + n) * 4) = acc[f][g];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < G.N) ((float *)out)[row + n + r] = acc[f][g][r];
        }
      }
    }
  }
}

// -------------------------------------------------------------- rows' results
// (m, s) of two parts of a row: the maximum in base 2 and the sum of 2^(. - m).  A NaN
// maximum stays; one of -infinity has no terms.
__device__ __forceinline__ void join(float &m, double &s, float om, double os) {
  const float t = sv_dev::fmax_nan(m, om), ref = fabsf(t) == __builtin_inff() ? 0.f : t;
  const float a = m == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(m - ref), b = om == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(om - ref);
  s = s * (double)a + os * (double)b;
  m = t;
}

// KL of a row over its stored entries, by a wave; l2: its normaliser.
__device__ __forceinline__ void kd_row(const Head &P, int at, int n, int F, double l2) {
  const int lane = threadIdx.x & 63;
  const float v = lane < TOP ? P.tval[(int64_t)n * TOP + lane] : NEG_INF;
  const int x = lane < TOP ? P.tidx[(int64_t)n * TOP + lane] : -1;
  const bool use = !F && v != NEG_INF && x != -1;
  const float mv = wave_max_f(use ? v : NEG_INF);
  const double a = use ? (double)v - (double)mv : 0.0;
  const double e = use ? exp(a) : 0.0;
  const double sv = wave_sum_d(e);
  const double pt = use ? e / sv : 0.0;
  double t = 0.0;
  if (use && pt > 0.0) t = pt * (a - log(sv) - ((double)P.zt[(int64_t)at * TOP + lane] - l2 * PER_LOG2E));
  const double kl = wave_sum_d(t);
  if (lane < TOP) P.pt[(int64_t)at * TOP + lane] = (float)pt;
  if (lane == 0) {
    const float w = P.w[n];
    P.rows[n] = F ? __builtin_nanf("") : (float)kl;
    if (P.status) P.status[n] = F;
    P.term[at] = (!F && w > 0.f) ? (double)w * kl : 0.0;
  }
}

// The normaliser of each row from its tiles and the row's results.  Lanes take (row,
// part of the tiles), waves take parts too, all joined in a fixed order; then one
// thread per row, and for the distillation one wave per row.  9 us at 4096 rows, 5 at
// 24: a chain of dependent steps, not bytes.
template <bool KD> __global__ __launch_bounds__(1024) void normaliser_kernel(Head P, int tiles, int per) {
  __shared__ float ms[16][64];
  __shared__ double ss[16][64], l2s[64];
  __shared__ int fs[64];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int M = P.counts[1], r0 = blockIdx.x * per;
  if (r0 >= M) return;
  const int r = lane & (per - 1), parts = 16 * (64 / per), q = wid * (64 / per) + lane / per;
  const int at = r0 + r;
  float m = NEG_INF;
  double s = 0.0;
  if (at < M)
#pragma unroll 4
    for (int t = q; t < tiles; t += parts) {
      const float2 v = P.part[(int64_t)t * P.N + at];
      join(m, s, v.x, (double)v.y);
    }
  for (int o = per; o < 64; o *= 2) join(m, s, __shfl_xor(m, o), __shfl_xor(s, o));
  if (lane < per) { ms[wid][r] = m; ss[wid][r] = s; }
  __syncthreads();
  if (threadIdx.x < (unsigned)per && at < M) {
    m = ms[0][r];
    s = ss[0][r];
    for (int w = 1; w < 16; ++w) join(m, s, ms[w][r], ss[w][r]);
    static_assert(SV_HEAD_NAN == SV_KD_NAN && SV_HEAD_POSINF == SV_KD_POSINF && SV_HEAD_EMPTY == SV_KD_EMPTY, "one set");
    int F = !(m == m) ? SV_HEAD_NAN : m == __builtin_inff() ? SV_HEAD_POSINF : m == NEG_INF ? SV_HEAD_EMPTY : 0;
    const double l2 = F ? 0.0 : (double)m + log2(s);
    const int n = P.perm[at];
    const float hi = (float)l2;
    P.lse2[at] = hi;
    float u;
    if constexpr (KD) {
      F |= P.flags[n];
      l2s[r] = l2;
      fs[r] = F;
      u = P.w[n];
    } else {
      u = P.row_weight ? P.row_weight[n] : 1.f;
      const double lse = l2 * PER_LOG2E;
      // (the target's logit is one of the normaliser's, so less than 0 is rounding)
      const double less = lse - (double)P.zt[at];
      const float nll = F ? __builtin_nanf("") : less < 0.0 ? 0.f : (float)less;
      P.rows[n] = nll;
      if (P.lse) P.lse[n] = F ? __builtin_nanf("") : (float)lse;
      if (P.status) P.status[n] = F;
      P.term[at] = (!F && u != 0.f) ? (double)u * (double)nll : 0.0;
    }
    if (P.grads) P.ga[at] = F ? 0.f : u * (float)(1.0 - (l2 - (double)hi) * LN2) * P.inv_t;
  }
  if constexpr (KD) {
    __syncthreads();
    for (int k = wid; k < per && r0 + k < M; k += 16) kd_row(P, r0 + k, P.perm[r0 + k], fs[k], l2s[k]);
  }
}

// The loss alone.
__global__ __launch_bounds__(256) void loss_kernel(Head P) {
  __shared__ double red[4];
  loss_part<SV_BF16>(P, 0, red);
}

// ------------------------------------------------------------------------ host
static_assert(Tile<8, 4, 2, 4>::BM == 256 && Tile<4, 4, 2, 2>::BM == 128 && Tile<2, 2, 2, 2>::BM == 64 &&
                  Tile<2, 2, 1, 4>::BM == 32 && Tile<4, 2, 1, 4>::BM == 2 * PAIR,
              "plan_for's bm");
typedef Tile<8, 4, 2, 4> Big;            // 256 x 256
typedef Tile<4, 4, 2, 2> Mid;            // 128 x 128
typedef Tile<2, 2, 2, 2> Square;         // 64 x 64
typedef Tile<2, 2, 1, 4> Few;            // 32 x 128
typedef Tile<4, 2, 1, 4> Pair;           // 64 x 128: dx of few rows in bf16
typedef Tile<1, 2, 2, 2> Narrow;         // 32 x 64

template <class T> Prod tiled(Prod G, int64_t M, int64_t N) {
  G.M = (int32_t)M;
  G.N = (int32_t)N;
  G.mt = (int32_t)cdiv(M, T::BM);
  G.nt = (int32_t)cdiv(N, T::BN);
  G.band = 8;
  return G;
}

template <int DT, class T, class TS = T> int enqueue(const Head &P, const Plan &L, bool kd, bool direct, hipStream_t st) {
  constexpr int E = Mma<DT>::E;
  const dim3 b256(256), b1024(1024);
  if (kd) hipLaunchKernelGGL(kd_rows_kernel, dim3((unsigned)cdiv(P.N, 4)), b256, 0, st, P);
  const bool find = P.N <= FIND_ROWS;
  auto stage = [&](auto KD) {
    constexpr bool kd = decltype(KD)::value;
    const dim3 rows(P.N), block(kd ? 1024 : 256);
    if (!find) hipLaunchKernelGGL((order_kernel<kd>), dim3(1), b1024, 0, st, P);
    if (P.h_scale && find) hipLaunchKernelGGL((stage_rows_kernel<SV_I8, DT, kd, true>), rows, block, 0, st, P);
    else if (P.h_scale) hipLaunchKernelGGL((stage_rows_kernel<SV_I8, DT, kd, false>), rows, block, 0, st, P);
    else if (find) hipLaunchKernelGGL((stage_rows_kernel<DT, DT, kd, true>), rows, block, 0, st, P);
    else hipLaunchKernelGGL((stage_rows_kernel<DT, DT, kd, false>), rows, block, 0, st, P);
  };
  if (kd) stage(std::true_type());
  else stage(std::false_type());

  Prod F = {};
  F.x = P.xs;
  F.x_ld = L.x_ld;
  F.nk = (int32_t)(L.Kp * E / STEP);
  auto weight_piece = [&](Prod &G, int64_t v0, int64_t cnt, bool copy) {
    G.v0 = v0;
    if (direct) {
      G.y = P.weight + v0 * P.w_ld;
      G.y_ld = P.w_ld;
    } else {
      if (copy) copy_rows(P.weight + v0 * P.w_ld, P.w_ld, (int64_t)P.H * E, P.wt, L.x_ld, L.Kp * E, cnt, st);
      G.y = P.wt;
      G.y_ld = L.x_ld;
    }
  };
  const int64_t fstep = direct ? P.V : L.piece;
  const int64_t most = sv_head_host::launch_columns(cdiv(P.N, TS::BM), TS::BN, TS::TPB);
  int tiles = 0;
  for (int64_t v0 = 0; v0 < P.V; v0 += fstep) {
    const int64_t cnt = P.V - v0 < fstep ? P.V - v0 : fstep;
    weight_piece(F, v0, cnt, true);
    // (logits that are kept are one piece of one launch: their columns count from its first)
    for (int64_t c = 0; c < cnt; c += most) {
      Prod G = tiled<TS>(F, P.N, cnt - c < most ? cnt - c : most);
      G.v0 = v0 + c;
      G.y += c * G.y_ld;
      G.tile0 = tiles;
      hipLaunchKernelGGL((stats_kernel<DT, TS>), dim3((unsigned)(G.mt * G.nt)), dim3(TS::TPB), 0, st, P, G);
      tiles += G.nt;
    }
  }
  // rows of a normaliser workgroup: a CU has one where that takes fewer than 64 (4096 rows 14.3
  // to 8.9 us, with the distillation's own part 24 to 11.6; 24 rows 9.1 to 6.5)
  int per = 1;
  while (per < 64 && per * (int64_t)sv_head_host::CUS < P.N) per *= 2;
  const dim3 ng((unsigned)cdiv(P.N, per));
  if (kd) hipLaunchKernelGGL((normaliser_kernel<true>), ng, b1024, 0, st, P, tiles, per);
  else hipLaunchKernelGGL((normaliser_kernel<false>), ng, b1024, 0, st, P, tiles, per);
  if (!P.grads) {
    hipLaunchKernelGGL(loss_kernel, dim3(1), b256, 0, st, P);
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
  }

  Prod X = tiled<T>(Prod{}, BOTH<DT, T> ? 2 * PAIR : P.N, P.H);
  X.x_ld = L.dz_ld;
  X.chunks = L.chunks;
  X.full = L.full;
  X.groups = L.groups;
  X.slots = L.slots;
  X.per0 = sv_head_host::RUN;
  constexpr bool FEW = T::BM == 32 || (DT == SV_BF16 && T::BM < 256);    // tiles that rows of one step take
  const bool few = FEW && P.gw && L.Np * E == STEP && P.terms == 1;
  const int64_t frags = (int64_t)X.mt * X.nt * T::NW * TERM<DT, T>;      // fragment rows of dx's tiles
  for (int64_t v0 = 0; v0 < P.V; v0 += L.piece) {
    const int64_t cnt = P.V - v0 < L.piece ? P.V - v0 : L.piece;
    const int64_t cp = sv_head_host::up(cnt, 256);       // columns of dz: whole tiles and steps
    Prod G = tiled<TS>(F, BOTH<DT, T> ? PAIR : L.Np, cp);
    weight_piece(G, v0, cnt, L.pieces > 1);              // (a single copied piece is still there)
    G.N = (int32_t)cnt;
    const int64_t loss = v0 ? 0 : P.gw ? L.Np * E / 16 + 1 : 1;
    if (P.keep) {
      G.M = (int32_t)cp;
      G.mt = (int32_t)(L.Np / 4);
      hipLaunchKernelGGL(dz_kept_kernel, dim3((unsigned)(G.mt + loss), (unsigned)cdiv(cp, 1024)), b256, 0, st, P, G);
    } else {
      auto dz = [&](auto terms) {
        constexpr bool TERMS = decltype(terms)::value;
        hipLaunchKernelGGL((dz_kernel<DT, TS, TERMS>), dim3((unsigned)(G.mt * G.nt + loss)), dim3(TS::TPB), 0, st, P, G);
      };
      if constexpr (DT == SV_BF16 && TS::BM > PAIR) {
        if (P.terms > 1) dz(std::true_type());
        else dz(std::false_type());
      } else {
        dz(std::false_type());
      }
    }
    if (kd) hipLaunchKernelGGL((fix_kernel<DT>), dim3((unsigned)cdiv((int64_t)P.N * TOP, 256)), b256, 0, st, P, G);
    if (P.gh) {
      X.y = G.y;
      X.y_ld = G.y_ld;
      X.M = (int32_t)cnt;
      X.nk = (int32_t)cdiv(cnt * E, STEP);
      for (int k = 0; k < P.terms; ++k) {
        X.x = P.dz + k * L.Np * L.dz_ld;
        X.first = v0 == 0 && k == 0;
        hipLaunchKernelGGL((dx_kernel<DT, T>), dim3((unsigned)L.groups), dim3(T::TPB), 0, st, P, X);
      }
    }
    if (P.gw) {
      Prod W = {};
      W.M = (int32_t)cnt;
      W.N = P.H;
      W.v0 = v0;
      W.x = P.dzw;
      W.x_ld = L.dzw_ld;
      W.y = P.xw;
      W.y_ld = L.xw_ld;
      if (few) {
        if constexpr (FEW) {             // (columns in parts that give every CU a few workgroups)
          const int64_t parts = cdiv(1024, cdiv(cnt, 256)), span = sv_head_host::up(cdiv(P.H, parts), 64);
          const int64_t sums = P.gh && v0 + cnt == P.V ? frags : 0;
          hipLaunchKernelGGL((dw_few_kernel<DT, T>), dim3((unsigned)(cdiv(cnt, 256) * cdiv(P.H, span) + sums)), b256, 0,
                             st, P, W, (int)span, X, (int)sums);
        }
      } else {
        auto product = [&](auto tile) {
          typedef decltype(tile) TW;
          const Prod Y = tiled<TW>(W, cnt, P.H);
          hipLaunchKernelGGL((dw_kernel<DT, TW>), dim3((unsigned)(Y.mt * Y.nt)), dim3(TW::TPB), 0, st, P, Y);
        };
        // by dW's own size: a small head would leave most CUs without one of the large tiles
        // (2772 rows of 192 x 4343: 42 us with 256, 23.5 with 128, 15.3 with 64; 4096 of 1024
        // x 8000, 504 tiles of 128: 57, and 77 with 64)
        if constexpr (DT == SV_BF16) {
          if (sv_head_host::large_tiles(cnt, P.H)) product(Big());
          else if (cdiv(cnt, 128) * cdiv(P.H, 128) >= sv_head_host::CUS) product(Mid());
          else product(Square());
        } else {
          product(Square());
        }
      }
    }
  }
  if (P.gh && !few) {
    constexpr int TPB = 64 * RUNS<T>;
    constexpr int64_t MOST = sv_head_host::max_groups(TPB);   // (2^20 rows of 4096 in fp32 are more)
    for (int64_t b = 0; b < frags; b += MOST)
      hipLaunchKernelGGL((dx_rows_kernel<DT, T>), dim3((unsigned)(frags - b < MOST ? frags - b : MOST)), dim3(TPB), 0, st, P,
                         X, (int)b);
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

int run(const sv_head_shape_t &s, bool kd, Head P, const void *hidden, const float *hidden_scale, const void *weight,
        void *gh, void *gw, void *workspace, hipStream_t st) {
  const bool direct = sv_head_host::weight_direct(&s, (uintptr_t)weight);
  const Plan L = sv_head_host::plan_for(&s, kd, direct);
  char *ws = (char *)workspace;
  const int he = sv_head_host::esize(s.hidden_dtype);
  P.N = s.N;
  P.H = s.H;
  P.V = s.V;
  P.T = kd ? TOP : 1;
  P.grads = s.grads & (SV_GRAD_HIDDEN | SV_GRAD_WEIGHT);
  P.ignore = s.ignore_index;
  P.inv_t = 1.f / s.temperature;
  P.Kp = L.Kp;
  P.x_ld = L.x_ld;
  P.dz_ld = L.dz_ld;
  P.keep = L.keep;
  P.split = s.dtype == SV_BF16 && L.bm == PAIR;
  P.terms = L.terms;
  P.Np = L.Np;
  P.hidden = (const char *)hidden;
  P.h_ld = (s.hidden_stride ? s.hidden_stride : s.H) * (int64_t)he;
  P.h_scale = s.hidden_dtype == SV_I8 ? hidden_scale : nullptr;
  P.weight = (const char *)weight;
  P.w_ld = (s.weight_stride ? s.weight_stride : s.H) * (int64_t)L.e;
  P.gh = (s.grads & SV_GRAD_HIDDEN) ? (char *)gh : nullptr;
  P.gw = (s.grads & SV_GRAD_WEIGHT) ? (char *)gw : nullptr;
  P.counts = (int32_t *)(ws + L.counts);
  P.perm = (int32_t *)(ws + L.perm);
  P.alpha = (float *)(ws + L.alpha);
  P.ga = (float *)(ws + L.ga);
  P.lse2 = (float *)(ws + L.lse2);
  P.w = (float *)(ws + L.w);
  P.flags = (int32_t *)(ws + L.flags);
  P.zt = (float *)(ws + L.zt);
  P.pt = (float *)(ws + L.pt);
  P.term = (double *)(ws + L.term);
  P.part = (float2 *)(ws + L.part);
  P.xs = ws + L.xs;
  P.dz = ws + L.dz;
  P.dzw = ws + L.dzw;
  P.xw = ws + L.xw;
  P.xw_ld = L.xw_ld;
  P.dzw_ld = L.dzw_ld;
  P.wt = ws + L.wt;
  P.acc = (float *)(ws + L.acc);
  // tiles by rows and entries (large_tiles); up to 32 rows 32 a tile, as the rest would
  // be multiplied in vain (33 to 64 rows of 4096 x 151936 in two of them 1340 to 1370 us
  // against 1240 to 1260), and where 128 columns a tile leave CUs without one, 64 do (24 x
  // 1024 x 20000: dz 12.3 to 10.8 us).  The fp32 matrix rate leaves time to read 64 x 64
  // tiles, which fill the chip sooner.
  if (s.dtype == SV_BF16)
    return L.bm == 256 ? enqueue<SV_BF16, Big>(P, L, kd, direct, st)
           : L.bm == 128 ? enqueue<SV_BF16, Mid>(P, L, kd, direct, st)
           : L.narrow    ? enqueue<SV_BF16, Pair, Narrow>(P, L, kd, direct, st)
                         : enqueue<SV_BF16, Pair, Few>(P, L, kd, direct, st);
  return L.bm == 64 ? enqueue<SV_F32, Square>(P, L, kd, direct, st)
         : L.narrow ? enqueue<SV_F32, Few, Narrow>(P, L, kd, direct, st)
                    : enqueue<SV_F32, Few>(P, L, kd, direct, st);
}

}  // namespace

extern "C" size_t sv_head_ce_workspace_bytes(const sv_head_shape_t *s) {
  if (!s || !sv_head_host::head_shape_ok(s, false)) return 0;
  return sv_head_host::head_bytes(s, false);
}

extern "C" size_t sv_head_kd_workspace_bytes(const sv_head_shape_t *s) {
  if (!s || !sv_head_host::head_shape_ok(s, true)) return 0;
  return sv_head_host::head_bytes(s, true);
}

extern "C" int sv_head_ce(const sv_head_shape_t *shape, const void *hidden, const float *hidden_scale,
                          const void *weight, const int32_t *targets, const float *row_weight, float *nll, float *lse,
                          int32_t *status, float *loss, void *grad_hidden, void *grad_weight, void *workspace,
                          size_t workspace_bytes, void *stream) {
  bool nothing;
  const int rc = sv_head_host::check_head(shape, false, hidden, hidden_scale, weight, targets, nullptr, nullptr,
                                          nullptr, nll, loss, grad_hidden, grad_weight, workspace, workspace_bytes,
                                          &nothing);
  if (rc != SV_OK || nothing) return rc;
  Head P = {};
  P.targets = targets;
  P.row_weight = row_weight;
  P.rows = nll;
  P.lse = lse;
  P.status = status;
  P.loss = loss;
  return run(*shape, false, P, hidden, hidden_scale, weight, grad_hidden, grad_weight, workspace, (hipStream_t)stream);
}

extern "C" int sv_head_kd(const sv_head_shape_t *shape, const void *hidden, const float *hidden_scale,
                          const void *weight, const float *topk_val, const int32_t *topk_idx,
                          const int32_t *row_sample, const float *rewards, float *kl, float *row_weight_out,
                          int32_t *status, float *loss, void *grad_hidden, void *grad_weight, void *workspace,
                          size_t workspace_bytes, void *stream) {
  bool nothing;
  const int rc = sv_head_host::check_head(shape, true, hidden, hidden_scale, weight, topk_val, topk_idx, row_sample,
                                          rewards, kl, loss, grad_hidden, grad_weight, workspace, workspace_bytes,
                                          &nothing);
  if (rc != SV_OK || nothing) return rc;
  Head P = {};
  P.tval = topk_val;
  P.tidx = topk_idx;
  P.row_sample = row_sample;
  P.rewards = rewards;
  P.S = shape->S;
  P.G = shape->group;
  P.w_max = shape->w_max;
  P.rows = kl;
  P.weight_out = row_weight_out;
  P.status = status;
  P.loss = loss;
  return run(*shape, true, P, hidden, hidden_scale, weight, grad_hidden, grad_weight, workspace, (hipStream_t)stream);
}
